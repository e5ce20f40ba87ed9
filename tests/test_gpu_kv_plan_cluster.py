"""The slot plan on a GPU that cannot hold its cluster: the "hooks" test build treats clusters above a
given size as not resident, and the smaller cluster or the single CTA gives the same."""
import numpy as np
import pytest

import serving_util as U
import test_gpu_kv_plan as plan
import test_gpu_kv_plan_edges as edges
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def hooks_lib():
    tsv.build(variant="hooks")
    lib = tsv.load("hooks")
    tsv.use_variant("hooks")
    yield lib
    lib.tsv_test_set_plan_cluster(16)
    tsv.use_variant(None)


@pytest.mark.parametrize("most", [16, 15, 8, 7, 1])
@pytest.mark.parametrize("B,bs,max_len,max_new,kw,past", [
    (257, 16, 700, 60, dict(ended=0.2, pad=37), 0), (64, 16, 2000, 0, dict(tree=64), 0), (8192, 8, 60, 5, dict(ended=0.1, pool="short"), 0),
    (900, 16, 300, 250, dict(ended=0.2), 1), (40, 16, 300, 80, dict(pool="short"), 5000), (300, 16, 200, 0, dict(tree=33, pool="exact"), 1), (0, 16, 9, 9, {}, 9)])
def test_smaller_clusters(hooks_lib, most, B, bs, max_len, max_new, kw, past):
    hooks_lib.tsv_test_set_plan_cluster(most)
    c = U.plan_case(np.random.default_rng(B), B, bs, max_len, max_new, **kw)
    if past:
        c["max_tokens"] = max(c["max_tokens"], edges.CLUSTER_TOKENS + past)
    edges.run_both(c)


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
import serving_util as U, test_gpu_kv_plan as plan
for B, pad in ((300, 0), (300, 70000), (8, 0)):
    c = U.plan_case(np.random.default_rng(B + pad), B, 16, 200, 9, ended=0.2, pad=pad)
    d = plan.device_plan(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.call(d)
    g.replay()
    plan.check(c, d)
print("captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    # the look-up of the cluster's size and the kernels' limits happen inside the capture
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(here), tests=here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
