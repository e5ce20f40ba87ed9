"""The "hooks" test build of the operators for several continuations: a wait of the tensor-core kernel that runs
out is reported and the context survives; block scans on a GPU that cannot hold their cluster."""
import time

import numpy as np
import pytest
import torch

import continuation_util as U
import test_gpu_pages as pages
import test_gpu_prefix_attn as prefix
import tree_speculative_decoding_03_gb300 as tsv
from oracle import continuations as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def hooks_lib():
    tsv.build(variant="hooks")
    lib = tsv.load("hooks")
    tsv.use_variant("hooks")
    yield lib
    lib.tsv_test_set_prefix_stall(0)
    lib.tsv_test_set_pages_cluster(1)
    tsv.use_variant(None)


# units of up to 128 rows, of more, several segments of a CTA
@pytest.mark.parametrize("members,prefix_lens", [([5], [700]), ([40, 3], [1500, 200]), ([4] * 60, [130] * 60)])
def test_a_wait_that_runs_out_is_reported(hooks_lib, members, prefix_lens):
    c = prefix.rounded(U.prefix_case(np.random.default_rng(1), members, prefix_lens, [3] * sum(members), 32, 4, 128, 16), torch.bfloat16)
    assert hooks_lib.tsv_test_set_prefix_stall(1) == 0
    d = prefix.on_device(c, torch.bfloat16)
    t0 = time.perf_counter()
    tsv.prefix_decode_attn(**d)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    err = d["seq_err"].cpu().numpy()
    assert (err & tsv.TSV_DERR_TIMEOUT).any() and not (err & ~tsv.TSV_DERR_TIMEOUT).any()
    flagged = err != 0
    assert torch.isnan(d["out"][torch.from_numpy(flagged).cuda()]).all()
    assert hooks_lib.tsv_test_set_prefix_stall(0) == 0
    tsv.prefix_decode_attn(**d)
    prefix.check(c, d)


@pytest.mark.parametrize("extra", [9000, 70000])
def test_scans_without_a_cluster(hooks_lib, extra):
    r = np.random.default_rng(extra)
    s = U.pages_state(r, 40, 8, 300, max_blocks=2000, extra=extra)
    keep = pages.releases(r, s, 8)
    a = pages.args(s)
    del a["seq_lens"]
    for on in (0, 1):
        hooks_lib.tsv_test_set_pages_cluster(on)
        pages.same(pages.run_release(s, keep, 8), C.release(keep, block_size=8, **a))
        pages.same(pages.run_compact(s), C.compact(s["table"], s["held"], s["shares"], s["free_blocks"]))
