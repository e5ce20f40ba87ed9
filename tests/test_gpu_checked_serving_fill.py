"""The second kernel of the slot plan in the checked test build: no index check fails, and the
outputs are the oracle's."""
import numpy as np
import pytest

import test_gpu_kv_plan as plan
import test_gpu_kv_plan_edges as edges
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked_lib():
    tsv.build(variant="checked")
    tsv.use_variant("checked")
    yield tsv.load("checked")
    tsv.use_variant(None)


@pytest.mark.parametrize("B,bs,max_len,max_new,kw", [
    (0, 16, 9, 3, {}), (1, 8, 9, 3, {}), (9, 16, 100, 0, dict(tree=15, ended=0.3)), (90, 16, 200, 20, dict(pool="short", ended=0.2)),
    (700, 16, 200, 250, dict(ended=0.2)), (6000, 8, 40, 0, dict(ended=0.2)), (70, 8, 40, 7, dict(pool="exact"))])
def test_filled_maps(B, bs, max_len, max_new, kw):
    c = edges.large(B, B, bs, max_len, max_new, past=1500, **kw)
    for in_place in (False, True):
        d = plan.device_plan(c, in_place=in_place)
        plan.call(d)
        plan.check(c, d)
