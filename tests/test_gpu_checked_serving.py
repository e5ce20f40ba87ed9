"""The serving operators in the checked test build (every global access through a computed
index is compared with its buffer's extent first): small cases on edge inputs give the
oracle's results, and no check fails."""
import numpy as np
import pytest
import torch

import serving_util as U
import test_gpu_decode_attn as decode
import test_gpu_kv_plan as plan
import test_gpu_rope_append as rope
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked_lib():
    tsv.build(variant="checked")
    tsv.use_variant("checked")
    yield tsv.load("checked")
    tsv.use_variant(None)


@pytest.mark.parametrize("B,bs,max_len,max_new,kw", [
    (1, 8, 9, 3, {}), (9, 16, 100, 0, dict(tree=15, ended=0.3)), (90, 16, 200, 20, dict(pool="short", ended=0.2)),
    (900, 16, 200, 60, dict(ended=0.2)), (70, 8, 40, 7, dict(pool="exact", pad=9))])
def test_plan(B, bs, max_len, max_new, kw):
    c = U.plan_case(np.random.default_rng(B), B, bs, max_len, max_new, **kw)
    for in_place in (False, True):
        d = plan.device_plan(c, in_place=in_place)
        plan.call(d)
        plan.check(c, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(dtype):
    d, h = rope.make(2, 33, 6, 3, 64, 48, dtype, sections=[9, 15], pad=4)
    tsv.rope_kv_append(**d, sections=h["sections"], order="rounds", pairs="neighbours")
    rope.check(d, h, "rounds", "neighbours")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [0, 9000])
@pytest.mark.parametrize("lens,Hq,Hkv,D,bs", [([1, 0, 17], 4, 2, 64, 8), ([700, 33, 129], 8, 4, 128, 16), ([64] * 50, 40, 1, 64, 32)])
def test_decode(dtype, cap, lens, Hq, Hkv, D, bs):
    h = decode.make(3, lens, Hq, Hkv, D, bs, dtype, cap=cap)
    d = decode.on_device(h)
    tsv.decode_attn(**d)
    decode.check(h, d)
