"""The rotary K/V append at every number of tokens a block takes (few heads and many tokens: 8 and
more), with ragged last blocks, far positions and frequencies above one."""
import numpy as np
import pytest
import torch

import test_gpu_rope_append as rope
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def tokens_a_block(T, Hq, Hkv, D, dtype):
    """The launch's rule, as its comment states it: up to 8 tokens while a thread has at most 8 heads,
    more while it has two, and at least three blocks an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lanes, heads, tok = 256 * (16 if dtype == torch.bfloat16 else 8) // D, Hq + 2 * Hkv, 1
    while 2 * tok <= lanes and T >= 3 * sms * 2 * tok and (heads * 2 * tok <= 8 * lanes if tok < 8 else heads * tok < 2 * lanes):
        tok *= 2
    return tok


CASES = [(3701, 4, 1, 128), (3700, 2, 2, 64), (7301, 1, 1, 128), (7333, 8, 1, 64), (14603, 1, 1, 64), (14601, 1, 1, 128), (29207, 1, 1, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("T,Hq,Hkv,D", CASES)
def test_many_tokens_of_few_heads(dtype, pairs, T, Hq, Hkv, D):
    R = D if T % 2 else D // 2
    d, h = rope.make(T + D, T, Hq, Hkv, D, R, dtype, far=2 ** 24, pad=T % 7, sections=[R // 8, 3 * R // 8] if T % 3 else None)
    tsv.rope_kv_append(**d, sections=h["sections"], order="rounds", pairs=pairs)
    rope.check(d, h, "rounds", pairs)


def test_the_cases_cover_the_rule():
    # every power of two from 8 to the largest a block can take, in both types
    for dtype, most in ((torch.bfloat16, 64), (torch.float32, 32)):
        seen = {tokens_a_block(*c, dtype) for c in CASES}
        assert {t for t in (8, 16, 32, 64) if t <= most} <= seen, (dtype, seen)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_frequencies_above_one(dtype):
    # the bound holds while position * inv_freq is below 2^24
    T, D = 500, 128
    d, h = rope.make(21, T, 4, 1, D, D, dtype, far=160000)
    h["inv"] = (h["inv"] * np.float32(100.0)).astype(np.float32)
    d["inv_freq"].copy_(torch.from_numpy(h["inv"]))
    tsv.rope_kv_append(**d)
    rope.check(d, h, "blocks", "halves")
