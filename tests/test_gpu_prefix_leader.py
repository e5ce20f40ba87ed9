"""A group whose first sequence has ended (or is shorter than the prefix): its table row still names the shared blocks, which
the other sequences attend to; it alone is told that its length does not fit."""
import numpy as np
import pytest
import torch

import continuation_util as U
import test_gpu_prefix_attn as prefix
import tree_speculative_decoding_03_gb300 as tsv
from oracle import continuations as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("left", [0, 1, 255, -1])
def test_a_first_sequence_that_is_shorter_than_the_prefix(dtype, left):
    c = prefix.rounded(U.prefix_case(np.random.default_rng(left + 2), [6, 40, 1], [256, 300, 20], list(range(1, 48)), 8, 2, 64, 16), dtype)
    c["seq_lens"][0] = c["seq_lens"][6] = left
    d = prefix.on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    _, _, err = prefix.check(c, d)
    assert err.tolist() == [4] + [0] * 5 + [4] + [0] * 40
    # a block of the prefix outside the cache is everybody's, the first sequence's too
    c["table"][6, 3] = -1
    d = prefix.on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    out, lse, err = C.prefix_attn(**c)
    assert err.tolist() == [4] + [0] * 5 + [4] + [2] * 39 + [0]
    err[6] |= C.DERR_BLOCK
    prefix.check(c, d, (out, lse, err))
