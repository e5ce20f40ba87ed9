"""The "hooks" test build: what a wait of the tensor-core kernel that runs out takes with it.  A CTA goes through many
groups; from the one in which a wait gives up to its last, none is complete, and the sequences of all of them are told.
Sequences that are not told have right results, whatever the workspace held."""
import time

import numpy as np
import pytest
import torch

import test_gpu_prefix_attn as prefix
import test_gpu_prefix_loop as loop
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def hooks_lib():
    tsv.build(variant="hooks")
    lib = tsv.load("hooks")
    tsv.use_variant("hooks")
    yield lib
    lib.tsv_test_set_prefix_stall(0)
    tsv.use_variant(None)


# members, prefix lengths, heads: units of few rows, of more than 128 (both streams on a tile), of two row groups
@pytest.mark.parametrize("members,lens,Hq,Hkv,D", [([1, 2, 0, 3] * 500, [100, 0, 7, 65, 128, 17, 3, 90] * 250, 4, 1, 64),
                                                   ([40] * 60, [70, 129, 0, 300, 128] * 12, 32, 8, 128), ([75] * 40, [10, 600, 128, 300] * 10, 32, 8, 64)])
@pytest.mark.parametrize("tile", [1, 2, 5])
def test_every_group_that_a_stalled_cta_loses_is_told(hooks_lib, members, lens, Hq, Hkv, D, tile):
    """The wait for the `tile`-th tile of each CTA's first stream runs out."""
    r = np.random.default_rng(tile)
    B = sum(members)
    c = prefix.rounded(loop.shared_case(r, members, lens, r.integers(1, 4, B), Hq, Hkv, D, 8), torch.bfloat16)
    out, lse, _ = loop.dense(c)
    d = prefix.on_device(c, torch.bfloat16)
    d["workspace"].fill_(0x41)  # finite floats
    assert hooks_lib.tsv_test_set_prefix_stall(tile) == 0
    t0 = time.perf_counter()
    tsv.prefix_decode_attn(**d)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert hooks_lib.tsv_test_set_prefix_stall(0) == 0
    got = d["seq_err"].cpu().numpy()
    told = got == tsv.TSV_DERR_TIMEOUT
    assert (told | (got == 0)).all() and told.any()
    shared = np.repeat(np.asarray(lens) > 0, members)
    assert not told[~shared].any()  # nothing of theirs is on the tensor cores
    if tile == 1:
        assert told[shared].all()  # every CTA's first tile
    elif Hkv == 1:  # (with more heads every group is on a CTA that has a `tile`-th)
        assert not told[shared].all()
    x, x_lse = d["out"].double().cpu().numpy(), d["lse"].double().cpu().numpy()
    assert np.isnan(x[told]).all() and np.isnan(x_lse[told]).all()
    top = np.nanmax(np.abs(c["v_cache"]))
    assert (np.abs(x - out)[~told] <= (2.0 ** -8 * np.abs(out) + 2.0 ** -13 * top)[~told]).all()
    assert (np.abs(x_lse - lse)[~told] <= 2.0 ** -14 * (1 + np.abs(lse))[~told]).all()
    tsv.prefix_decode_attn(**d)
    prefix.check(c, d, (out, lse, np.zeros(B, np.int32)))
