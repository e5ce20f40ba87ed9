"""Single-token attention where the exact result leaves no room: small score errors, so that the
rounding of the result is all that is left of the tolerance; infinite values."""
import numpy as np
import pytest
import torch

import test_gpu_decode_attn as decode
from oracle import serving as S
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


# Bound of a bf16 result, element by element, with u = 2^-24, A = sum_t p_t |v_t| and S the largest
# scale * sum_i |q_i k_i| of a row (small here: q is small).  A weight is off by (D + 8) u S from its
# score, 2^-21 from the exponential and 2^-15 from its two bf16 parts; the sum of the weights has the
# first two as well.  Both sums take at most two products of 16 keys for each 16 keys, each within 2 u
# of its terms' size, and 64 u for the join and the division.  So before its own rounding the
# result is within d = A (2 ((D + 8) u S + 2^-21) + 2^-15 + 2 (4 ceil(L / 16) + 64) u), and after
# it within d + 2^-8 (|result| + d).  (Weights in one bf16 part would be up to 2^-8 off.)
@pytest.mark.parametrize("cap", [0, 50000])
@pytest.mark.parametrize("lens,Hq,Hkv,D,bs", [
    ([5, 100, 0, 63], 8, 2, 128, 16), ([100, 17, 200], 6, 2, 64, 8), ([129, 90], 32, 1, 128, 16), ([70, 33, 1], 40, 1, 64, 32),
    ([300] * 9, 16, 4, 128, 16), ([1000, 40], 8, 8, 64, 64)])
def test_bf16_result_is_off_by_its_own_rounding(lens, Hq, Hkv, D, bs, cap):
    h = decode.make(60 + len(lens) + Hq, lens, Hq, Hkv, D, bs, torch.bfloat16, cap=cap, size=0.05)
    d = decode.on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    out, _, err, mass = S.decode_attn(h["q"], h["kc"], h["vc"], h["table"], h["lens"], h["scale"])
    assert not err.any() and not d["seq_err"].any()
    got = d["out"].float().cpu().numpy()
    u = 2.0 ** -24
    for b, L in enumerate(lens):
        if L == 0:
            continue
        rows = h["kc"][h["table"][b, : -(-L // bs)]].reshape(-1, Hkv, D)[:L]
        big = np.array([h["scale"] * (np.abs(rows[:, i * Hkv // Hq]) @ np.abs(h["q"][b, i])).max() for i in range(Hq)])
        off = mass[b] * (2 * ((D + 8) * u * big + 2.0 ** -21) + 2.0 ** -15 + 2 * (4 * (-(-L // 16)) + 64) * u)[:, None]
        assert (np.abs(got[b] - out[b]) <= off + 2.0 ** -8 * (np.abs(out[b]) + off)).all(), (b, L)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [1, 40, 2500])
@pytest.mark.parametrize("cap", [0, 50000])
def test_infinite_values_stay_infinite(dtype, L, cap):
    # every key has a weight of about 1 / L: an infinite value is its column's result, in its head alone
    h = decode.make(71, [L, L], 4, 2, 64, 16, dtype, cap=cap, size=0.05)
    t = L // 2
    where = h["table"][0, t // 16], t % 16
    h["vc"][where][0, 7], h["vc"][where][0, 8] = np.inf, -np.inf
    d = decode.on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    got = d["out"].float().cpu().numpy()
    assert (got[0, :2, 7] == np.inf).all() and (got[0, :2, 8] == -np.inf).all()
    got[0, :2, 7:9] = 0.0
    assert np.isfinite(got).all() and torch.isfinite(d["lse"]).all() and not d["seq_err"].any()
