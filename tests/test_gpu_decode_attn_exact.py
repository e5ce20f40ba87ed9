"""Single-token attention where the exact result leaves no room: small score errors, so that the
rounding of the result is all that is left of the tolerance; infinite values; long caches of which
every key counts, and single keys far into them."""
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


LONG = [([20011], 8, 2, 128, 16), ([131071], 4, 1, 64, 64), ([4096] * 8, 32, 8, 128, 16), ([9000, 1, 4500, 0, 12345], 14, 2, 64, 8),
        ([17, 1, 16, 15, 33, 8191], 40, 1, 128, 16), ([3, 0, 40] * 70, 2, 2, 64, 16), ([2049, 3000, 77, 640] * 3, 12, 4, 128, 32)]


# With q = 0 every score is 0 and every weight 1, exactly (bf16: 255/256 + 1/256).  The values are whole
# numbers of at most 8, so all sums are exact in fp32 (multiples of 2^-8 below 2^16): l = L, and the
# numerator is the sum of the values.  lse = ln L within 2^-23 for the logarithm, 2 * 2^-24 for the
# factor ln 2 and its product; the result within 2 * 2^-24 for the division by multiplying and, in bf16,
# its rounding.  A key that is lost or taken twice moves lse by 1 / L: 7.6e-6 at the longest, where the
# tolerance is 3.1e-6.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [0, 150000])
@pytest.mark.parametrize("lens,Hq,Hkv,D,bs", LONG)
def test_every_key_counts_once(dtype, cap, lens, Hq, Hkv, D, bs):
    h = decode.make(80 + len(lens), lens, Hq, Hkv, D, bs, dtype, cap=cap)
    h["q"][:] = 0.0
    used = np.isfinite(h["vc"])
    h["vc"][used] = np.random.default_rng(81).integers(-8, 9, int(used.sum()))
    d = decode.on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    got, lse = d["out"].double().cpu().numpy(), d["lse"].double().cpu().numpy()
    assert not d["seq_err"].any()
    for b, L in enumerate(lens):
        if L == 0:
            continue
        rows = h["vc"][h["table"][b, : -(-L // bs)]].reshape(-1, Hkv, D)[:L].astype(np.float64)
        want = np.repeat(rows.sum(0), Hq // Hkv, 0) / L
        assert (np.abs(lse[b] - np.log(L)) <= 2.0 ** -22 * (np.log(L) + 1)).all(), (b, L)
        tol = 2.0 ** -21 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
        assert (np.abs(got[b] - want) <= tol * np.abs(want)).all(), (b, L)


# q = 8 k of one key: its score is 8 |k|^2 / sqrt(D), far above the others', so the result is that key's
# value.  `rest` is the weight of all others, small for these inputs (below 2^-12: asserted); scores are
# within (D + 8) u S < 2^-8 of theirs (S < 200), so the others' part of the result is below
# 2.01 rest max |v|, and what is left is the rounding of the result (and 2^-21 for the sum and the division).
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [0, 150000])
@pytest.mark.parametrize("L,D,bs", [(20011, 128, 16), (70001, 64, 64), (4099, 128, 8)])
def test_single_keys_of_a_long_cache(dtype, cap, L, D, bs):
    # sequences that share all their blocks, each with its own key: the first and last ones, the borders
    # of tiles and blocks, and some in between
    at = [0, 1, 7, 8, 15, 16, 31, 32, 63, 64, L // 3, L // 2, L - 17, L - 16, L - 2, L - 1]
    at += list(np.random.default_rng(5).integers(0, L, 16))
    one = decode.make(90, [L], 1, 1, D, bs, dtype, cap=cap)
    B = len(at)
    order = one["table"][0, : -(-L // bs)]
    k, v = (one[n][order].reshape(-1, D)[:L] for n in ("kc", "vc"))
    h = dict(one, q=(8.0 * k[at])[:, None], table=np.repeat(one["table"], B, 0), lens=np.full(B, L, np.int32))
    d = decode.on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    got = d["out"].double().cpu().numpy()[:, 0]
    assert not d["seq_err"].any()
    for b, t in enumerate(at):
        s = h["scale"] * (k.astype(np.float64) @ h["q"][b, 0].astype(np.float64))
        rest = np.exp(np.delete(s, t) - s[t]).sum()
        assert rest < 2.0 ** -12 and s[t] < 200
        tol = 2.01 * rest * np.abs(v).max() + (2.0 ** -21 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)) * np.abs(v[t])
        assert (np.abs(got[b] - v[t]) <= tol).all(), (t, L)
