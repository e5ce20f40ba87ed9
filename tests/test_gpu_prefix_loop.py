"""Attention over shared prefixes where every CTA takes many tiles of a unit: maxima that rise along the keys, units of
more and of fewer than 128 rows one after the other, ends of a prefix inside a tile behind full ones.

A call has at least `TILES` 128-key tiles for each SM, and the tensor-core kernel no more CTAs than there are SMs, so a CTA
has at least that many in a row; of units of up to 128 rows each of its two softmax streams takes every other one.

Bounds: those of test_gpu_prefix_attn, with larger scores: a score is a sum of D products in fp32, off by at most
D 2^-24 of sum |q k| scale, and by that much in natural units its weight is off (relative); `score_bound` works it out."""
import numpy as np
import pytest
import torch

import test_gpu_prefix_attn as prefix
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu

TILES = 5


def tiles_of(c):
    members, (Hq, Hkv) = np.diff(c["group_offsets"]), (c["q"].shape[1], c["k_cache"].shape[2])
    rows = members * (Hq // Hkv)
    return int((-(-c["prefix_lens"] // 128) * -(-rows // 256)).sum()) * Hkv


def shared_case(r, members, lens, own, Hq, Hkv, D, bs, scale=None):
    """A case of continuation_util's form, with no blocks but the needed ones; slots outside the keys are NaN, table entries
    outside them anything."""
    G, B = len(members), sum(members)
    off = np.concatenate([[0], np.cumsum(members)]).astype(np.int32)
    of = np.repeat(np.arange(G), members)
    P = np.asarray(lens)
    L = P[of] + np.asarray(own)
    first = np.where(np.arange(B) == off[of], 0, P[of] // bs)  # the first block that is the sequence's own
    need = -(-L // bs)
    nb = int((need - first).clip(0).sum()) + 1
    table = r.integers(-5, nb + 5, (B, int(need.max()))).astype(np.int32)
    ids = r.permutation(nb)
    kc, vc = (np.full((nb, bs, Hkv, D), np.nan, np.float32) for _ in range(2))
    for b in range(B):
        n = max(int(need[b] - first[b]), 0)
        table[b, first[b]: need[b]], ids = ids[:n], ids[n:]
        t = np.arange(0 if b == off[of[b]] else P[of[b]], L[b])
        for x in (kc, vc):
            x[table[b, t // bs], t % bs] = r.standard_normal((len(t), Hkv, D))
    return dict(q=r.standard_normal((B, Hq, D)).astype(np.float32), k_cache=kc, v_cache=vc, table=table, seq_lens=L.astype(np.int32),
                group_offsets=off, prefix_lens=P.astype(np.int32), scale=scale or D ** -0.5)


def dense(c):
    """fp64, a sequence after the other: out, lse, and for each row sum |q k| scale at its largest and max |v|."""
    B, Hq, D = c["q"].shape
    bs, Hkv = c["k_cache"].shape[1:3]
    of = np.repeat(np.arange(len(c["prefix_lens"])), np.diff(c["group_offsets"]))
    out, lse, mass = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq, 1))
    for b in range(B):
        t = np.arange(c["seq_lens"][b])
        ids = c["table"][np.where(t < c["prefix_lens"][of[b]], c["group_offsets"][of[b]], b), t // bs]
        k, v = (np.moveaxis(c[n][ids, t % bs].astype(np.float64), 1, 0) for n in ("k_cache", "v_cache"))  # [Hkv, L, D]
        q = c["q"][b].astype(np.float64).reshape(Hkv, Hq // Hkv, D)
        z = q @ k.transpose(0, 2, 1) * c["scale"]
        m = z.max(-1, keepdims=True)
        w = np.exp(z - m)
        s = w.sum(-1, keepdims=True)
        lse[b], out[b] = (m + np.log(s)).reshape(Hq), (w @ v / s).reshape(Hq, D)
        mass[b] = (np.abs(q) @ np.abs(k).transpose(0, 2, 1)).max(-1).reshape(Hq, 1) * c["scale"]
    return out, lse, mass


def check(c, d):
    out, lse, mass = dense(c)
    assert not d["seq_err"].any()
    D, bf = c["q"].shape[2], d["out"].dtype == torch.bfloat16
    score_bound = D * 2.0 ** -24 * mass  # of a score, and so relative of a weight; 2^-13 besides for its parts and the sums
    top = np.nanmax(np.abs(c["v_cache"]))
    got, got_lse = d["out"].double().cpu().numpy(), d["lse"].double().cpu().numpy()
    tol = (2.0 ** -8 * np.abs(out) if bf else 0) + (2 * score_bound + 2.0 ** -13) * top
    assert (np.abs(got - out) <= tol).all(), (np.abs(got - out) / tol).max()
    assert (np.abs(got_lse - lse) <= 2.0 ** -14 * (1 + np.abs(lse)) + score_bound[..., 0]).all()
    return tol


def rising(c, r, per_tile):
    """Adds to every key a part along one direction, which the queries have too, so that a row's largest score rises by up to
    `per_tile` (in log2, some rows' not at all, some rows' falls) from a tile of 128 keys to the next."""
    D, bs = c["q"].shape[2], c["k_cache"].shape[1]
    u = r.choice([-1.0, 1.0], D)
    c["q"] += (u * r.choice([-1.0, 0.0, 0.4, 1.0, 1.0], c["q"].shape[:2])[..., None]).astype(np.float32)
    for g, b in enumerate(c["group_offsets"][:-1]):
        if c["group_offsets"][g + 1] == b:
            continue
        t = np.arange(c["prefix_lens"][g])
        step = per_tile * np.log(2.0) / (D * c["scale"])  # q . k rises by D times the factor of u
        c["k_cache"][c["table"][b, t // bs], t % bs] += (u * (step * (t / 128.0))[:, None])[:, None, :].astype(np.float32)
    return c


CASES = [  # members, prefix, Hq, Hkv, D, bs, rise of a tile: rows of a group and kv head are members * Hq / Hkv
    ([40] * 10, [1280, 1281, 1407, 1290, 1300] * 2, 32, 8, 128, 16, 9.0),     # 160 rows: two streams on the same tiles, rescaled at every tile
    ([60, 20, 64] * 4, [1000, 1409, 1664] * 4, 32, 8, 64, 32, 12.0),          # 240, 80 and 256 rows
    ([75, 70] * 4, [900, 769] * 4, 32, 8, 128, 64, 9.0),                      # 300 and 280 rows: units of 256 and of 44 and 24 in turn
    ([75] * 12, [385, 640, 511] * 4, 32, 8, 64, 8, 12.0),                     # the same with units of three to five tiles: CTAs cross them
    ([3] * 10, [1280, 1281, 1407, 1290, 1300] * 2, 32, 8, 128, 16, 9.0),      # 12 rows, 120 in all: one Q tile, rows twice in a tile
    ([30], [3201], 128, 32, 64, 128, 5.0),                                    # 120 rows: a stream on every other tile, one Q tile
    ([30, 1, 40, 2] * 3, [1200, 1025, 1153, 999] * 3, 24, 8, 128, 16, 9.0),   # 90, 3, 120 and 6 rows with two Q tiles
    ([40] * 10, [1280, 1281, 1407, 1290, 1300] * 2, 32, 8, 64, 16, 0.0),      # nothing rises
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_many_tiles_of_a_unit(i):
    members, lens, Hq, Hkv, D, bs, rise = CASES[i]
    r = np.random.default_rng(i)
    c = shared_case(r, members, lens, r.integers(0, 4, sum(members)), Hq, Hkv, D, bs)
    c = prefix.rounded(rising(c, r, rise), torch.bfloat16)
    assert tiles_of(c) >= TILES * torch.cuda.get_device_properties(0).multi_processor_count
    d = prefix.on_device(c, torch.bfloat16)
    tsv.prefix_decode_attn(**d)
    tol = check(c, d)
    assert np.median(tol) < 2.0 ** -6  # (V is standard normal)
    first = d["out"].clone()
    d["workspace"].fill_(0x41)  # finite floats
    tsv.prefix_decode_attn(**d)
    assert torch.equal(first, d["out"])


@pytest.mark.parametrize("members,D", [(40, 128), (30, 64)])
def test_infinite_values_behind_full_tiles(members, D):
    """A V row that is infinite under a weight of any size makes that element infinite, in whatever tile; V rows behind the
    prefix's end, in its last tile, make nothing."""
    r = np.random.default_rng(2)
    c = prefix.rounded(shared_case(r, [members], [12300], [1] * members, 32, 8, D, 16), torch.bfloat16)
    c["scale"] = 1.0 / 256
    assert tiles_of(c) >= TILES * torch.cuda.get_device_properties(0).multi_processor_count
    for t in (0, 700, 12299):
        c["v_cache"][c["table"][0, t // 16], t % 16, t % 8, t % D] = np.inf
    last = c["table"][0, 12300 // 16]
    c["k_cache"][last, 12300 % 16:], c["v_cache"][last, 12300 % 16:] = np.nan, np.inf
    c["k_cache"][c["table"][0, 12300 // 16], 12300 % 16], c["v_cache"][c["table"][0, 12300 // 16], 12300 % 16] = 0.5, 1.0  # its own key
    d = prefix.on_device(c, torch.bfloat16)
    tsv.prefix_decode_attn(**d)
    out = d["out"].float()
    assert not d["seq_err"].any()
    want = torch.zeros(32, D, dtype=torch.bool)
    for t in (0, 700, 12299):
        want[4 * (t % 8): 4 * (t % 8) + 4, t % D] = True
    inf = torch.isposinf(out).cpu()
    assert (inf == want).all() and torch.isfinite(out.cpu()[~want.expand_as(inf)]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("members,lens,Hq,Hkv,D", [([12, 5], [1024, 96], 8, 2, 128), ([40, 3], [4096, 2048], 32, 8, 64)])
def test_each_element_is_that_of_single_token_attention(dtype, members, lens, Hq, Hkv, D):
    """Two results, each within its bound of the exact one, on tables that hold the same blocks: element by element, so that a
    part of the keys that one of them leaves out shows (results of a thousand keys are some 0.05, a key's share far above the bound)."""
    r = np.random.default_rng(4)
    B = sum(members)
    c = prefix.rounded(shared_case(r, members, lens, r.integers(1, 50, B), Hq, Hkv, D, 16), dtype)
    d = prefix.on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    table = d["block_table"].clone()
    for g in range(len(members)):
        a, z = c["group_offsets"][g: g + 2]
        table[a:z, : lens[g] // 16] = table[a, : lens[g] // 16]
    ref, err, lse = torch.empty_like(d["out"]), torch.empty_like(d["seq_err"]), torch.empty_like(d["lse"])
    n = tsv.decode_attn_workspace_size(B, Hq, Hkv, D, 16, table.shape[1], tsv.TSV_BF16 if dtype == torch.bfloat16 else tsv.TSV_F32)
    tsv.decode_attn(d["q"], d["k_cache"], d["v_cache"], table, d["seq_lens"], ref, c["scale"],
                    workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), seq_err=err, lse=lse)
    assert not err.any() and not d["seq_err"].any()
    top = float(np.nanmax(np.abs(c["v_cache"])))
    ref = ref.double()
    # (the exact value is within the bound of ref)
    tol = 2 * (2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 2.0 ** -13 * top) if dtype == torch.bfloat16 else torch.full_like(ref, 2 * 2.0 ** -14 * top)
    assert ((d["out"].double() - ref).abs() <= tol).all()
    assert (tol < ref.abs()).double().mean() > 0.9  # a result of zero would not pass
    assert (d["lse"] - lse).abs().max() <= 2 * 2.0 ** -14 * (1 + lse.abs().max())
