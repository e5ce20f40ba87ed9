"""Attention over shared prefixes against the fp64 oracle.

Bounds.  bf16: the result's rounding is 2^-8 of itself; a weight is within 2^-15 of itself, and its exponent and the sums
are fp32 (scores are off by D roundings of fp32 of sum |q k| scale, below 2^-14 here), which moves the result by at
most 2^-13 of sum p |v| <= max |v|.  fp32: the scores and sums alone, 2^-14 of max |v|.  lse: the score's bound."""
import numpy as np
import pytest
import torch

from oracle import continuations as C
import continuation_util as U
from serving_util import bf16_round
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def on_device(c, dtype):
    def t(x, dt=None):
        x = torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return x if dt is None else x.to(dt)

    B, Hq, D = c["q"].shape
    Hkv, bs = c["k_cache"].shape[2], c["k_cache"].shape[1]
    n = tsv.prefix_decode_attn_workspace_size(B, len(c["prefix_lens"]), Hq, Hkv, D, bs, c["table"].shape[1],
                                              tsv.TSV_BF16 if dtype == torch.bfloat16 else tsv.TSV_F32)
    return dict(q=t(c["q"], dtype), k_cache=t(c["k_cache"], dtype), v_cache=t(c["v_cache"], dtype), block_table=t(c["table"]),
                seq_lens=t(c["seq_lens"]), group_offsets=t(c["group_offsets"]), prefix_lens=t(c["prefix_lens"]),
                out=torch.full((B, Hq, D), 7.0, dtype=dtype, device="cuda"), scale=c["scale"],
                workspace=torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda"),
                seq_err=torch.full((B,), -9, dtype=torch.int32, device="cuda"), lse=torch.full((B, Hq), 7.0, device="cuda"))


def rounded(c, dtype):
    if dtype == torch.bfloat16:
        with np.errstate(invalid="ignore"):
            for n in ("q", "k_cache", "v_cache"):
                x = bf16_round(c[n])
                c[n] = np.where(np.isnan(c[n]), np.nan, x).astype(np.float32)
    return c


def check(c, d, want=None):
    out, lse, err = want or C.prefix_attn(**c)
    assert np.array_equal(d["seq_err"].cpu().numpy(), err)
    got, got_lse = d["out"].double().cpu().numpy(), d["lse"].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(out)) and np.array_equal(np.isnan(got_lse), np.isnan(lse))
    top = np.nanmax(np.abs(c["v_cache"])) if np.isfinite(c["v_cache"]).any() else 1.0
    bf = d["out"].dtype == torch.bfloat16
    tol = (2.0 ** -8 * np.abs(out) + 2.0 ** -13 * top) if bf else np.full(out.shape, 2.0 ** -14 * top)
    fine = ~np.isnan(out)
    assert (np.abs(got - out)[fine] <= tol[fine]).all(), (np.abs(got - out)[fine] / tol[fine]).max()
    flat = np.isinf(lse)
    assert np.array_equal(np.isinf(got_lse), flat)
    ok = ~flat & ~np.isnan(lse)
    assert (np.abs(got_lse[ok] - lse[ok]) <= 2.0 ** -14 * (1 + np.abs(lse[ok]))).all()
    return out, lse, err


CASES = [  # members, prefix, suffix, Hq, Hkv, D, bs
    ([1], [0], [1], 4, 4, 64, 8), ([1], [1], [0], 4, 2, 64, 8), ([2], [3], [0, 1], 8, 2, 128, 16), ([3], [16], [1, 2, 0], 8, 2, 64, 16),
    ([4], [130], [7, 1, 40, 16], 8, 8, 128, 16), ([2, 0, 3], [37, 9, 5], [1, 9, 30, 5, 2], 4, 2, 64, 8),
    ([9, 1, 16, 2], [513, 0, 255, 1000], list(range(28)), 16, 2, 128, 32), ([40], [777], [1] * 40, 8, 1, 64, 64),
    ([5, 3], [128, 2049], [300, 1, 0, 17, 129, 64, 63, 2], 28, 4, 128, 128), ([64], [300], list(range(64)), 8, 8, 64, 16),
    ([1] * 30, [0, 5, 60] * 10, list(range(30)), 6, 3, 128, 8), ([33], [4100], [3] * 33, 5, 5, 128, 16), ([7], [90], [1] * 7, 64, 1, 64, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(dtype, i):
    for cap in (0, 40000):
        c = rounded(U.prefix_case(np.random.default_rng(i), *CASES[i], cap=cap), dtype)
        d = on_device(c, dtype)
        tsv.prefix_decode_attn(**d)
        want = check(c, d)
        first = d["out"].clone()
        for _ in range(3):  # the same bits, whatever the workspace holds
            tsv.prefix_decode_attn(**{**d, "lse": None})
            assert torch.equal(first.nan_to_num(9.0), d["out"].nan_to_num(9.0))
    assert want is not None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_it_is_single_token_attention_on_joined_tables(dtype):
    c = rounded(U.prefix_case(np.random.default_rng(3), [12, 5], [1030, 96], [50] * 17, 8, 2, 128, 16), dtype)
    d = on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    # the same keys with a table row of each sequence's own (the shared part in whole blocks)
    table, off = d["block_table"].clone(), c["group_offsets"]
    kc, vc = d["k_cache"].clone(), d["v_cache"].clone()
    for g in range(2):
        full, rest = divmod(int(c["prefix_lens"][g]), 16)
        for b in range(off[g] + 1, off[g + 1]):
            table[b, :full] = table[off[g], :full]
            if rest:
                for x in (kc, vc):
                    x[table[b, full], :rest] = x[table[off[g], full], :rest]
    ref, err, lse = torch.empty_like(d["out"]), torch.empty_like(d["seq_err"]), torch.empty_like(d["lse"])
    n = tsv.decode_attn_workspace_size(17, 8, 2, 128, 16, table.shape[1], tsv.TSV_BF16 if dtype == torch.bfloat16 else tsv.TSV_F32)
    tsv.decode_attn(d["q"], kc, vc, table, d["seq_lens"], ref, c["scale"], workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"),
                    seq_err=err, lse=lse)
    assert not err.any() and not d["seq_err"].any()
    # two results within their bounds of the exact one
    top = float(np.nanmax(np.abs(c["v_cache"])))
    assert (d["out"].float() - ref.float()).abs().max() <= 2 * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -14) * top
    assert (d["lse"] - lse).abs().max() <= 2.0 ** -10


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,G", [(1023, 1), (1024, 1), (1500, 400), (2100, 2100)])
def test_many_sequences(dtype, B, G):
    """More items than the plan has threads, and just as many; groups of none to many."""
    r = np.random.default_rng(B)
    members = np.bincount(r.integers(0, G, B), minlength=G) if G > 1 else np.array([B])
    prefix = r.integers(0, 40, G) * (r.random(G) < 0.8)
    c = rounded(U.prefix_case(r, list(members), list(prefix), list(r.integers(0, 20, B)), 2, 1, 64, 8), dtype)
    d = on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    check(c, d)


def test_slots_past_32_bits():
    """Rows of the cache beyond 2^31 elements: one prefix and the sequences' own keys at its far end."""
    nb, bs, Hkv, D = 70000, 128, 4, 128  # 4.6e9 elements a cache
    kc, vc = (torch.zeros(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    r = np.random.default_rng(1)
    c = rounded(U.prefix_case(r, [3], [200], [5, 1, 140], 8, Hkv, D, bs), torch.bfloat16)
    d = on_device(c, torch.bfloat16)
    far = nb - len(c["k_cache"])
    kc[far:], vc[far:] = d["k_cache"], d["v_cache"]
    tsv.prefix_decode_attn(**{**d, "k_cache": kc, "v_cache": vc, "block_table": d["block_table"] + far})
    check(c, d)
    src, dst = torch.tensor([0, nb - 1], dtype=torch.int32, device="cuda"), torch.tensor([nb - 2, 1], dtype=torch.int32, device="cuda")
    kc[0], vc[0], kc[nb - 1] = 3.0, 5.0, 7.0
    err = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    tsv.kv_copy_blocks(kc, vc, src, dst, err)
    assert not err.any() and (kc[nb - 2] == 3).all() and (vc[nb - 2] == 5).all() and (kc[1] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_errors(dtype):
    c = rounded(U.prefix_case(np.random.default_rng(5), [3, 2, 2, 3], [40, 16, 24, 33], [5, 1, 9, 2, 30, 1, 1, 4, 20, 3], 8, 2, 64, 8), dtype)
    nb = len(c["k_cache"])
    c["table"][1, 5] = nb            # an own block of one sequence: [40, 49) is entry 5, 6
    c["table"][3, 1] = -1            # a shared block: the group of 3 and 4
    c["seq_lens"][5] = -1            # lengths
    c["seq_lens"][6] = 23            # shorter than its prefix
    c["seq_lens"][9] = c["table"].shape[1] * 8 + 1
    d = on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    want = check(c, d)
    assert want[2].tolist() == [0, 2, 0, 2, 2, 4, 4, 0, 0, 4]
    for bad in (-1, c["table"].shape[1] * 8 + 1, 2 ** 31 - 1):
        c["prefix_lens"][3] = bad
        d = on_device(c, dtype)
        tsv.prefix_decode_attn(**d)
        assert check(c, d)[2][7:].tolist() == [4, 4, 4]
    for off in ([1, 3, 5, 7, 10], [0, 3, 5, 7, 9], [0, 5, 3, 7, 10], [0, 3, 11, 7, 10], [0, -1, 5, 7, 10], [0, 3, 5, 2 ** 31 - 1, 10]):
        c["group_offsets"] = np.array(off, np.int32)
        d = on_device(c, dtype)
        tsv.prefix_decode_attn(**d)
        assert (check(c, d)[2] == C.DERR_SEQ).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_and_infinite_values(dtype):
    """Scores far apart (one key takes all), and V rows that are infinite under a positive weight."""
    c = U.prefix_case(np.random.default_rng(6), [3, 2], [200, 40], [30, 1, 2, 9, 300], 8, 2, 64, 16)
    c["q"] *= 40
    rounded(c, dtype)
    c["scale"] = 0.02
    d = on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    check(c, d)
    c["scale"] = 1.0 / 4000  # every weight is positive
    b, t = 0, 17
    c["v_cache"][c["table"][b, t // 16], t % 16] = np.inf
    d = on_device(c, dtype)
    tsv.prefix_decode_attn(**d)
    out, err = d["out"].float(), d["seq_err"]
    assert not err.any() and torch.isposinf(out[:3]).all() and torch.isfinite(out[3:]).all()


def test_no_sequences():
    c = U.prefix_case(np.random.default_rng(0), [0, 0], [5, 0], [], 4, 2, 64, 8)
    tsv.prefix_decode_attn(**on_device(c, torch.bfloat16))


def test_two_streams_with_a_workspace_each():
    cs = [rounded(U.prefix_case(np.random.default_rng(i), [6, 3], [900, 70], [20] * 9, 8, 2, 64, 16), torch.bfloat16) for i in range(2)]
    ds, streams = [on_device(c, torch.bfloat16) for c in cs], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(ds, streams):
            tsv.prefix_decode_attn(**d, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cs, ds):
        check(c, d)


def test_captured_with_lengths_that_change():
    """One capture serves later steps: the schedule follows the lengths on the device."""
    B, bs, mb = 9, 16, 64
    cs = [rounded(U.prefix_case(np.random.default_rng(i), m, p, s, 8, 2, 128, bs, cap=mb * bs), torch.bfloat16)
          for i, (m, p, s) in enumerate([([9], [800], list(range(9))), ([4, 5], [16, 300], [40] * 9), ([0, 9], [3, 5], [1] * 9)])]
    nb = max(len(c["k_cache"]) for c in cs)
    for c in cs:
        c["prefix_lens"], c["group_offsets"] = np.resize(c["prefix_lens"], 2), np.resize(c["group_offsets"], 3) if len(c["group_offsets"]) == 3 else \
            np.array([0, 9, 9], np.int32)
        for n in ("k_cache", "v_cache"):
            c[n] = np.concatenate([c[n], np.full((nb - len(c[n]), *c[n].shape[1:]), np.nan, np.float32)])
    d = on_device(cs[0], torch.bfloat16)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        tsv.prefix_decode_attn(**d)
    for c in cs + cs[:1]:
        e = on_device(c, torch.bfloat16)
        for n in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "group_offsets", "prefix_lens"):
            d[n].copy_(e[n])
        graph.replay()
        torch.cuda.synchronize()
        check(c, d)
