"""The rotary K/V append against its fp64 oracle.

Bound of an element x' = x cos - y sin: the angle is within 2^-22 of a turn (2^-22 * 2 pi
radians), cos and sin are within 2^-22 of theirs, and three fp32 roundings add 3 * 2^-24, so
|error| <= (2^-22 (2 pi + 1) + 3 * 2^-24) (|x| + |y|) <= 2^-19 (|x| + |y|); a bf16 result is
rounded once more, by at most 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import serving as S
import serving_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def make(seed, T, Hq, Hkv, D, R, dtype, bs=16, sections=None, far=5000, fused=True, pad=0, blocks=None):
    r = np.random.default_rng(seed)
    sections = sections or [R // 2]
    x = r.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)
    nb = -(-max(T, 1) // bs) + 3 if blocks is None else blocks
    cache = r.standard_normal((2, nb, bs, Hkv, D)).astype(np.float32)
    if dtype == torch.bfloat16:
        x, cache = U.bf16_round(x), U.bf16_round(cache)
    pos = r.integers(0, far, (len(sections), T)).astype(np.int32)
    slots = r.permutation(nb * bs)[:T].astype(np.int64)
    slots[T - pad:] = -1
    inv = (10000.0 ** (-np.arange(R // 2) / (R // 2))).astype(np.float32)
    rows = torch.from_numpy(x).to(dtype).cuda()
    if fused:
        q, k, v = rows[:, :Hq], rows[:, Hq: Hq + Hkv], rows[:, Hq + Hkv:]
    else:
        q, k, v = (t.contiguous() for t in (rows[:, :Hq], rows[:, Hq: Hq + Hkv], rows[:, Hq + Hkv:]))
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    kc, vc = (cu(c).to(dtype) for c in cache)
    d = dict(q=q, k=k, v=v, positions=cu(pos if len(sections) > 1 else pos[0]), inv_freq=cu(inv),
             q_out=torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda"), k_cache=kc, v_cache=vc, slot_map=cu(slots),
             tok_err=torch.full((T,), -9, dtype=torch.int32, device="cuda"))
    host = dict(q=x[:, :Hq], k=x[:, Hq: Hq + Hkv], v=x[:, Hq + Hkv:], pos=pos, inv=inv, cache=cache, slots=slots, sections=sections)
    return d, host


def check(d, h, order, pairs, slots=None):
    torch.cuda.synchronize()
    bf = d["q_out"].dtype == torch.bfloat16
    slots = h["slots"] if slots is None else slots
    kc, vc = (d[n].float().cpu().numpy() for n in ("k_cache", "v_cache"))
    nb, bs, Hkv, D = kc.shape
    kc, vc = kc.reshape(-1, Hkv, D), vc.reshape(-1, Hkv, D)
    good = (slots >= 0) & (slots < nb * bs)
    R = 2 * len(h["inv"])

    def bound(x, want):
        size = np.abs(x.astype(np.float64))
        partner = np.zeros_like(size)
        if pairs == "halves":
            partner[..., : R // 2], partner[..., R // 2: R] = size[..., R // 2: R], size[..., : R // 2]
        else:
            partner[..., 0:R:2], partner[..., 1:R:2] = size[..., 1:R:2], size[..., 0:R:2]
        turned = 2.0 ** -19 * (size + partner)
        turned[..., R:] = 0.0
        return turned + (2.0 ** -8 * np.abs(want) if bf else 0.0) * (turned > 0)

    got = d["q_out"].float().cpu().numpy()
    want = S.rope(h["q"], h["pos"], h["inv"], h["sections"], order, pairs)
    assert (np.abs(got - want)[good] <= bound(h["q"], want)[good]).all()
    assert (got[slots < 0] == 0).all() and np.isnan(got[slots >= nb * bs]).all()
    want = S.rope(h["k"], h["pos"], h["inv"], h["sections"], order, pairs)
    assert (np.abs(kc[slots[good]] - want[good]) <= bound(h["k"], want)[good]).all()
    assert np.array_equal(vc[slots[good]], h["v"][good])
    # every other row of the caches is what it was
    rest = np.setdiff1d(np.arange(nb * bs), slots[good])
    old = h["cache"].reshape(2, -1, Hkv, D)
    assert np.array_equal(kc[rest], old[0][rest]) and np.array_equal(vc[rest], old[1][rest])
    assert np.array_equal(d["tok_err"].cpu().numpy(), np.where(slots >= nb * bs, tsv.TSV_DERR_BLOCK, 0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,kw", [
    (1, 8, 2, 128, 128, {}), (1, 1, 1, 64, 64, {}), (3, 5, 5, 64, 16, {}), (17, 12, 3, 128, 112, dict(pairs="neighbours")),
    (129, 8, 1, 128, 64, dict(sections=[5, 9, 18])), (300, 32, 8, 128, 128, dict(sections=[16, 24, 24], order="rounds")),
    (77, 7, 7, 64, 48, dict(sections=[0, 24], pairs="neighbours", order="rounds")), (640, 4, 4, 64, 32, dict(fused=False)),
    (1300, 3, 1, 128, 128, dict(sections=[1, 1, 1, 61], pad=13)), (2000, 9, 3, 64, 64, dict(far=2 ** 24)),
    (5, 64, 8, 128, 128, dict(pad=5)), (609, 2, 2, 128, 16, dict(bs=128))])
def test_rope(dtype, T, Hq, Hkv, D, R, kw):
    kw = dict(kw)
    order, pairs = kw.pop("order", "blocks"), kw.pop("pairs", "halves")
    d, h = make(T + D, T, Hq, Hkv, D, R, dtype, **kw)
    tsv.rope_kv_append(**d, sections=h["sections"], order=order, pairs=pairs)
    check(d, h, order, pairs)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_in_place_on_the_projections_rows(pairs):
    d, h = make(4, 200, 8, 2, 128, 96, torch.bfloat16)
    d["q_out"] = d["q"]
    keep = d["k"].clone(), d["v"].clone()
    tsv.rope_kv_append(**d, sections=h["sections"], pairs=pairs)
    check(d, h, "blocks", pairs)
    assert torch.equal(d["k"], keep[0]) and torch.equal(d["v"], keep[1])


def test_slots_outside_the_cache():
    d, h = make(6, 50, 4, 2, 64, 64, torch.bfloat16)
    slots = h["slots"].copy()
    slots[[3, 20, 49]] = [2 ** 40, d["k_cache"].shape[0] * 16, 2 ** 62]
    slots[[7, 8]] = [-1, -2 ** 62]
    d["slot_map"].copy_(torch.from_numpy(slots))
    tsv.rope_kv_append(**d)
    check(d, h, "blocks", "halves", slots)


def test_negative_and_farthest_positions():
    # past 2^24 the angle loses a bit for each doubling: 2^-22 turns become 2^-15 at 2^31
    T, D = 64, 64
    d, h = make(9, T, 2, 1, D, D, torch.float32)
    pos = np.concatenate([-np.arange(32) * 1000, 2 ** 31 - 1 - np.arange(32)]).astype(np.int64)
    h["pos"] = pos[None].astype(np.int32)
    d["positions"].copy_(torch.from_numpy(h["pos"][0]))
    tsv.rope_kv_append(**d)
    torch.cuda.synchronize()
    want = S.rope(h["q"], h["pos"], h["inv"], h["sections"])
    off = np.abs(d["q_out"].cpu().numpy() - want)
    size = np.abs(h["q"]).max()
    assert off[:32].max() <= 2.0 ** -19 * 2 * size and off[32:].max() <= 2.0 ** -15 * 7 * 2 * size


def test_infinities_stay_in_their_pairs():
    d, h = make(11, 4, 2, 1, 64, 32, torch.float32, fused=False)
    d["q"][1, 0, 3] = float("inf")
    d["q"][2, 1, 40] = float("nan")  # passes through
    tsv.rope_kv_append(**d)
    torch.cuda.synchronize()
    got = d["q_out"].cpu()
    bad = ~torch.isfinite(got)
    assert bad.nonzero().tolist() == [[1, 0, 3], [1, 0, 19], [2, 1, 40]]


def test_offsets_past_32_bits():
    # a cache of more than 2^32 bytes and 2^31 elements; the row is written far into it
    D, Hkv, bs = 128, 8, 16
    nb = 2 ** 31 // (bs * Hkv * D) + 50
    d, h = make(12, 3, 8, Hkv, D, D, torch.bfloat16, blocks=4)
    big = [torch.zeros(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([nb * bs - 1, nb * bs - 40, 5], device="cuda")
    d.update(k_cache=big[0], v_cache=big[1], slot_map=slots)
    tsv.rope_kv_append(**d)
    torch.cuda.synchronize()
    for t in range(3):
        assert torch.equal(big[1].view(-1, Hkv, D)[slots[t]], d["v"][t])
    assert int(big[1].view(-1, Hkv * D).ne(0).any(1).sum()) == 3


def test_captured_and_replayed():
    d, h = make(14, 40, 8, 2, 128, 128, torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tsv.rope_kv_append(**d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsv.rope_kv_append(**d)
    e, h2 = make(15, 40, 8, 2, 128, 128, torch.bfloat16)
    for k in ("positions", "slot_map", "k_cache", "v_cache"):
        d[k].copy_(e[k])
    for n in "qkv":
        d[n].copy_(e[n])
    g.replay()
    check(d, h2, "blocks", "halves")
