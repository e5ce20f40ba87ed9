"""Single-token attention against its fp64 oracle.

Bounds, element by element, with A = sum_t p_t |v_t| (the oracle's `mass`), S = the largest
scale * sum_i |q_i k_i| of a row, and u = 2^-24: a score is within (D + 8) u S of its value
and the exponential within 2^-21, so the weights and the lse are within e = 2 (D + 8) u S +
2^-20; sums over L keys add (L + 64) u.  fp32: |error| <= A (2 e + (L + 64) u).  bf16: the
weights are rounded by 2^-8 each and the result by 2^-8 of it: A (2^-7 + 2 e + (L + 64) u)."""
import numpy as np
import pytest
import torch

from oracle import serving as S
import serving_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def make(seed, lens, Hq, Hkv, D, bs, dtype, cap=0, size=1.0, spare=3):
    """Caches whose unused slots and blocks are NaN, a table whose unused entries are anything."""
    r = np.random.default_rng(seed)
    B = len(lens)
    lens = np.asarray(lens, np.int32)
    blocks = -(-lens.astype(np.int64) // bs)
    mb = max(1, int(blocks.max()), -(-cap // bs))
    nb = int(blocks.sum()) + spare
    ids = r.permutation(nb).astype(np.int32)
    table = r.choice(np.array([-1, 2 ** 31 - 1, -2 ** 31], np.int64), (B, mb)).astype(np.int32)
    table[np.arange(mb)[None] < blocks[:, None]] = ids[: blocks.sum()]
    kc, vc = (np.full((nb, bs, Hkv, D), np.nan, np.float32) for _ in range(2))
    for b in range(B):
        if lens[b]:
            x = r.standard_normal((2, blocks[b] * bs, Hkv, D)).astype(np.float32)
            x[:, lens[b]:] = np.nan
            kc[table[b, : blocks[b]]], vc[table[b, : blocks[b]]] = x.reshape(2, blocks[b], bs, Hkv, D)
    q = (r.standard_normal((B, Hq, D)) * size).astype(np.float32)
    if dtype == torch.bfloat16:
        q = U.bf16_round(q)
        for c in (kc, vc):
            ok = np.isfinite(c)
            c[ok] = U.bf16_round(c[ok])
    return dict(q=q, kc=kc, vc=vc, table=table, lens=lens, scale=D ** -0.5, dtype=dtype)


def on_device(h):
    B, Hq, D = h["q"].shape
    nb, bs, Hkv, _ = h["kc"].shape
    dt = h["dtype"]
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    n = tsv.decode_attn_workspace_size(B, Hq, Hkv, D, bs, h["table"].shape[1], tsv.TSV_BF16 if dt == torch.bfloat16 else tsv.TSV_F32)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None  # NaN wherever it is read unwritten
    return dict(q=cu(h["q"]).to(dt), k_cache=cu(h["kc"]).to(dt), v_cache=cu(h["vc"]).to(dt), block_table=cu(h["table"]),
                seq_lens=cu(h["lens"]), out=torch.full((B, Hq, D), 7.0, dtype=dt, device="cuda"), scale=h["scale"], workspace=ws,
                seq_err=torch.full((B,), -9, dtype=torch.int32, device="cuda"), lse=torch.full((B, Hq), 7.0, device="cuda"))


def check(h, d):
    torch.cuda.synchronize()
    out, lse, err, mass = S.decode_attn(h["q"], h["kc"], h["vc"], h["table"], h["lens"], h["scale"])
    got, got_lse = d["out"].float().cpu().numpy(), d["lse"].cpu().numpy()
    assert np.array_equal(d["seq_err"].cpu().numpy(), err)
    B, Hq, D = out.shape
    Hkv = h["kc"].shape[2]
    for b in range(B):
        if err[b]:
            assert np.isnan(got[b]).all() and np.isnan(got_lse[b]).all()
            continue
        L = int(h["lens"][b])
        if L == 0:
            assert (got[b] == 0).all() and (got_lse[b] == -np.inf).all()
            continue
        rows = h["kc"][h["table"][b, : -(-L // h["kc"].shape[1])]].reshape(-1, Hkv, D)[:L]
        big = np.array([h["scale"] * (np.abs(rows[:, i * Hkv // Hq]) @ np.abs(h["q"][b, i])).max() for i in range(Hq)])
        e = 2 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -20
        e = 2 * e + (L + 64) * 2.0 ** -24
        tol = mass[b] * (e[:, None] + (2.0 ** -7 if h["dtype"] == torch.bfloat16 else 0.0))
        assert (np.abs(got[b] - out[b]) <= tol).all(), (b, L, np.abs(got[b] - out[b]).max(), tol.min())
        assert (np.abs(got_lse[b] - lse[b]) <= e + 2.0 ** -22 * np.abs(lse[b])).all(), (b, L)


SHAPES = [  # lens, Hq, Hkv, D, bs
    ([1], 1, 1, 64, 8), ([0], 4, 2, 128, 16), ([0, 0, 5], 8, 2, 64, 16), ([7, 8, 9, 15, 16, 17], 6, 3, 128, 8),
    ([31, 32, 33, 63, 64, 65, 127], 8, 1, 128, 16), ([128, 129, 1, 0, 255, 256, 257], 16, 2, 64, 32), ([1000, 3, 0, 77], 32, 8, 128, 16),
    ([511, 513], 20, 4, 64, 64), ([300] * 3, 17, 1, 128, 16), ([205, 1, 400], 32, 1, 64, 16), ([260, 33], 40, 1, 128, 128),
    ([190], 64, 1, 128, 16), ([20011], 8, 2, 128, 16), ([9000, 1, 4500, 0, 12345], 14, 2, 64, 8), (list(range(90)), 4, 4, 64, 16),
    ([5] * 400, 8, 8, 64, 16), ([3, 0, 40] * 500, 2, 2, 64, 16), ([2049, 3000, 77, 640] * 9, 12, 4, 128, 32), ([4096] * 8, 32, 8, 128, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [0, 50000])  # a long table: lanes for more tiles than there are
@pytest.mark.parametrize("lens,Hq,Hkv,D,bs", SHAPES)
def test_decode(dtype, cap, lens, Hq, Hkv, D, bs):
    h = make(len(lens) + Hq + D, lens, Hq, Hkv, D, bs, dtype, cap=cap)
    d = on_device(h)
    tsv.decode_attn(**d)
    check(h, d)
    first, first_lse = d["out"].clone(), d["lse"].clone()
    if d["workspace"] is not None:
        d["workspace"].fill_(127)
    d["lse"] = None
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       d["out"].view(torch.int16 if dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_table_with_room_for_much_longer_sequences(dtype):
    h = make(5, [100, 2000, 1, 0], 8, 2, 128, 16, dtype, cap=100000)
    d = on_device(h)
    tsv.decode_attn(**d)
    check(h, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_scores(dtype):
    # one key of each row takes nearly all of the weight, and the running maximum moves often
    h = make(6, [700, 64, 65], 8, 2, 128, 16, dtype, size=12.0)
    d = on_device(h)
    tsv.decode_attn(**d)
    check(h, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [40, 5000])
@pytest.mark.parametrize("cap", [0, 50000])
def test_infinities(dtype, L, cap):
    h = make(7, [L, L], 2, 2, 64, 16, dtype, cap=cap)
    h["q"] = np.abs(h["q"])
    where = h["table"][0, (L // 2) // 16]
    h["kc"][where, (L // 2) % 16, 0] = -np.inf  # a key that no row attends to
    h["vc"][where, (L // 2) % 16, 0] = 3.0
    d = on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    h2 = dict(h, kc=np.where(np.isinf(h["kc"]), -3e38, h["kc"]).astype(np.float32))
    out, lse, err, _ = S.decode_attn(h2["q"].astype(np.float64), h2["kc"], h2["vc"], h2["table"], h2["lens"], h2["scale"])
    got = d["out"].float().cpu().numpy()
    assert np.isfinite(got).all() and np.abs(got - out).max() < 0.02
    # every key of one head at -infinity: 0 / 0; a NaN key or value: NaN in its own rows alone
    h["kc"][h["table"][1, : -(-L // 16)], :, 1] = -np.inf
    h["vc"][where, 3, 0, 5] = np.nan
    d = on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    got, got_lse = d["out"].float().cpu().numpy(), d["lse"].cpu().numpy()
    assert np.isnan(got[1, 1]).all() and got_lse[1, 1] == -np.inf
    assert np.isnan(got[0, 0, 5]) and np.isfinite(np.delete(got[0, 0], 5)).all() and np.isfinite(got[0, 1]).all()
    assert np.isfinite(got[1, 0]).all() and not d["seq_err"].any()
    h["kc"][h["table"][0, 0], 2, 0, 1] = np.nan
    d = on_device(h)
    tsv.decode_attn(**d)
    torch.cuda.synchronize()
    got = d["out"].float().cpu().numpy()
    assert np.isnan(got[0, 0]).all() and np.isnan(d["lse"].cpu().numpy()[0, 0]) and np.isfinite(got[0, 1]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [0, 70000])
def test_bad_lengths_and_blocks(dtype, cap):
    h = make(8, [100, 9000, 33, 700, 5000, 1], 8, 2, 64, 16, dtype, cap=cap)
    nb = h["kc"].shape[0]
    h["lens"][2] = -1
    h["lens"][3] = h["table"].shape[1] * 16 + 1
    h["table"][1, 300] = nb
    h["table"][4, 0] = -1
    h["table"][5, 0] = 2 ** 31 - 1
    d = on_device(h)
    tsv.decode_attn(**d)
    check(h, d)
    assert d["seq_err"].tolist() == [0, 2, 4, 4, 2, 2]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [-1, -2, -2 ** 31, None])
@pytest.mark.parametrize("cap", [0, 50000])
def test_every_bad_id_is_found(dtype, block, cap):
    h = make(40, [300, 17], 4, 2, 64, 16, dtype, cap=cap)
    h["table"][0, 9] = h["kc"].shape[0] if block is None else block
    d = on_device(h)
    tsv.decode_attn(**d)
    check(h, d)
    assert d["seq_err"].tolist() == [2, 0]


@pytest.mark.parametrize("cap", [3000, 40000])
def test_two_graphs_share_a_workspace(cap):
    a, b = (make(s, lens, 8, 2, 128, 16, torch.bfloat16, cap=cap) for s, lens in ((9, [3000, 10, 801]), (10, [1, 2500, 0])))
    da, db = on_device(a), on_device(b)
    db["workspace"] = da["workspace"]  # of the same size
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tsv.decode_attn(**da)
        tsv.decode_attn(**db)
    torch.cuda.synchronize()
    graphs = []
    for d in (da, db):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tsv.decode_attn(**d)
        graphs.append(g)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    check(a, da)
    check(b, db)
    # new lengths in the captured call
    da["seq_lens"].copy_(torch.tensor([1, 0, 800]))
    a["lens"][:] = [1, 0, 800]
    graphs[0].replay()
    check(a, da)


def test_two_streams_with_a_workspace_each():
    hs = [make(20 + i, [4000, 17, 2300], 16, 2, 128, 16, torch.bfloat16, cap=60000 * i) for i in range(2)]
    ds = [on_device(h) for h in hs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(ds, streams):
            tsv.decode_attn(**d, stream=s)
    for h, d in zip(hs, ds):
        check(h, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(dtype):
    # a cache of more than 2^31 elements; the sequence's blocks lie at its far end
    D, Hkv, bs = 128, 8, 16
    nb = 2 ** 31 // (bs * Hkv * D) + 64
    h = make(30, [500], 16, Hkv, D, bs, dtype)
    d = on_device(h)
    used = h["table"][0, : -(-500 // bs)].astype(np.int64)
    far = nb - 1 - np.arange(len(used))
    for n in ("k_cache", "v_cache"):
        big = torch.zeros(nb, bs, Hkv, D, dtype=dtype, device="cuda")
        big[torch.from_numpy(far).cuda()] = d[n][torch.from_numpy(used).cuda()]
        d[n] = big
    d["block_table"][0, : len(used)] = torch.from_numpy(far.astype(np.int32)).cuda()
    tsv.decode_attn(**d)
    check(h, d)


def test_workspace_of_another_size_is_refused():
    h = make(31, [4000], 8, 2, 128, 16, torch.bfloat16, cap=100000)
    d = on_device(h)
    d["workspace"] = d["workspace"][:-16]
    with pytest.raises(tsv.TsvError, match="workspace"):
        tsv.decode_attn(**d)
    with pytest.raises(ValueError, match="device"):
        tsv.decode_attn(**{**on_device(h), "lse": torch.zeros(1, 8)})


def test_host_threads_at_once():
    import threading
    hs = [make(50 + i, [700 * i + 5, 33], 8, 2, 128 if i % 2 else 64, 16, torch.bfloat16 if i < 3 else torch.float32) for i in range(4)]
    ds, failed = [on_device(h) for h in hs], []
    torch.cuda.synchronize()

    def work(d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    tsv.decode_attn(**d)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test below
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(d,)) for d in ds]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for h, d in zip(hs, ds):
        check(h, d)
