"""Forks, releases, compaction and block copies against the oracle, exactly."""
import numpy as np
import pytest
import torch

from oracle import continuations as C
import continuation_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def out(n, in_place, t):
    return t if in_place else torch.full((n,) if isinstance(n, int) else n, -9, dtype=torch.int32, device="cuda")


def run_fork(s, src, dst, bs, in_place=False, again=False):
    B, mb, nb, F = *s["table"].shape, len(s["shares"]), len(src)
    lens, table, held, shares, pool, count = (dev(s[n]) for n in ("seq_lens", "table", "held", "shares", "free_blocks", "free_count"))
    count = count.reshape(1)
    lo, ho, so, co = (out(n, in_place, t) for n, t in ((B, lens), (B, held), (nb, shares), (1, count)))
    cs, cd, cr, err = (out(F, False, None) for _ in range(4))
    for _ in range(2 if again else 1):
        tsv.kv_fork_seqs(dev(src), dev(dst), lens, lo, table, held, ho, shares, so, pool, count, co, cs, cd, cr, bs, err)
    got = dict(table=table, seq_lens=lo, held=ho, shares=so, count=co, copy_src=cs, copy_dst=cd, copy_rows=cr, err=err)
    got = {k: v.cpu().numpy() for k, v in got.items()}
    assert np.array_equal(pool.cpu().numpy(), s["free_blocks"])
    return got


def run_release(s, keep, bs, in_place=False, again=False):
    B, nb = len(keep), len(s["shares"])
    table, held, shares, pool, count = (dev(s[n]) for n in ("table", "held", "shares", "free_blocks", "free_count"))
    count = count.reshape(1)
    ho, so, co = (out(n, in_place, t) for n, t in ((B, held), (nb, shares), (1, count)))
    err = out(B, False, None)
    for _ in range(2 if again else 1):
        tsv.kv_release_seqs(dev(keep), table, held, ho, shares, so, pool, count, co, bs, err)
    assert np.array_equal(table.cpu().numpy(), s["table"])
    return {k: v.cpu().numpy() for k, v in dict(held=ho, shares=so, pool=pool, count=co, err=err).items()}


def run_compact(s, in_place=False, again=False):
    (B, mb), nb = s["table"].shape, len(s["shares"])
    table, held, shares, pool = (dev(s[n]) for n in ("table", "held", "shares", "free_blocks"))
    to, so = out((B, mb), in_place, table), out(nb, in_place, shares)
    co, cc, cs, cd, err = (out(n, False, None) for n in (1, 1, nb // 2, nb // 2, B))
    ws = torch.full((tsv.kv_compact_workspace_size(nb),), 0xab, dtype=torch.uint8, device="cuda")
    for _ in range(2 if again else 1):
        tsv.kv_compact_blocks(table, to, held, shares, so, pool, co, cs, cd, cc, err, ws)
    return {k: v.cpu().numpy() for k, v in dict(table=to, shares=so, pool=pool, count=co, copy_src=cs, copy_dst=cd, copy_count=cc,
                                                err=err).items()}


def same(got, want):
    for k in want:
        assert np.array_equal(got[k].reshape(-1), np.asarray(want[k]).reshape(-1)), (k, got[k], want[k])


def args(s):
    return {k: s[k] for k in ("seq_lens", "table", "held", "shares", "free_blocks", "free_count")}


SIZES = [(1, 8, 1, {}), (3, 16, 40, {}), (40, 16, 300, {}), (40, 128, 300, dict(empty=0.8)), (300, 8, 700, {}), (1500, 16, 90, dict(empty=0.5, free=900)),
         (2, 8, 30000, dict(empty=0.5)), (8, 8, 20000, dict(max_blocks=9001)), (8192, 8, 9, dict(empty=0.7, free=8000)),
         (600, 8, 300, dict(max_blocks=200, free=400)), (90, 16, 3000, dict(extra=17000))]


@pytest.mark.parametrize("B,bs,max_len,kw", SIZES)
def test_fork(B, bs, max_len, kw):
    r = np.random.default_rng(B)
    s = U.pages_state(r, B, bs, max_len, **kw)
    src, dst = U.fork_list(r, s)
    src, dst = src[:8192], dst[:8192]
    want = C.fork(src, dst, block_size=bs, **args(s))
    for in_place in (False, True):
        same(run_fork(s, src, dst, bs, in_place), want)
    same(run_fork(s, src, dst, bs, again=True), want)  # a repeated call


@pytest.mark.parametrize("free", [0, 1, 7])
def test_fork_with_a_pool_that_runs_dry(free):
    r = np.random.default_rng(free)
    s = U.pages_state(r, 60, 8, 90, free=free)
    src, dst = U.fork_list(r, s)
    want = C.fork(src, dst, block_size=8, **args(s))
    assert (want["err"] == C.DERR_POOL).any()
    same(run_fork(s, src, dst, 8), want)


def test_fork_errors():
    r = np.random.default_rng(5)
    s = U.pages_state(r, 12, 8, 60, empty=0.0, shared=0.0)
    for b in (6, 7, 8, 9, 10, 11):
        s["held"][b] = 0
    s["seq_lens"][:6] = [17, -1, 500, 12, 16, 9]
    s["held"][3] = s["table"].shape[1] + 1
    s["table"][5, 0], s["table"][4, 1] = -4, len(s["shares"])
    s["table"][0, :3] = [1, 2, 3]
    s["held"][0] = 3
    #      out of the batch, twice, not empty, bad lengths, bad blocks, itself, padding
    src = np.array([12, 0, 0, 0, 0, 0, 1, 2, 3, 4, 5, 0, -1, 99], np.int32)
    dst = np.array([6, 12, -1, 7, 7, 1, 8, 8, 8, 9, 10, 0, 11, 11], np.int32)
    want = C.fork(src, dst, block_size=8, **args(s))
    assert set(want["err"]) == {0, C.DERR_SEQ, C.DERR_BLOCK}
    same(run_fork(s, src, dst, 8), want)
    dst[7], dst[8] = 11, 6
    src[0], dst[12], dst[13] = -1, -1, -1
    want = C.fork(src, dst, block_size=8, **args(s))
    assert C.DERR_CAPACITY in want["err"]
    same(run_fork(s, src, dst, 8), want)
    for count in (-1, len(s["shares"]) + 1):
        s["free_count"] = count
        want = C.fork(src, dst, block_size=8, **args(s))
        assert C.DERR_POOL in want["err"]
        for in_place in (False, True):
            same(run_fork(s, src, dst, 8, in_place), want)


def test_fork_of_nothing():
    s = U.pages_state(np.random.default_rng(0), 4, 8, 30)
    none = np.zeros(0, np.int32)
    same(run_fork(s, none, none, 8), C.fork(none, none, block_size=8, **args(s)))


def releases(r, s, bs, ended=0.5):
    B = len(s["held"])
    keep = np.where(r.random(B) < ended, 0, s["seq_lens"])
    cut = r.random(B) < 0.2
    return np.where(cut, keep // 2, keep).astype(np.int32)


@pytest.mark.parametrize("B,bs,max_len,kw", SIZES + [(30, 8, 90, dict(extra=9000)), (30, 8, 90, dict(extra=40000))])
def test_release(B, bs, max_len, kw):
    r = np.random.default_rng(B)
    s = U.pages_state(r, B, bs, max_len, **kw)
    keep = releases(r, s, bs)
    a = args(s)
    del a["seq_lens"]
    want = C.release(keep, block_size=bs, **a)
    assert not want["err"].any()
    for in_place in (False, True):
        same(run_release(s, keep, bs, in_place), want)
    same(run_release(s, keep, bs, again=True), want)


@pytest.mark.parametrize("extra", [3, 20000])
def test_release_errors(extra):
    r = np.random.default_rng(6)
    s = U.pages_state(r, 12, 8, 60, empty=0.0, shared=0.0, extra=extra)
    keep = np.zeros(12, np.int32)
    keep[1], keep[7] = -1, 2 ** 31 - 1
    s["held"][2], s["held"][3] = -1, s["table"].shape[1] + 1
    s["table"][4, 0], s["table"][5, 0] = -2, len(s["shares"])
    s["held"][4:6] = np.maximum(s["held"][4:6], 1)
    a = args(s)
    del a["seq_lens"]
    want = C.release(keep, block_size=8, **a)
    assert {C.DERR_CAPACITY, C.DERR_BLOCK} < set(want["err"])
    for in_place in (False, True):
        same(run_release(s, keep, 8, in_place), want)
    # a block that two sequences hold and only one reference is counted for
    s["table"][8, 0] = s["table"][9, 0]
    s["held"][8:10] = np.maximum(s["held"][8:10], 1)
    a = args(s)
    del a["seq_lens"]
    want = C.release(keep, block_size=8, **a)
    assert want["err"][8] == want["err"][9] == C.DERR_POOL and want["err"][10] == 0
    same(run_release(s, keep, 8), want)
    # a pool without places, and counts that cannot be
    for count in (len(s["shares"]), len(s["shares"]) - 2, -1, len(s["shares"]) + 1):
        s["free_count"] = a["free_count"] = count
        want = C.release(keep, block_size=8, **a)
        assert C.DERR_POOL in want["err"]
        for in_place in (False, True):
            same(run_release(s, keep, 8, in_place), want)


@pytest.mark.parametrize("B,bs,max_len,kw", SIZES + [(30, 8, 90, dict(extra=9000)), (30, 8, 900, dict(extra=40000)), (3, 8, 90, dict(free=0, extra=0)),
                                             (40, 8, 300, dict(max_blocks=2000, extra=9000)), (40, 8, 300, dict(max_blocks=2000, extra=70000)),
                                             (3, 8, 90, dict(extra=70000)), (40, 8, 900, dict(extra=12000)), (5, 16, 90, dict(extra=1, free=31))])
def test_compact(B, bs, max_len, kw):
    r = np.random.default_rng(B)
    s = U.pages_state(r, B, bs, max_len, **kw)
    want = C.compact(s["table"], s["held"], s["shares"], s["free_blocks"])
    for in_place in (False, True):
        same(run_compact(s, in_place), want)
    same(run_compact(s, again=True), want)
    # once more on the result: nothing moves
    s.update(table=want["table"], shares=want["shares"])
    got = run_compact(s)
    assert got["copy_count"][0] == 0 and np.array_equal(got["table"], want["table"])


def test_compact_errors():
    r = np.random.default_rng(8)
    s = U.pages_state(r, 12, 8, 60, empty=0.0)
    s["held"][2], s["held"][3] = -1, s["table"].shape[1] + 1
    s["table"][4, 0], s["table"][5, 0] = -2, len(s["shares"])
    s["held"][4:6] = np.maximum(s["held"][4:6], 1)
    want = C.compact(s["table"], s["held"], s["shares"], s["free_blocks"])
    assert {C.DERR_CAPACITY, C.DERR_BLOCK} < set(want["err"])
    for in_place in (False, True):
        same(run_compact(s, in_place), want)


@pytest.mark.parametrize("nb", [1, 2, 3, 31, 32, 33])
@pytest.mark.parametrize("held", [0, 1])
def test_caches_of_few_blocks(nb, held):
    """One sequence on the last block, or none: it moves to block 0, and everything else is free."""
    s = dict(seq_lens=np.array([5 * held], np.int32), table=np.array([[nb - 1, 99]], np.int32), held=np.array([held], np.int32),
             shares=np.zeros(nb, np.int32), free_blocks=np.arange(nb, dtype=np.int32), free_count=nb - held)
    want = C.compact(s["table"], s["held"], s["shares"], s["free_blocks"])
    assert want["copy_count"] == (held if nb > 1 else 0)
    for in_place in (False, True):
        same(run_compact(s, in_place), want)
    keep = np.zeros(1, np.int32)
    a = args(s)
    del a["seq_lens"]
    same(run_release(s, keep, 8), C.release(keep, block_size=8, **a))


def test_empty_batches():
    s = U.pages_state(np.random.default_rng(0), 4, 8, 30)
    s.update(table=np.zeros((0, 3), np.int32), held=np.zeros(0, np.int32), seq_lens=np.zeros(0, np.int32), shares=0 * s["shares"])
    a = args(s)
    del a["seq_lens"]
    same(run_release(s, np.zeros(0, np.int32), 8), C.release(np.zeros(0, np.int32), block_size=8, **a))
    same(run_compact(s), C.compact(s["table"], s["held"], s["shares"], s["free_blocks"]))
    pad = np.array([-1, 0], np.int32)
    same(run_fork(s, pad, pad, 8), C.fork(pad, pad, block_size=8, **args(s)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,D,bs,nb,n", [(1, 64, 8, 5, 2), (8, 128, 16, 40, 20), (3, 64, 128, 20, 9), (5, 128, 32, 900, 440), (40, 128, 64, 7, 3)])
def test_copy(dtype, Hkv, D, bs, nb, n):
    r = np.random.default_rng(n)
    cache = r.standard_normal((2, nb, bs, Hkv, D)).astype(np.float32)
    cache = torch.from_numpy(cache).to(dtype)
    ids = r.permutation(nb)
    src, dst = ids[:n].copy(), ids[n: 2 * n].copy()
    src[0] = src[-1]  # a source twice
    src[n // 2] = -1
    rows = r.integers(-3, bs + 4, n)
    for use_rows in (False, True):
        for count in (None, -1, 0, n - 1, n + 5):
            k, v = cache[0].clone().cuda(), cache[1].clone().cuda()
            err = torch.full((n,), -9, dtype=torch.int32, device="cuda")
            tsv.kv_copy_blocks(k, v, dev(src), dev(dst), err, copy_rows=dev(rows) if use_rows else None,
                               copy_count=None if count is None else dev([count]))
            for got, was in ((k, cache[0]), (v, cache[1])):
                want, e = C.copy_blocks(was.float().numpy(), src, dst, rows if use_rows else None, count)
                assert torch.equal(got.float().cpu(), torch.from_numpy(want)) and np.array_equal(err.cpu().numpy(), e)


def test_copy_errors_and_blocks_onto_themselves():
    cache = torch.randn(2, 6, 8, 1, 64)
    src, dst = np.array([6, 0, 1, 2, 3], np.int32), np.array([4, -1, 6, 2, 5], np.int32)
    k, v = cache[0].cuda(), cache[1].cuda()
    err = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    tsv.kv_copy_blocks(k, v, dev(src), dev(dst), err)
    want, e = C.copy_blocks(cache[0].numpy(), src, dst)
    assert e.tolist() == [2, 2, 2, 0, 0] == err.tolist() and np.array_equal(k.cpu().numpy(), want)


def test_captured_and_replayed_on_a_stream_of_its_own():
    r = np.random.default_rng(9)
    s = U.pages_state(r, 40, 16, 300)
    src, dst = U.fork_list(r, s)
    want = C.fork(src, dst, block_size=16, **args(s))
    nb, B, F = len(s["shares"]), 40, len(src)
    lens, table, held, shares, pool, count = (dev(s[n]) for n in ("seq_lens", "table", "held", "shares", "free_blocks", "free_count"))
    count = count.reshape(1)
    lo, ho, so, co, cs, cd, cr, err = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (B, B, nb, 1, F, F, F, F))
    k, v = torch.randn(2, nb, 16, 2, 64, device="cuda").unbind(0)
    k0, v0 = k.clone(), v.clone()
    cerr, ds, dd = torch.empty_like(err), dev(src), dev(dst)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        tsv.kv_fork_seqs(ds, dd, lens, lo, table, held, ho, shares, so, pool, count, co, cs, cd, cr, 16, err)
        tsv.kv_copy_blocks(k, v, cs, cd, cerr, copy_rows=cr)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same({n: t.cpu().numpy() for n, t in dict(table=table, seq_lens=lo, held=ho, shares=so, count=co, copy_src=cs, copy_dst=cd, copy_rows=cr,
                                              err=err).items()}, want)
    for got, was in ((k, k0), (v, v0)):
        assert np.array_equal(got.cpu().numpy(), C.copy_blocks(was.cpu().numpy(), want["copy_src"], want["copy_dst"], want["copy_rows"])[0])
