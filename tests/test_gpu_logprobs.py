"""Token log probabilities, entropy and alternatives against the fp64 oracle.

Bounds: the sums are fp32, at most V / 1000 + 64 additions and roundings deep (a thread of 512 adds every
512th entry in two chains; then trees), each off by 2^-24 of the sum; a log probability adds three
roundings of its own size, and the entropy is the difference of ln s and a mean of at most itself."""
import numpy as np
import pytest
import torch

from oracle import continuations as C
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def run(x, tok, temperature=1.0, top=0, entropy=True, **kw):
    """x: a torch tensor [T, V] on the device (rows may be strided)."""
    T = x.shape[0]
    lp, ent, err = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda"), torch.full((T,), -9, dtype=torch.int32, device="cuda")
    ids = torch.full((T, top), -9, dtype=torch.int32, device="cuda") if top else None
    tops = torch.full((T, top), 7.0, device="cuda") if top else None
    tsv.token_logprobs(x, torch.from_numpy(np.asarray(tok, np.int32)).cuda(), lp, err, temperature=temperature, entropy=ent if entropy else None,
                       top_ids=ids, top_logprobs=tops, **kw)
    got = dict(logprobs=lp, err=err)
    if entropy:
        got["entropy"] = ent
    if top:
        got.update(top_ids=ids, top_logprobs=tops)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check(x, tok, got, temperature=1.0, top=0):
    V = x.shape[1]
    o = C.logprobs(x.float().cpu().numpy(), tok, temperature, top)
    assert np.array_equal(got["err"], o["err"])
    step = 2.0 ** -24
    sums = (V / 1000 + 64) * step

    def near(a, b, tol):
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        fine = np.isfinite(b)
        assert (np.abs(a - b)[fine] <= tol[fine]).all(), (np.abs(a - b)[fine] / tol[fine]).max()

    with np.errstate(invalid="ignore"):
        near(got["logprobs"], o["logprobs"], 4 * step * np.abs(o["logprobs"]) + sums)
        if "entropy" in got:
            near(got["entropy"], o["entropy"], sums * (2 + 2 * np.abs(o["entropy"])))
        if top:
            assert np.array_equal(got["top_ids"], o["top_ids"])
            near(got["top_logprobs"], o["top_logprobs"], 4 * step * np.abs(o["top_logprobs"]) + sums)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,top,temp,extra", [
    (1, 1, 1, 1.0, 0), (1, 2, 2, 0.5, 1), (3, 7, 5, 1.0, 0), (2, 31, 31, 1.0, 2), (5, 1000, 0, 1.0, 0), (1, 1000, 20, 0.75, 0), (7, 4097, 32, 1.0, 3),
    (1, 32000, 5, 1.0, 0), (2, 128256, 20, 1.0, 0), (9, 128256, 1, 1.3, 8), (40, 32001, 16, 0.75, 5), (700, 1003, 3, 1.0, 1), (330, 50001, 32, 1.0, 0)])
def test_against_the_oracle(dtype, T, V, top, temp, extra):
    r = np.random.default_rng(V)
    x = torch.from_numpy((3 * r.standard_normal((T, V + extra))).astype(np.float32)).to(dtype).cuda()[:, :V]
    tok = r.integers(0, V, T)
    tok[T // 2] = -1 if T > 2 else tok[T // 2]
    for entropy in (True, False):
        check(x, tok, run(x, tok, temp, top, entropy), temp, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_every_alignment(dtype):
    r = np.random.default_rng(1)
    flat = torch.from_numpy(r.standard_normal(60000).astype(np.float32)).to(dtype).cuda()
    for first in range(9):
        for V in (5, 8, 3001):
            x = flat[first: first + 3 * (V + 1)].view(3, V + 1)[:, :V]
            check(x, [0, V - 1, V // 2], run(x, [0, V - 1, V // 2], 1.0, 4), 1.0, 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 40000), (400, 6000)])
def test_values_in_every_order(dtype, T, V):
    """Rising, falling, equal, few distinct, masked, one finite entry, large and small: the alternatives are found
    wherever they lie, ties by the lower index."""
    r = np.random.default_rng(2)
    rows = [np.linspace(-30, 30, V), np.linspace(30, -30, V), np.zeros(V), r.integers(0, 3, V), np.where(r.random(V) < 0.999, -np.inf, 1.0),
            np.where(np.arange(V) == V - 3, 5.0, -np.inf), 1e30 * r.standard_normal(V), np.where(r.random(V) < 0.5, 0.0, -0.0), np.full(V, -1e38),
            np.repeat(r.standard_normal(V // 50 + 1), 50)[:V], 1e-40 * r.standard_normal(V)]
    for row in rows:
        x = torch.from_numpy(np.tile(row.astype(np.float32), (T, 1))).to(dtype).cuda()
        for top in (1, 20, 32):
            got = run(x[:2], [V - 3, 0][:T], 1.0, top)
            check(x[:2], [V - 3, 0][:T], got, 1.0, top)
        many = run(x, [V - 3] * T, 1.0, 20)
        one = run(x[:1], [V - 3], 1.0, 20)
        assert (many["top_ids"] == many["top_ids"][0]).all() and np.array_equal(many["top_ids"][0], one["top_ids"][0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [9, 5000, 128256])
def test_rows_without_a_distribution(dtype, V):
    r = np.random.default_rng(3)
    x = r.standard_normal((7, V)).astype(np.float32)
    x[0, V // 2], x[1, V - 1], x[2] = np.nan, np.inf, -np.inf
    x[3, 0], x[5, V // 3] = -np.nan, -np.inf
    tok = [0, 1, 2, 3, V, V // 3, -5]
    xs = torch.from_numpy(x).to(dtype).cuda()
    got = run(xs, tok, 1.0, 5)
    check(xs, tok, got, 1.0, 5)
    assert got["err"].tolist() == [16, 16, 16, 16, 8, 0, 0] and got["logprobs"][5] == -np.inf and got["logprobs"][6] == 0
    assert (got["top_ids"][[0, 1, 2, 3, 4, 6]] == -1).all()


def test_a_token_far_below_the_rest():
    x = torch.zeros(1, 50, device="cuda")
    x[0, 7] = -3.0e38
    got = run(x, [7], 1.0, 3)
    assert abs(got["logprobs"][0] / -3.0e38 - 1) < 1e-6 and abs(got["entropy"][0] - np.log(49)) < 1e-5


def test_no_rows_and_repeats():
    assert run(torch.zeros(0, 9, device="cuda"), [], 1.0, 3)["logprobs"].shape == (0,)
    x = torch.randn(20, 40000, device="cuda")
    a, b = run(x, np.arange(20), 1.0, 20), run(x, np.arange(20), 1.0, 20)
    assert all(np.array_equal(a[k], b[k]) for k in a)


def test_captured_on_a_stream_of_its_own():
    x, tok = torch.randn(33, 32000, device="cuda"), torch.arange(33, dtype=torch.int32, device="cuda")
    lp, err = torch.empty(33, device="cuda"), torch.empty(33, dtype=torch.int32, device="cuda")
    ids, tops = torch.empty(33, 8, dtype=torch.int32, device="cuda"), torch.empty(33, 8, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        tsv.token_logprobs(x, tok, lp, err, top_ids=ids, top_logprobs=tops)
    for seed in range(3):
        x.copy_(torch.randn(33, 32000, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        check(x, np.arange(33), dict(logprobs=lp.cpu().numpy(), err=err.cpu().numpy(), top_ids=ids.cpu().numpy(),
                                     top_logprobs=tops.cpu().numpy()), 1.0, 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [33, 64, 65, 200, 256, 257, 400, 1024, 1025, 1500, 2999, 5000])
def test_rows_of_few_entries(dtype, V):
    """Rows that a warp holds, and rows with fewer slices than there are groups: random, rising, equal, few distinct,
    masked, without a distribution, padding and wrong tokens among them."""
    r = np.random.default_rng(V)
    rows = [r.standard_normal(V), 9 * r.standard_normal(V), np.linspace(-30, 30, V), np.linspace(30, -30, V), np.zeros(V), r.integers(0, 3, V),
            np.where(r.random(V) < 0.97, -np.inf, r.standard_normal(V)), np.where(np.arange(V) == V - 3, 5.0, -np.inf), np.full(V, -np.inf),
            np.where(np.arange(V) == V - 1, np.nan, 0.0), np.where(np.arange(V) == 1, np.inf, 0.0), np.repeat(r.standard_normal(V), 7)[:V],
            np.full(V, -1e38), 1e30 * r.standard_normal(V), np.where(r.random(V) < 0.5, 0.0, -0.0), r.standard_normal(V), r.standard_normal(V),
            r.standard_normal(V)]
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dtype).cuda()
    tok = [V - 3] * 15 + [-1, V, 0]
    for top, temp, entropy in ((0, 1.0, True), (1, 0.75, True), (5, 1.0, False), (20, 1.5, True), (32, 1.0, True)):
        check(x, tok, run(x, tok, temp, top, entropy), temp, top)
        check(x[2:3], tok[2:3], run(x[2:3], tok[2:3], temp, top, entropy), temp, top)
