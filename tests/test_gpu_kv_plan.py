"""The slot plan on the device against its oracle: whole numbers, all equal."""
import numpy as np
import pytest
import torch

from oracle import serving as S
import serving_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


def device_plan(c, in_place=False, stream=None):
    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    d = {k: dev(c[k]) for k in ("seq_lens", "new_lens", "table", "held", "free_blocks")}
    d["count"] = torch.tensor([c["free_count"]], dtype=torch.int32, device="cuda")
    d["parent"] = None if c.get("parent") is None else dev(c["parent"])
    B, T = len(c["seq_lens"]), c["max_tokens"]
    i32 = dict(dtype=torch.int32, device="cuda")
    d["held_out"] = d["held"] if in_place else torch.full((B,), -9, **i32)
    d["count_out"] = d["count"] if in_place else torch.full((1,), -9, **i32)
    d["total"] = d["seq_lens"] if in_place else torch.full((B,), -9, **i32)
    d.update(offsets=torch.full((B + 1,), -9, **i32), slots=torch.full((T,), -9, dtype=torch.int64, device="cuda"),
             positions=torch.full((T,), -9, **i32), err=torch.full((B,), -9, **i32), bs=c["block_size"])
    return d


def call(d, stream=None):
    tsv.kv_plan_slots(d["seq_lens"], d["new_lens"], d["table"], d["held"], d["held_out"], d["free_blocks"], d["count"],
                      d["count_out"], d["total"], d["offsets"], d["slots"], d["positions"], d["bs"], d["err"],
                      parent=d["parent"], stream=stream)


def results(d):
    torch.cuda.synchronize()
    return dict(table=d["table"].cpu().numpy(), held=d["held_out"].cpu().numpy(), pool=d["free_blocks"].cpu().numpy(),
                count=int(d["count_out"]), total=d["total"].cpu().numpy(), offsets=d["offsets"].cpu().numpy(),
                slots=d["slots"].cpu().numpy(), positions=d["positions"].cpu().numpy(), err=d["err"].cpu().numpy())


def check(c, d):
    got, want = results(d), S.plan_slots(**c)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    return want


@pytest.mark.parametrize("B,bs,max_len,max_new,kw", [
    (1, 16, 0, 1, {}), (1, 8, 40, 3, {}), (2, 128, 300, 200, {}), (7, 16, 100, 1, dict(ended=0.3)),
    (64, 16, 2000, 0, dict(tree=64)), (33, 32, 500, 0, dict(tree=128)), (5, 8, 50, 0, dict(tree=1)),
    (257, 16, 700, 60, dict(ended=0.2, pad=37)), (1025, 64, 900, 20, dict(ended=0.1)), (8192, 8, 60, 9, dict(ended=0.1, pad=5)),
    (2330, 16, 300, 40, dict(ended=0.1, tree=7)), (64, 16, 200, 7, dict(pad=60)), (65, 16, 200, 3, {}), (300, 16, 100, 0, dict(tree=64)),
    (3000, 16, 90, 0, dict(tree=6, pad=900)), (700, 32, 300, 60, dict(pool="short", ended=0.1)),
    (3, 16, 20, 9000, {}), (40, 16, 300, 40, dict(pool="exact")), (40, 16, 300, 40, dict(pool="exact", ended=0.4)),
    (60, 16, 300, 80, dict(pool="short")), (60, 16, 300, 0, dict(pool="short", tree=33)), (12, 16, 90, 0, dict(spare=1.0))])
def test_plan(B, bs, max_len, max_new, kw):
    for seed in range(2):
        c = U.plan_case(np.random.default_rng(100 * B + seed), B, bs, max_len, max_new, **kw)
        d = device_plan(c)
        call(d)
        want = check(c, d)
        if kw.get("pool") != "short":
            assert not want["err"].any()
        call(d)  # separate outputs: the same call again gives the same
        check(c, d)
        d = device_plan(c, in_place=True)
        call(d)
        check(c, d)


def test_nothing_to_write():
    # requests end, no token is written; the map may be empty
    c = U.plan_case(np.random.default_rng(5), 9, 16, 100, 0, ended=1.0)
    assert c["max_tokens"] == 0
    d = device_plan(c)
    call(d)
    check(c, d)


def _broken(seed, **kw):
    return U.plan_case(np.random.default_rng(seed), 24, 16, 200, 20, ended=0.2, **kw)


@pytest.mark.parametrize("what", ["length", "new", "held", "held_low", "capacity", "tokens", "count", "count_low", "ids",
                                  "back_ids", "pool_ids", "pool_ids_taken", "pool_full", "huge"])
def test_bad_data_is_reported_and_the_others_served(what):
    c = _broken(7) if what != "pool_ids_taken" else U.plan_case(np.random.default_rng(7), 24, 16, 200, 20, spare=0.0)
    mb = c["table"].shape[1]
    r = np.random.default_rng(8)
    if what == "length":
        c["seq_lens"][3] = -1
    elif what == "new":
        c["new_lens"][[4, 9]] = [-5, -2147483648]
    elif what == "held":
        c["held"][5] = mb + 1
    elif what == "held_low":
        c["held"][5] = -1
    elif what == "capacity":
        c["new_lens"][6] = mb * 16 - c["seq_lens"][6] + 1
        c["max_tokens"] = int(c["new_lens"].sum())
    elif what == "tokens":
        c["max_tokens"] -= 25
    elif what == "count":
        c["free_count"] = len(c["free_blocks"]) + 1
    elif what == "count_low":
        c["free_count"] = -1
    elif what == "ids":
        c["table"][np.arange(24), np.maximum(c["held"] - 1, 0)] = r.choice([-1, len(c["free_blocks"]), 2 ** 31 - 1], 24)
    elif what == "back_ids":
        gone = np.flatnonzero((c["seq_lens"] == 0) & (c["held"] > 0))
        c["held"][gone] = mb
        c["table"][gone] = -5
    elif what.startswith("pool_ids"):
        c["free_blocks"][: c["free_count"]] = 2 ** 30
    elif what == "pool_full":
        c["held"][c["seq_lens"] == 0] = mb
        c["free_count"] = len(c["free_blocks"]) - 2
        c["free_blocks"][:] = 0
    elif what == "huge":
        c["seq_lens"][2] = c["new_lens"][2] = 2 ** 31 - 1
        c["new_lens"][11] = 2 ** 31 - 1
    d = device_plan(c)
    call(d)
    want = check_saturated(c, d) if what == "huge" else check(c, d)
    # (with "pool_ids" the returned blocks, which are popped first, are enough)
    assert want["err"].any() == (what != "pool_ids")


@pytest.mark.parametrize("what", ["length", "capacity", "tokens", "ids", "pool_ids", "pool_ids_taken", "trees"])
def test_bad_data_in_a_large_batch(what):
    # the slot map is filled by a second kernel
    r = np.random.default_rng(12)
    c = U.plan_case(r, 900, 16, 300, 40, ended=0.0 if what == "pool_ids_taken" else 0.1, tree=33 if what == "trees" else None,
                    spare=0.1, pad=50)
    some = r.permutation(900)[:40]
    if what == "length":
        c["seq_lens"][some] = -3
    elif what == "capacity":
        c["held"][some] = c["table"].shape[1] + 7
    elif what == "tokens":
        c["max_tokens"] = c["max_tokens"] * 2 // 3
    elif what == "ids":
        c["table"][some, np.maximum(c["held"][some] - 1, 0)] = -1
    elif what.startswith("pool_ids"):
        c["free_blocks"][r.integers(0, c["free_count"], 40)] = 2 ** 30
    else:
        c["parent"][some, r.integers(1, 33, 40)] = 99
        c["new_lens"][some[:5]] = 40
    d = device_plan(c)
    call(d)
    # (with "pool_ids" the returned blocks, which are popped first, are enough)
    assert check(c, d)["err"].any() == (what != "pool_ids")


def check_saturated(c, d):
    # running sums past 2^31 are reported as 2^31 - 1
    got, want = results(d), S.plan_slots(**{**c, "new_lens": np.minimum(c["new_lens"], 10 ** 6)})
    ends = np.concatenate([[0], np.cumsum(c["new_lens"].astype(np.int64))])
    want["offsets"] = np.minimum(ends, 2 ** 31 - 1).astype(np.int32)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    return want


@pytest.mark.parametrize("fault", ["root", "self", "later", "below"])
def test_rows_that_are_no_trees(fault):
    c = U.plan_case(np.random.default_rng(3), 10, 16, 100, 0, tree=20)
    row = c["parent"][4]
    if fault == "root":
        row[0] = 0
    elif fault == "self":
        row[7] = 7
    elif fault == "later":
        row[5] = 11
    else:
        row[9] = -3
    d = device_plan(c)
    call(d)
    want = check(c, d)
    assert want["err"][4] == tsv.TSV_DERR_PARENT and not np.delete(want["err"], 4).any()


def test_more_tokens_than_nodes():
    c = U.plan_case(np.random.default_rng(3), 6, 16, 100, 0, tree=8)
    c["new_lens"][2] = 9
    c["max_tokens"] += 1
    d = device_plan(c)
    call(d)
    assert check(c, d)["err"].tolist() == [0, 0, tsv.TSV_DERR_PARENT, 0, 0, 0]


def test_captured_and_replayed_on_another_stream():
    cases = [U.plan_case(np.random.default_rng(s), 20, 16, 120, 9, ended=0.2, pad=180) for s in (1, 2)]
    T = max(c["max_tokens"] for c in cases)
    nb, mb = (max(x) for x in zip(*[(len(c["free_blocks"]), c["table"].shape[1]) for c in cases]))
    for c in cases:
        c["max_tokens"] = T
        c["free_blocks"] = np.resize(c["free_blocks"], nb)
        assert c["table"].shape[1] == mb
    d = device_plan(cases[0], in_place=True)
    start = {k: d[k].clone() for k in ("seq_lens", "new_lens", "table", "held", "free_blocks", "count")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d)
    for c in cases:
        e = device_plan(c)
        for k in start:
            d[k].copy_(e[k])
        g.replay()
        check(c, d)
    # a second replay continues from the state the first one left: all tokens cached now
    again = {**cases[1], **{k: results(d)[k2] for k, k2 in (("seq_lens", "total"), ("held", "held"), ("table", "table"),
                                                            ("free_blocks", "pool"), ("free_count", "count"))}}
    again = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in again.items()}
    g.replay()
    check(again, d)
