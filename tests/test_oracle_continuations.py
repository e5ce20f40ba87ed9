"""Pins of the oracle of the operators for several continuations (CPU): invariants and independent routes."""
import numpy as np
import pytest
import torch

from oracle import continuations as C
from oracle import serving as S
import continuation_util as U


def owned(o, nb):
    return U.refs(o["table"], o["held"], nb)


@pytest.mark.parametrize("seed", range(6))
def test_every_reference_is_counted(seed):
    r = np.random.default_rng(seed)
    s = U.pages_state(r, 23, 8, 90)
    nb = len(s["shares"])
    src, dst = U.fork_list(r, s)
    f = C.fork(src, dst, block_size=8, **s)
    n = owned(f, nb)
    assert not f["err"].any() and np.array_equal(np.maximum(n - 1, 0), f["shares"])
    free = set(s["free_blocks"][:f["count"]])
    assert not free & set(np.flatnonzero(n)) and len(free) == f["count"]
    # then some end, some are cut back to a full block
    keep = np.where(r.random(23) < 0.5, 0, f["seq_lens"])
    g = C.release(keep, f["table"], f["held"], f["shares"], s["free_blocks"], f["count"], 8)
    n = U.refs(f["table"], g["held"], nb)
    assert not g["err"].any() and np.array_equal(np.maximum(n - 1, 0), g["shares"])
    pool = g["pool"][:g["count"]]
    assert len(set(pool)) == len(pool) and not set(pool) & set(np.flatnonzero(n))
    # nothing is lost: every block that was in use or free still is
    before = set(np.flatnonzero(U.refs(s["table"], s["held"], nb))) | set(s["free_blocks"][:s["free_count"]])
    assert set(pool) | set(np.flatnonzero(n)) == before


def test_fork_by_hand():
    table = np.array([[4, 2, 9, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]], np.int32)
    o = C.fork(np.array([0, -1, 0]), np.array([2, 5, 1]), np.array([19, 0, 0]), table, np.array([3, 0, 0]), np.zeros(10, np.int32),
               np.array([6, 7, 8] + [0] * 7), 3, 8)
    assert o["table"].tolist() == [[4, 2, 9, -1], [4, 2, 7, -1], [4, 2, 8, -1]] and o["count"] == 1
    assert o["shares"].tolist() == [0, 0, 2, 0, 2, 0, 0, 0, 0, 0] and o["seq_lens"].tolist() == [19] * 3
    assert (o["copy_src"].tolist(), o["copy_dst"].tolist(), o["copy_rows"].tolist()) == ([9, -1, 9], [8, -1, 7], [3, 0, 3])


def test_release_by_hand():
    table = np.array([[1, 5, 3], [1, 5, 0], [1, 2, -1]], np.int32)
    o = C.release(np.array([0, 17, 0]), table, np.array([3, 3, 2]), np.array([0, 2, 0, 0, 0, 1]), np.array([4, -1, -1, -1, -1, -1]), 1, 8)
    assert o["held"].tolist() == [0, 3, 0] and o["shares"].tolist() == [0] * 6
    assert o["pool"].tolist() == [4, 2, 3, -1, -1, -1] and o["count"] == 3


@pytest.mark.parametrize("seed", range(5))
def test_compaction_keeps_every_sequences_rows(seed):
    r = np.random.default_rng(seed)
    s = U.pages_state(r, 15, 16, 200, free=30, extra=9)
    nb = len(s["shares"])
    cache = r.standard_normal((nb, 16, 2))
    o = C.compact(s["table"], s["held"], s["shares"], s["free_blocks"])
    after, err = C.copy_blocks(cache, o["copy_src"], o["copy_dst"], count=o["copy_count"])
    assert not err.any() and not o["err"].any()
    for b in range(15):
        h = s["held"][b]
        assert np.array_equal(cache[s["table"][b, :h]], after[o["table"][b, :h]])
    n = U.refs(o["table"], s["held"], nb)
    assert (n[: nb - o["count"]] > 0).all() and not n[nb - o["count"]:].any()
    assert np.array_equal(np.maximum(n - 1, 0), o["shares"])
    assert sorted(o["pool"][: o["count"]]) == list(range(nb - o["count"], nb))


def test_prefix_attention_is_single_token_attention_over_joined_tables():
    r = np.random.default_rng(3)
    c = U.prefix_case(r, [3, 1, 2], [37, 0, 16], [1, 9, 30, 5, 2, 1], 4, 2, 64, 8)
    out, lse, err = C.prefix_attn(**c)
    assert not err.any()
    off, bs = c["group_offsets"], 8
    for g in range(3):
        for b in range(off[g], off[g + 1]):
            t = np.arange(c["seq_lens"][b])
            ids = c["table"][np.where(t < c["prefix_lens"][g], off[g], b), t // bs]
            k, v = (torch.from_numpy(c[n][ids, t % bs]).double().transpose(0, 1).repeat_interleave(2, 0) for n in ("k_cache", "v_cache"))
            q = torch.from_numpy(c["q"][b]).double()[:, None]
            want = torch.nn.functional.scaled_dot_product_attention(q, k, v)
            assert torch.allclose(torch.from_numpy(out[b]), want[:, 0], atol=1e-12)
    assert S.__doc__


def test_logprobs_against_torch():
    r = np.random.default_rng(4)
    x = r.standard_normal((6, 50)).astype(np.float32) * 3
    x[2, ::3] = -np.inf
    tok = np.array([0, 49, 1, -1, 50, 7], np.int32)
    o = C.logprobs(x, tok, 0.5, 5)
    want = torch.log_softmax(torch.from_numpy(x).double() / 0.5, -1).numpy()
    for t in (0, 1, 2, 5):
        assert abs(o["logprobs"][t] - want[t, tok[t]]) < 1e-12
        p = np.exp(want[t])
        assert abs(o["entropy"][t] + np.sum(p[p > 0] * want[t][p > 0])) < 1e-12
        assert np.allclose(o["top_logprobs"][t], np.sort(want[t])[::-1][:5])
    assert o["err"].tolist() == [0, 0, 0, 0, 8, 0] and o["logprobs"][3] == 0 and np.isnan(o["logprobs"][4])
    flat = C.logprobs(np.array([[0.0, -0.0, 1.0, 0.0]]), np.array([1]), 1.0, 4)
    assert flat["top_ids"].tolist() == [[2, 0, 1, 3]]
