"""Pins of the serving operators' oracle (CPU): invariants and independent routes."""
import numpy as np
import pytest
import torch

from oracle import serving as S
import serving_util as U


@pytest.mark.parametrize("seed", range(6))
def test_plan_keeps_every_block_owned_once(seed):
    c = U.plan_case(np.random.default_rng(seed), B=17, bs=8, max_len=90, max_new=30, ended=0.2)
    o = S.plan_slots(**c)
    assert not o["err"].any()
    owned = [x for b in range(17) for x in o["table"][b, :o["held"][b]]] + list(o["pool"][:o["count"]])
    before = [x for b in range(17) for x in c["table"][b, :c["held"][b]]] + list(c["free_blocks"][:c["free_count"]])
    assert sorted(owned) == sorted(before) and len(set(owned)) == len(owned)
    used = o["slots"][o["slots"] >= 0]
    assert len(set(used)) == len(used) == c["new_lens"].sum()


def test_plan_by_hand():
    # two blocks come back from an ended request, the next takes them from the top
    table = np.array([[5, 6, 7], [1, -1, -1], [2, -1, -1]], np.int32)
    o = S.plan_slots(np.array([0, 6, 0], np.int32), np.array([0, 4, 9], np.int32), table, np.array([2, 1, 1], np.int32),
                     np.array([3, 0, 0, 0, 0, 0, 0, 0], np.int32), 1, 8, 14)
    assert o["held"].tolist() == [0, 2, 2] and o["count"] == 1
    assert o["table"][1].tolist() == [1, 6, -1] and o["table"][2].tolist() == [2, 5, -1]
    assert o["slots"].tolist() == [14, 15, 48, 49, 16, 17, 18, 19, 20, 21, 22, 23, 40, -1]
    assert o["positions"].tolist() == [6, 7, 8, 9, 0, 1, 2, 3, 4, 5, 6, 7, 8, -1]
    assert o["offsets"].tolist() == [0, 0, 4, 13] and o["total"].tolist() == [0, 10, 9]


def test_plan_tree_positions_are_depths():
    par = np.array([[-1, 0, 0, 1, 3]], np.int32)
    o = S.plan_slots(np.array([7], np.int32), np.array([5], np.int32), np.array([[0, 1]], np.int32),
                     np.array([2], np.int32), np.zeros(2, np.int32), 0, 8, 5, parent=par)
    assert (o["positions"] - 7).tolist() == [0, 1, 1, 2, 3]


def test_rope_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(1)
    inv = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    q, k = r.standard_normal((1, 1, 32)), r.standard_normal((1, 1, 32))
    for pairs in ("halves", "neighbours"):
        def score(i, j):
            a = S.rope(q, np.array([[i]]), inv, [16], pairs=pairs)
            b = S.rope(k, np.array([[j]]), inv, [16], pairs=pairs)
            return float((a * b).sum())
        assert abs(score(107, 100) - score(7, 0)) < 1e-9 and abs(score(107, 100) - score(107, 90)) > 1e-3
        assert abs(np.linalg.norm(S.rope(q, np.array([[55]]), inv, [16], pairs=pairs)) - np.linalg.norm(q)) < 1e-9


def test_rope_axes():
    assert S.axis_of_pairs([2, 1, 3], "blocks").tolist() == [0, 0, 1, 2, 2, 2]
    assert S.axis_of_pairs([2, 1, 3], "rounds").tolist() == [0, 1, 2, 0, 2, 2]
    assert S.axis_of_pairs([2, 0, 1], "rounds").tolist() == [0, 2, 0]
    # equal positions on all axes: the one-axis rotation
    r = np.random.default_rng(2)
    x, inv, pos = r.standard_normal((5, 2, 16)), np.ones(8, np.float32), np.arange(5)[None]
    one = S.rope(x, pos, inv, [8])
    assert np.allclose(S.rope(x, np.repeat(pos, 3, 0), inv, [3, 1, 4], "rounds"), one)


def test_decode_is_attention_of_the_last_row():
    r = np.random.default_rng(3)
    B, Hq, Hkv, D, bs = 3, 6, 2, 64, 8
    lens = np.array([1, 37, 0], np.int32)
    kc, vc = r.standard_normal((20, bs, Hkv, D)), r.standard_normal((20, bs, Hkv, D))
    table = r.permutation(18).reshape(3, 6).astype(np.int32)
    q = r.standard_normal((B, Hq, D))
    out, lse, err, mass = S.decode_attn(q, kc, vc, table, lens, 0.3)
    assert not err.any() and (out[2] == 0).all() and (lse[2] == -np.inf).all()
    for b in (0, 1):
        k = kc[table[b]].reshape(-1, Hkv, D)[: lens[b]]
        v = vc[table[b]].reshape(-1, Hkv, D)[: lens[b]]
        t = [torch.from_numpy(np.repeat(x, Hq // Hkv, 1).transpose(1, 0, 2)) for x in (k, v)]
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b])[:, None], *t, scale=0.3)
        assert np.abs(out[b] - want[:, 0].numpy()).max() < 1e-12
    assert np.abs(lse[0] - 0.3 * np.einsum("hd,hd->h", q[0], np.repeat(kc[table[0, 0], 0], 3, 0))).max() < 1e-12
