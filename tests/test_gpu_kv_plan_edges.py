"""The slot plan at the edges of its three launch forms: empty batches; slot maps so large that a
second kernel fills them."""
import os
import re

import numpy as np
import pytest
import torch

import serving_util as U
import test_gpu_kv_plan as plan
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu

# the largest slot map that the first kernel fills itself, from its source: the cases below lie past it
SOURCE = os.path.join(os.path.dirname(tsv.HERE), "tree_speculative_decoding_03_gb300", "csrc", "serving", "kv_plan.cu")
CLUSTER_TOKENS = int(re.search(r"kPlanClusterTokens = (\d+);", open(SOURCE).read()).group(1))
FILL_CTA = 1024  # tokens of one of its CTAs


@pytest.mark.parametrize("tokens", [0, 1, 37, 600, 70000])
@pytest.mark.parametrize("tree", [None, 7])
def test_an_empty_batch_leaves_no_slot_of_the_step_before(tokens, tree):
    c = U.plan_case(np.random.default_rng(1), 0, 16, 100, 5, tree=tree, pad=tokens)
    assert c["max_tokens"] == tokens
    for in_place in (False, True):
        d = plan.device_plan(c, in_place=in_place)
        d["slots"].fill_(11)  # the step before used these
        d["positions"].fill_(3)
        plan.call(d)
        plan.check(c, d)


def test_nothing_is_appended_after_an_empty_batch():
    # a map of fixed size, as a captured step has it: the rows of the step before stay as they are
    T, i32 = 24, dict(dtype=torch.int32, device="cuda")
    c = U.plan_case(np.random.default_rng(2), 0, 16, 100, 5, pad=T)
    d = plan.device_plan(c)
    d["slots"].copy_(torch.arange(T))
    d["positions"].fill_(3)
    plan.call(d)
    rows = torch.randn(T, 6, 64, device="cuda")
    caches = [torch.randn(4, 16, 1, 64, device="cuda") for _ in range(2)]
    before = [x.clone() for x in caches]
    q, err = torch.empty(T, 4, 64, device="cuda"), torch.empty(T, **i32)
    tsv.rope_kv_append(rows[:, :4], rows[:, 4:5], rows[:, 5:], d["positions"], torch.ones(32, device="cuda"), q, *caches, d["slots"], err)
    assert all(torch.equal(x, y) for x, y in zip(caches, before)) and not q.any() and not err.any()


def large(seed, B, bs, max_len, max_new, past=0, **kw):
    """A case whose slot map is filled by the second kernel: `past` places at least past the limit."""
    c = U.plan_case(np.random.default_rng(seed), B, bs, max_len, max_new, **kw)
    c["max_tokens"] = max(c["max_tokens"], CLUSTER_TOKENS + past)
    assert c["max_tokens"] > CLUSTER_TOKENS
    return c


def run_both(c):
    """Separate outputs, the same call again, in place."""
    d = plan.device_plan(c)
    plan.call(d)
    want = plan.check(c, d)
    plan.call(d)
    plan.check(c, d)
    d = plan.device_plan(c, in_place=True)
    plan.call(d)
    plan.check(c, d)
    return want


# the token counts: well past the limit in the first group, a padded map in the second
@pytest.mark.parametrize("B,bs,max_len,max_new,kw", [
    (900, 16, 300, 250, dict(ended=0.2)), (8192, 8, 60, 24, dict(ended=0.1)), (2500, 64, 900, 70, dict(ended=0.1, pad=5)),
    (700, 16, 200, 0, dict(tree=128)), (8000, 16, 100, 0, dict(tree=11, ended=0.1)), (800, 32, 300, 300, dict(pool="exact", ended=0.3)),
    (900, 16, 300, 250, dict(pool="short", ended=0.1)), (700, 16, 200, 0, dict(tree=128, pool="short"))])
def test_large_maps(B, bs, max_len, max_new, kw):
    c = large(B + bs, B, bs, max_len, max_new, **kw)
    assert c["new_lens"].sum() > CLUSTER_TOKENS
    want = run_both(c)
    assert want["err"].any() == (kw.get("pool") == "short")


@pytest.mark.parametrize("B,bs,max_len,max_new,kw", [
    (1, 16, 0, 1, {}), (1, 8, 40, 3, {}), (7, 16, 100, 1, dict(ended=0.3)), (3, 16, 20, 9000, {}), (33, 32, 500, 0, dict(tree=128)),
    (40, 16, 300, 80, dict(pool="short")), (60, 16, 300, 0, dict(pool="short", tree=33)), (5000, 8, 60, 3, dict(ended=0.5))])
@pytest.mark.parametrize("past", [1, FILL_CTA, 70000])
def test_padded_maps(B, bs, max_len, max_new, kw, past):
    run_both(large(B, B, bs, max_len, max_new, past=past, **kw))


def test_one_sequence_fills_the_map():
    c = large(3, 3, 128, 200, 4, past=1)
    mb = 2000
    c["table"] = np.pad(c["table"], ((0, 0), (0, mb - c["table"].shape[1])), constant_values=-1)
    c["new_lens"][:] = [5, 100001, 0]
    need = 3 + int((-(-(c["seq_lens"] + c["new_lens"]) // 128)).sum())
    c["free_blocks"] = (np.arange(need) + len(c["free_blocks"])).astype(np.int32)
    c["free_blocks"] = np.concatenate([c["free_blocks"], np.full(len(c["free_blocks"]) + 40, -7, np.int32)])
    c["free_count"], c["max_tokens"] = need, 100001 + 5
    assert not run_both(c)["err"].any()


@pytest.mark.parametrize("tree", [None, 30])
@pytest.mark.parametrize("gaps", [[0, 5999], [0, 1500, 1501, 4000, 5998], [5999], [2, 1025, 1026, 2052]])
def test_more_sequences_between_two_tokens_than_a_cta_copies(gaps, tree):
    # the second kernel then searches the offsets in global memory
    c = large(4, 6000, 16, 40, 30, past=3000, tree=tree)
    new = np.zeros(6000, np.int32)
    new[gaps] = 30
    c["new_lens"] = new
    assert not run_both(c)["err"].any()


@pytest.mark.parametrize("what", ["length", "new", "held", "held_low", "capacity", "tokens", "count", "count_low", "ids", "back_ids",
                                  "pool_ids", "pool_ids_taken", "pool_full", "trees", "nodes"])
def test_bad_data_in_a_large_map(what):
    r = np.random.default_rng(31)
    tree = 120 if what in ("trees", "nodes") else None
    c = large(32, 900, 16, 300, 0 if tree else 250, tree=tree, ended=0.0 if what in ("pool_ids_taken",) else 0.1,
              spare=0.0 if what == "pool_ids_taken" else 0.1, pad=50)
    mb, nb = c["table"].shape[1], len(c["free_blocks"])
    some = r.permutation(900)[:40]
    if what == "length":
        c["seq_lens"][some] = -3
    elif what == "new":
        c["new_lens"][some] = r.choice([-1, -2 ** 31], 40)
    elif what == "held":
        c["held"][some] = mb + 7
    elif what == "held_low":
        c["held"][some] = -1
    elif what == "capacity":
        c["new_lens"][some] = mb * 16 - c["seq_lens"][some] + 1
        c["max_tokens"] = int(c["new_lens"].sum())
    elif what == "tokens":
        c["max_tokens"] = c["max_tokens"] * 2 // 3
    elif what == "count":
        c["free_count"] = nb + 1
    elif what == "count_low":
        c["free_count"] = -1
    elif what == "ids":
        c["table"][some, np.maximum(c["held"][some] - 1, 0)] = r.choice([-1, nb, 2 ** 31 - 1], 40)
    elif what == "back_ids":
        gone = np.flatnonzero((c["seq_lens"] == 0) & (c["held"] > 0) & (c["new_lens"] == 0))
        c["table"][gone] = -5
    elif what.startswith("pool_ids"):
        c["free_blocks"][r.integers(0, c["free_count"], 40)] = 2 ** 30
    elif what == "pool_full":
        c["held"][c["seq_lens"] == 0] = mb
        c["free_count"] = nb - 2
        c["free_blocks"][:] = 0
    elif what == "trees":
        c["parent"][some, r.integers(1, 120, 40)] = 121
    else:
        c["new_lens"][some[:5]] = 121
        c["max_tokens"] += 5
    assert c["max_tokens"] > CLUSTER_TOKENS
    d = plan.device_plan(c)
    plan.call(d)
    assert plan.check(c, d)["err"].any()
    d = plan.device_plan(c, in_place=True)
    plan.call(d)
    plan.check(c, d)


def test_sums_past_31_bits_in_a_large_map():
    c = large(8, 30, 16, 200, 20, past=1, ended=0.2)
    c["seq_lens"][2] = c["new_lens"][2] = 2 ** 31 - 1
    c["new_lens"][11] = 2 ** 31 - 1
    d = plan.device_plan(c)
    plan.call(d)
    assert plan.check_saturated(c, d)["err"].any()


def test_a_large_map_captured_and_replayed():
    # the second kernel reads what the first of the same replay wrote
    cases = [large(s, 700, 16, 200, 250, ended=0.2) for s in (51, 52)]
    T, nb, mb = (max(f(c) for c in cases) for f in (lambda c: c["max_tokens"], lambda c: len(c["free_blocks"]), lambda c: c["table"].shape[1]))
    for c in cases:
        c["max_tokens"], c["free_blocks"] = T, np.resize(c["free_blocks"], nb)
        assert c["table"].shape[1] == mb
    d = plan.device_plan(cases[0], in_place=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        plan.call(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.call(d)
    for c in cases + cases:
        e = plan.device_plan(c)
        for k in ("seq_lens", "new_lens", "table", "held", "free_blocks", "count"):
            d[k].copy_(e[k])
        g.replay()
        plan.check(c, d)
