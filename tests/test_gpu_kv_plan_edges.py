"""The slot plan at the edges of its three launch forms: empty batches."""
import numpy as np
import pytest
import torch

import serving_util as U
import test_gpu_kv_plan as plan
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


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
