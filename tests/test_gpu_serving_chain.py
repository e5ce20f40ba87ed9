"""The serving operators one behind the other in a stream, with no other kernel between them: each
may be resident while the one before still writes what it reads.  The outputs are those of the
same calls with a synchronisation after each."""
import numpy as np
import pytest
import torch

import serving_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, MB, STEPS = 48, 8, 2, 64, 16, 24, 8


def run(wait, graph=False):
    """STEPS steps of plan (in place), append and attention; single tokens and small prompts."""
    r = np.random.default_rng(3)
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    nb = B * MB
    lens, held, table = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.full((B, MB), -1, **i32)
    pool, count = cu(r.permutation(nb).astype(np.int32)), torch.tensor([nb], **i32)
    kc, vc = (torch.full((nb, BS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    inv = cu((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
    ws = torch.empty(tsv.decode_attn_workspace_size(B, HQ, HKV, D, BS, MB, tsv.TSV_BF16), dtype=torch.uint8, device="cuda")
    T = B * 30
    # made before the first call: what the steps write is allocated, not computed
    new = [cu(r.integers(0, 30, B).astype(np.int32)) if s % 3 == 0 else torch.ones(B, **i32) for s in range(STEPS)]
    rows = [cu(U.bf16_round(r.standard_normal((T, HQ + 2 * HKV, D)).astype(np.float32))).bfloat16() for _ in range(STEPS)]
    q = cu(U.bf16_round(r.standard_normal((B, HQ, D)).astype(np.float32))).bfloat16()
    kept = []
    for s in range(STEPS):
        kept.append(dict(offs=torch.empty(B + 1, **i32), slots=torch.empty(T, dtype=torch.int64, device="cuda"), pos=torch.empty(T, **i32),
                         err=torch.empty(B, **i32), terr=torch.empty(T, **i32), qo=torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda"),
                         out=torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, HQ, device="cuda"),
                         derr=torch.empty(B, **i32), lens=None))
    torch.cuda.synchronize()

    def steps():
        for s, k in enumerate(kept):
            x = rows[s]
            tsv.kv_plan_slots(lens, new[s], table, held, held, pool, count, count, lens, k["offs"], k["slots"], k["pos"], BS, k["err"])
            wait()
            tsv.rope_kv_append(x[:, :HQ], x[:, HQ: HQ + HKV], x[:, HQ + HKV:], k["pos"], inv, k["qo"], kc, vc, k["slots"], k["terr"])
            wait()
            tsv.decode_attn(q, kc, vc, table, lens, k["out"], 0.125, workspace=ws, seq_err=k["derr"], lse=k["lse"])
            wait()

    if graph:
        state = [lens, held, table, pool, count, kc, vc]
        start = [x.clone() for x in state]
        steps()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        for x, y in zip(state, start):
            x.copy_(y)
        g.replay()
    else:
        steps()
    torch.cuda.synchronize()
    return [x for k in kept for x in (k["offs"], k["slots"], k["pos"], k["err"], k["terr"], k["qo"], k["out"], k["lse"], k["derr"])] + [
        lens, held, table, pool, count, kc.nan_to_num(), vc.nan_to_num()]


@pytest.mark.parametrize("graph", [False, True])
def test_chained_calls_read_what_the_calls_before_wrote(graph):
    want = run(torch.cuda.synchronize)
    assert not want[3].any() and int(want[-7].max()) > 60
    for _ in range(5):
        got = run(lambda: None, graph)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_plan_in_place_then_attention():
    # nothing between the two: the attention reads the lengths and the table that the plan has just written
    r = np.random.default_rng(5)
    i32 = dict(dtype=torch.int32, device="cuda")
    nb = B * MB
    kc, vc = (torch.randn(nb, BS, HKV, D, device="cuda") for _ in range(2))
    q = torch.randn(B, HQ, D, device="cuda")
    new = [torch.from_numpy(r.integers(0, 20, B).astype(np.int32)).cuda() for _ in range(STEPS)]
    ids = torch.from_numpy(r.permutation(nb).astype(np.int32)).cuda()
    ws = torch.empty(tsv.decode_attn_workspace_size(B, HQ, HKV, D, BS, MB, tsv.TSV_F32), dtype=torch.uint8, device="cuda")

    def steps(wait):
        lens, held, table = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.full((B, MB), -1, **i32)
        pool, count = ids.clone(), torch.tensor([nb], **i32)
        outs = [(torch.empty(B, HQ, D, device="cuda"), torch.empty(B, HQ, device="cuda"), torch.empty(B, **i32)) for _ in new]
        offs, err = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        slots, pos = torch.empty(B * 20, dtype=torch.int64, device="cuda"), torch.empty(B * 20, **i32)
        torch.cuda.synchronize()
        for n, (out, lse, derr) in zip(new, outs):
            tsv.kv_plan_slots(lens, n, table, held, held, pool, count, count, lens, offs, slots, pos, BS, err)
            wait()
            tsv.decode_attn(q, kc, vc, table, lens, out, 0.125, workspace=ws, seq_err=derr, lse=lse)
            wait()
        torch.cuda.synchronize()
        assert not err.any()
        return [x for o in outs for x in o] + [lens, table]

    want = steps(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(steps(lambda: None), want))
