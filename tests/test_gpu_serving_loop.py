"""The operators together, as a decoding program uses them: requests of different lengths,
one ending and another beginning on its blocks, single tokens and draft trees on one cache.
The K/V rows every step wrote are kept in order on the side, and attention is computed
from that record in fp64."""
import numpy as np
import pytest
import torch

from oracle import serving as S
import serving_util as U
import tree_speculative_decoding_03_gb300 as tsv
import workloads as W

pytestmark = pytest.mark.gpu


class Cache:
    def __init__(self, B, Hq, Hkv, D, bs, nb, mb, seed, dtype=torch.bfloat16):
        self.B, self.Hq, self.Hkv, self.D, self.bs, self.dtype = B, Hq, Hkv, D, bs, dtype
        i32 = dict(dtype=torch.int32, device="cuda")
        self.r = np.random.default_rng(seed)
        self.k, self.v = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.table = torch.full((B, mb), -1, **i32)
        self.held, self.lens = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.pool, self.count = torch.from_numpy(self.r.permutation(nb).astype(np.int32)).cuda(), torch.tensor([nb], **i32)
        self.inv = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
        self.record = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(B)]

    def step(self, new, parent=None, lens_out=None):
        """Plan and append random rows; returns q as turned on the device, and the plan."""
        B, i32 = self.B, dict(dtype=torch.int32, device="cuda")
        n = torch.tensor(new, **i32)
        T = int(sum(new)) + 3
        offs, slots = torch.empty(B + 1, **i32), torch.empty(T, dtype=torch.int64, device="cuda")
        pos, err, terr = torch.empty(T, **i32), torch.empty(B, **i32), torch.empty(T, **i32)
        total = torch.empty(B, **i32) if lens_out is None else lens_out
        tsv.kv_plan_slots(self.lens, n, self.table, self.held, self.held, self.pool, self.count, self.count, total, offs,
                          slots, pos, self.bs, err, parent=parent)
        heads = self.Hq + 2 * self.Hkv
        rows = U.bf16_round(self.r.standard_normal((T, heads, self.D)).astype(np.float32))
        x = torch.from_numpy(rows).to(self.dtype).cuda()
        q = torch.empty(T, self.Hq, self.D, dtype=self.dtype, device="cuda")
        tsv.rope_kv_append(x[:, : self.Hq], x[:, self.Hq: self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:], pos,
                           torch.from_numpy(self.inv).cuda(), q, self.k, self.v, slots, terr)
        assert not err.any() and not terr.any()
        p = pos.cpu().numpy()
        turned = U.bf16_round(S.rope(rows[:, self.Hq: self.Hq + self.Hkv], p[None], self.inv, [self.D // 2]).astype(np.float32))
        return q, turned, rows[:, self.Hq + self.Hkv:], offs.cpu().numpy(), total, p

    def attention(self, b, q, extra=None):
        """fp64 attention of q [Hq, D] over the record of sequence b (then `extra` rows)."""
        k, v = self.record[b]
        if extra is not None:
            k, v = np.concatenate([k, extra[0]]), np.concatenate([v, extra[1]])
        G = self.Hq // self.Hkv
        out = np.zeros((self.Hq, self.D))
        for h in range(self.Hq):
            s = k[:, h // G] @ q[h] * self.D ** -0.5
            w = np.exp(s - s.max())
            out[h] = w @ v[:, h // G] / w.sum()
        return out


# The bounds below: weights and results are rounded to bf16 (2^-7 of sum p |v|, see the
# attention's own test), and a K element may be the bf16 neighbour of the record's where the two
# angles' difference straddles a rounding (2^-7 of the element: a score moves by at most
# 2^-7 * scale * sum |q k|, on a few elements only).  |v| < 5 here: 0.05 covers both.
TOL = 0.05


def test_single_tokens_with_requests_that_come_and_go():
    c = Cache(B=5, Hq=8, Hkv=2, D=64, bs=16, nb=40, mb=12, seed=1)
    prompts = [0, 37, 16, 100, 0]
    B = c.B

    def append(new):
        q, k, v, offs, total, _ = c.step(new)
        for b in range(B):
            s = slice(offs[b], offs[b + 1])
            c.record[b] = [np.concatenate([c.record[b][0], k[s]]), np.concatenate([c.record[b][1], v[s]])]
        c.lens.copy_(total)
        return q, offs

    append(prompts)
    for step in range(20):
        if step == 6:  # request 3 ends, its blocks go back; request 4 begins
            c.lens[3] = 0
            c.record[3] = [x[:0] for x in c.record[3]]
            append([0, 0, 0, 0, 60])
            assert int(c.held[3]) == 0
        live = [b for b in range(B) if len(c.record[b][0]) > 0] if step else [1, 2, 3]
        new = [1 if b in live else 0 for b in range(B)]
        q, offs = append(new)
        out, lse = torch.empty(B, c.Hq, c.D, dtype=c.dtype, device="cuda"), torch.empty(B, c.Hq, device="cuda")
        err = torch.empty(B, dtype=torch.int32, device="cuda")
        ws = torch.empty(tsv.decode_attn_workspace_size(B, c.Hq, c.Hkv, c.D, c.bs, c.table.shape[1], tsv.TSV_BF16),
                         dtype=torch.uint8, device="cuda")
        qb = torch.zeros(B, c.Hq, c.D, dtype=c.dtype, device="cuda")
        for b in live:
            qb[b] = q[offs[b]]
        tsv.decode_attn(qb, c.k, c.v, c.table, c.lens, out, c.D ** -0.5, workspace=ws, seq_err=err, lse=lse)
        assert not err.any()
        got = out.float().cpu().numpy()
        for b in range(B):
            if b in live:
                assert np.abs(got[b] - c.attention(b, qb[b].double().cpu().numpy())).max() < TOL, (step, b)
            else:
                assert (got[b] == 0).all()
        held = c.held.cpu().numpy()
        owned = [int(x) for b in range(B) for x in c.table[b, : held[b]]] + c.pool[: int(c.count)].tolist()
        assert sorted(owned) == list(range(40))


def test_draft_trees_then_single_tokens():
    B, N = 4, 24
    c = Cache(B=B, Hq=8, Hkv=2, D=128, bs=16, nb=120, mb=16, seed=2)
    q, k, v, offs, total, _ = c.step([30, 1, 77, 16])
    for b in range(B):
        s = slice(offs[b], offs[b + 1])
        c.record[b] = [k[s], v[s]]
    c.lens.copy_(total)
    i32 = dict(dtype=torch.int32, device="cuda")
    for step in range(4):
        par = np.stack([W.random_tree(np.random.default_rng(10 * step + b), N, 6) for b in range(B)])
        parent = torch.from_numpy(par).cuda()
        q, k, v, offs, total, pos = c.step([N] * B, parent=parent)
        qt = q[: B * N].view(B, N, c.Hq, c.D).contiguous()
        out, err = torch.empty_like(qt), torch.empty(B, **i32)
        ws = torch.empty(max(16, tsv.attn_workspace_size(B, N, c.Hq, c.Hkv, c.D, c.bs, c.table.shape[1], tsv.TSV_BF16)),
                         dtype=torch.uint8, device="cuda")
        tsv.tree_verify_attn(qt, c.k, c.v, c.table, c.lens, parent, out, c.D ** -0.5, workspace=ws, seq_err=err)
        assert not err.any()
        got = out.float().cpu().numpy()
        paths = []
        for b in range(B):
            path = [int(np.random.default_rng(b + step).integers(0, N))]
            while par[b, path[0]] >= 0:
                path.insert(0, int(par[b, path[0]]))
            paths.append(path)
            at = [offs[b] + j for j in path]
            assert [int(pos[i]) for i in at] == [int(c.lens[b]) + d for d in range(len(path))]
            want = c.attention(b, qt[b, path[-1]].double().cpu().numpy(), extra=(k[at], v[at]))
            assert np.abs(got[b, path[-1]] - want).max() < TOL, (step, b)
            c.record[b] = [np.concatenate([c.record[b][0], k[at]]), np.concatenate([c.record[b][1], v[at]])]
        nodes = np.full((B, N), -1, np.int32)
        for b, p in enumerate(paths):
            nodes[b, : len(p)] = p
        new_lens = torch.empty(B, **i32)
        tsv.kv_compact_accepted(c.k, c.v, c.table, c.lens, torch.from_numpy(nodes).cuda(),
                                torch.tensor([len(p) - 1 for p in paths], **i32), new_lens, err)
        assert not err.any()
        c.lens.copy_(new_lens)
        # the moved rows keep their depth's position: a single token reads the accepted path as a chain
        q, k, v, offs, total, _ = c.step([1] * B)
        for b in range(B):
            s = slice(offs[b], offs[b + 1])
            c.record[b] = [np.concatenate([c.record[b][0], k[s]]), np.concatenate([c.record[b][1], v[s]])]
        c.lens.copy_(total)
        out1, lse = torch.empty(B, c.Hq, c.D, dtype=c.dtype, device="cuda"), torch.empty(B, c.Hq, device="cuda")
        ws = torch.empty(tsv.decode_attn_workspace_size(B, c.Hq, c.Hkv, c.D, c.bs, c.table.shape[1], tsv.TSV_BF16),
                         dtype=torch.uint8, device="cuda")
        tsv.decode_attn(q[:B].contiguous(), c.k, c.v, c.table, c.lens, out1, c.D ** -0.5, workspace=ws, seq_err=err, lse=lse)
        got = out1.float().cpu().numpy()
        for b in range(B):
            assert np.abs(got[b] - c.attention(b, q[b].double().cpu().numpy())).max() < TOL, (step, b)


def test_single_token_attention_is_the_tree_attention_of_one_node():
    # a tree of the root alone, whose own row is the last key
    w = W.CONFIGS[3].replace(B=4, Hq=16, Hkv=4, D=128, prefix=(0, 700), N=1, tree="chain", V=16, seed=77)
    inp = W.generate(w)
    from gpu_util import device_inputs, run_attn
    want, err = run_attn(inp)
    assert not err.any()
    d = device_inputs(inp, verify=False)
    out = torch.empty(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(tsv.decode_attn_workspace_size(4, 16, 4, 128, 16, inp["max_blocks"], tsv.TSV_BF16), dtype=torch.uint8, device="cuda")
    tsv.decode_attn(d["q"].view(4, 16, 128), d["k_cache"], d["v_cache"], d["block_table"], d["seq_lens"] + 1, out, inp["scale"],
                    workspace=ws, seq_err=e)
    # both are within 2^-7 sum p |v| of the exact result, |v| < 5
    assert not e.any() and np.abs(out.float().cpu().numpy().reshape(want.shape) - want).max() <= 2 * 2.0 ** -7 * 5


def test_a_step_on_a_stream_of_its_own():
    # all three operators on a side stream, against the same step on the default one
    def step(stream):
        c = Cache(B=3, Hq=4, Hkv=2, D=64, bs=8, nb=30, mb=8, seed=9)
        i32 = dict(dtype=torch.int32, device="cuda")
        n, T = torch.tensor([5, 17, 0], **i32), 22
        offs, slots, pos = torch.empty(4, **i32), torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, **i32)
        err, terr, total, derr = (torch.empty(k, **i32) for k in (3, T, 3, 3))
        x = torch.from_numpy(U.bf16_round(c.r.standard_normal((T, 8, 64)).astype(np.float32))).to(c.dtype).cuda()
        q, out = torch.empty(T, 4, 64, dtype=c.dtype, device="cuda"), torch.empty(3, 4, 64, dtype=c.dtype, device="cuda")
        inv, lse = torch.from_numpy(c.inv).cuda(), torch.empty(3, 4, device="cuda")
        ws = torch.empty(tsv.decode_attn_workspace_size(3, 4, 2, 64, 8, 8, tsv.TSV_BF16), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        tsv.kv_plan_slots(c.lens, n, c.table, c.held, c.held, c.pool, c.count, c.count, total, offs, slots, pos, 8, err, stream=stream)
        tsv.rope_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], pos, inv, q, c.k, c.v, slots, terr, stream=stream)
        tsv.decode_attn(q[:3], c.k, c.v, c.table, total, out, 0.125, workspace=ws, seq_err=derr, lse=lse, stream=stream)
        torch.cuda.synchronize()
        assert not err.any() and not terr.any() and not derr.any()
        return [c.table, c.held, c.pool[:20], c.count, total, offs, slots, pos, q, out, lse]

    for a, b in zip(step(None), step(torch.cuda.Stream())):
        assert torch.equal(a, b)
    assert torch.isfinite(a[:2]).all() and (a[2] == -float("inf")).all()
