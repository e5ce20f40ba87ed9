"""The operators together, as a beam search uses them: a prompt forked, single tokens appended to every beam on shared
blocks, attention over the shared prefix, log probabilities whose alternatives choose the next beams, dropped beams
released and others forked in their places, the cache compacted in between.  The K/V rows of every beam are kept in
order on the side, and attention is computed from that record in fp64."""
import numpy as np
import pytest
import torch

from oracle import continuations as C
from test_gpu_serving_loop import TOL, Cache
import continuation_util as U
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_search(dtype):
    beams, bs, V = 5, 8, 300
    c = Cache(B=beams + 1, Hq=8, Hkv=2, D=64, bs=bs, nb=70, mb=20, seed=3, dtype=dtype)
    B, nb, i32 = c.B, 70, dict(dtype=torch.int32, device="cuda")
    shares = torch.zeros(nb, **i32)
    lists = [torch.empty(beams, **i32) for _ in range(4)]
    head = torch.randn(8 * 64, V, generator=torch.Generator().manual_seed(1)).cuda() * 0.2
    code = tsv.TSV_BF16 if dtype == torch.bfloat16 else tsv.TSV_F32
    ws = torch.empty(tsv.prefix_decode_attn_workspace_size(B, 2, 8, 2, 64, bs, 20, code), dtype=torch.uint8, device="cuda")
    seq_err = torch.empty(B, **i32)

    def append(new):
        q, k, v, offs, total, _ = c.step(new)
        for b in range(B):
            s = slice(offs[b], offs[b + 1])
            if dtype == torch.float32:  # the record holds rows rounded to bf16; the cache of a fp32 call does not
                t = np.arange(int(c.lens[b]), int(total[b]))
                at = c.table[b].cpu().numpy()[t // bs]
                k[s] = c.k[at, t % bs].double().cpu().numpy()
                v[s] = c.v[at, t % bs].double().cpu().numpy()
            c.record[b] = [np.concatenate([c.record[b][0], k[s]]), np.concatenate([c.record[b][1], v[s]])]
        c.lens.copy_(total)
        return q, offs

    def fork(pairs):
        src, dst = (torch.tensor([p[i] for p in pairs] + [-1] * (beams - len(pairs)), **i32) for i in range(2))
        err = torch.empty(beams, **i32)
        tsv.kv_fork_seqs(src, dst, c.lens, c.lens, c.table, c.held, c.held, shares, shares, c.pool, c.count, c.count, *lists[:3], bs, err)
        cerr = torch.empty(beams, **i32)
        tsv.kv_copy_blocks(c.k, c.v, lists[0], lists[1], cerr, copy_rows=lists[2])
        assert not err.any() and not cerr.any()
        for s, d in pairs:
            c.record[d] = [x.copy() for x in c.record[s]]

    def release(gone):
        keep = c.lens.clone()
        for b in gone:
            keep[b] = 0
            c.record[b] = [x[:0] for x in c.record[b]]
        tsv.kv_release_seqs(keep, c.table, c.held, c.held, shares, shares, c.pool, c.count, c.count, bs, seq_err)
        assert not seq_err.any()
        c.lens.copy_(keep)

    def compact():
        src, dst, n, err = torch.empty(nb // 2, **i32), torch.empty(nb // 2, **i32), torch.empty(1, **i32), torch.empty(nb // 2, **i32)
        tsv.kv_compact_blocks(c.table, c.table, c.held, shares, shares, c.pool, c.count, src, dst, n, seq_err,
                              torch.empty(tsv.kv_compact_workspace_size(nb), dtype=torch.uint8, device="cuda"))
        tsv.kv_copy_blocks(c.k, c.v, src, dst, err, copy_count=n)
        assert not seq_err.any() and not err.any()

    def sound():
        n = U.refs(c.table.cpu().numpy(), c.held.cpu().numpy(), nb)
        assert np.array_equal(np.maximum(n - 1, 0), shares.cpu().numpy())
        free = c.pool[: int(c.count)].cpu().numpy()
        assert len(set(free)) == len(free) and sorted(set(free) | set(np.flatnonzero(n))) == list(range(nb)) and not n[free].any()

    # a prompt of 45 tokens in row 0, an unrelated request in the last row
    append([45] + [0] * (beams - 1) + [9])
    fork([(0, b) for b in range(1, beams)])
    sound()
    score = np.zeros(beams)
    offsets = torch.tensor([0, beams, B], **i32)
    for step in range(9):
        q, offs = append([1] * B)
        sound()
        prefix = torch.tensor([45, 0], **i32)
        out, lse, err = torch.empty(B, 8, 64, dtype=dtype, device="cuda"), torch.empty(B, 8, device="cuda"), torch.empty(B, **i32)
        qb = q[:B].contiguous()
        tsv.prefix_decode_attn(qb, c.k, c.v, c.table, c.lens, offsets, prefix, out, c.D ** -0.5, workspace=ws, seq_err=err, lse=lse)
        assert not err.any()
        got = out.double().cpu().numpy()
        for b in range(B):
            assert np.abs(got[b] - c.attention(b, qb[b].double().cpu().numpy())).max() < TOL, (step, b)
        # the beams' alternatives
        logits = out[:beams].reshape(beams, -1).float() @ head
        tok = logits.argmax(-1).int()
        lp, terr = torch.empty(beams, device="cuda"), torch.empty(beams, **i32)
        ids, tops = torch.empty(beams, beams, **i32), torch.empty(beams, beams, device="cuda")
        tsv.token_logprobs(logits, tok, lp, terr, top_ids=ids, top_logprobs=tops)
        want = C.logprobs(logits.cpu().numpy(), tok.cpu().numpy(), 1.0, beams)
        assert not terr.any() and np.array_equal(ids.cpu().numpy(), want["top_ids"])
        assert np.allclose(tops.cpu().numpy(), want["top_logprobs"], atol=1e-5)
        assert np.allclose(lp.cpu().numpy(), tops[:, 0].cpu().numpy(), atol=1e-6)
        total = score[:, None] + want["top_logprobs"]
        best = np.argsort(-total.reshape(-1), kind="stable")[:beams]
        parents, score = best // beams, total.reshape(-1)[best]
        # each beam that has children goes on as one of them; the others' rows take the rest
        left = list(parents)
        for b in set(parents):
            left.remove(b)
        gone = [b for b in range(beams) if b not in parents]
        release(gone)
        fork(list(zip(left, gone)))
        order = {b: s for b, s in zip(sorted(set(parents)) + gone, score)}
        score = np.array([order[b] for b in range(beams)])
        sound()
        if step % 3 == 1:
            compact()
            sound()
            assert int(c.pool[int(c.count) - 1]) == nb - int(c.count)  # the lowest free id is next
    release(range(beams))
    sound()
    # what is left belongs to the unrelated request
    n = U.refs(c.table.cpu().numpy(), c.held.cpu().numpy(), nb)
    assert n.sum() == int(c.held[beams]) == -(-18 // bs) and not shares.any()
