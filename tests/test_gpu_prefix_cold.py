"""Attention over shared prefixes on caches that nothing has touched since they were written: loads land late and out of order
then, some of a stream's after those of the other stream's next tile.  Heads of 128 (a ring of 5 or 6 slots, which
both streams use) and groups of up to 128 rows; the first call's results are those of the next ones, and of single-token
attention."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("groups,mlo,mhi,plo,phi,slo,shi,Hq,Hkv,D,bs", [
    (24, 1, 16, 0, 8191, 1, 999, 32, 8, 128, 16), (8, 8, 8, 2000, 2000, 500, 1500, 32, 8, 128, 16), (1, 16, 16, 16384, 16384, 1, 90, 32, 8, 128, 16),
    (1, 4, 4, 30000, 30000, 1, 9, 32, 8, 128, 128), (40, 6, 6, 3000, 6000, 100, 700, 16, 4, 64, 32)])
def test_the_first_call(groups, mlo, mhi, plo, phi, slo, shi, Hq, Hkv, D, bs, seed):
    r = np.random.default_rng(seed)
    members = r.permutation(np.rint(np.linspace(mlo, mhi, groups)).astype(int))
    P = r.permutation(np.rint(np.linspace(plo, phi, groups)).astype(int)) // bs * bs  # whole blocks, so that tables can be joined
    B = int(members.sum())
    of = np.repeat(np.arange(groups), members)
    off = np.concatenate([[0], np.cumsum(members)])
    L = P[of] + r.integers(slo, shi + 1, B)
    first = np.where(np.arange(B) == off[of], 0, P[of] // bs)
    need = -(-L // bs)
    nb = int((need - first).clip(0).sum()) + 1
    ids, table = r.permutation(nb), np.zeros((B, int(need.max())), np.int32)
    for b in range(B):
        n = max(int(need[b] - first[b]), 0)
        table[b, first[b]: need[b]], ids = ids[:n], ids[n:]
        table[b, : first[b]] = table[off[of[b]], : first[b]]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def ints(x):
        return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()

    q, kc, vc = randn(B, Hq, D), randn(nb, bs, Hkv, D), randn(nb, bs, Hkv, D)
    table, lens, off, P = ints(table), ints(L), ints(off), ints(P)
    out, err, lse = torch.empty_like(q), torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, device="cuda")
    ws = torch.empty(tsv.prefix_decode_attn_workspace_size(B, groups, Hq, Hkv, D, bs, table.shape[1], tsv.TSV_BF16), dtype=torch.uint8, device="cuda")
    results = []
    for _ in range(3):
        tsv.prefix_decode_attn(q, kc, vc, table, lens, off, P, out, D ** -0.5, workspace=ws, seq_err=err, lse=lse)
        results.append((out.clone(), lse.clone(), err.clone()))
    assert not results[0][2].any()
    assert all(torch.equal(a, b) for x in results[1:] for a, b in zip(results[0], x))
    ref, ref_lse = torch.empty_like(q), torch.empty_like(lse)
    n = tsv.decode_attn_workspace_size(B, Hq, Hkv, D, bs, table.shape[1], tsv.TSV_BF16)
    tsv.decode_attn(q, kc, vc, table, lens, ref, D ** -0.5, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), seq_err=err, lse=ref_lse)
    assert not err.any()
    # two results within 2^-8 of themselves and 2^-13 of max |V| of the exact one
    tol = 2 * (2.0 ** -8 * (1 + 2.0 ** -7) * ref.float().abs() + 2.0 ** -13 * vc.abs().max().float())
    assert ((out.float() - ref.float()).abs() <= tol).all()
    assert (lse - ref_lse).abs().max() <= 2 * 2.0 ** -14 * (1 + ref_lse.abs().max())
