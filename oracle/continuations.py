"""Plain fp64 oracle of the operators for several continuations of one prompt: cache blocks by
reference, attention over shared prefixes, token log probabilities.  Written from their
definitions, one sequence, block or row after the other, with no code shared with the library."""
from __future__ import annotations

import numpy as np

DERR_BLOCK, DERR_CAPACITY, DERR_TOKEN, DERR_NONFINITE, DERR_POOL, DERR_SEQ = 2, 4, 8, 16, 128, 256


def fork(fork_src, fork_dst, seq_lens, table, held, shares, free_blocks, free_count, block_size):
    B, max_blocks = table.shape
    nb, F, bs = len(shares), len(fork_src), block_size
    table, lens_out, held_out, shares = table.copy(), seq_lens.copy(), held.copy(), shares.copy()
    count_ok = 0 <= free_count <= nb
    stack = list(free_blocks[:free_count]) if count_ok else []
    err = np.zeros(F, np.int32)
    src, dst, rows = (np.full(F, v, np.int32) for v in (-1, -1, 0))
    named = [d for s, d in zip(fork_src, fork_dst) if s >= 0]
    dry = False
    for i, (s, d) in enumerate(zip(fork_src, fork_dst)):
        if s < 0:
            continue
        if s >= B or not 0 <= d < B or named.count(d) > 1 or held[d] != 0:
            err[i] = DERR_SEQ
            continue
        L, h = int(seq_lens[s]), int(held[s])
        if L < 0 or not 0 <= h <= max_blocks or -(-L // bs) > h:
            err[i] = DERR_CAPACITY
            continue
        if not count_ok:
            err[i] = DERR_POOL
            continue
        full, rest = divmod(L, bs)
        if rest:
            if dry or not stack:
                dry, err[i] = True, DERR_POOL
                continue
            fresh, last = stack.pop(), table[s, full]
            table[d, full] = fresh
            if 0 <= last < nb and 0 <= fresh < nb:
                src[i], dst[i], rows[i] = last, fresh, rest
            else:
                err[i] |= DERR_BLOCK
        for j in range(full):
            table[d, j] = table[s, j]
            if 0 <= table[s, j] < nb:
                shares[table[s, j]] += 1
            else:
                err[i] |= DERR_BLOCK
        lens_out[d], held_out[d] = L, full + (rest > 0)
    return dict(table=table, seq_lens=lens_out, held=held_out, shares=shares, count=len(stack) if count_ok else free_count, copy_src=src,
                copy_dst=dst, copy_rows=rows, err=err)


def release(keep_lens, table, held, shares, free_blocks, free_count, block_size):
    B, max_blocks = table.shape
    nb = len(shares)
    pool, held_out = free_blocks.copy(), held.copy()
    left = shares.astype(np.int64) + 1  # references
    count_ok = 0 <= free_count <= nb
    err, given = np.zeros(B, np.int32), [[] for _ in range(B)]
    for b in range(B):
        if keep_lens[b] < 0 or not 0 <= held[b] <= max_blocks:
            err[b] = DERR_CAPACITY
            continue
        if not count_ok:
            err[b] = DERR_POOL
            continue
        held_out[b] = min(int(held[b]), -(-int(keep_lens[b]) // block_size))
        for j in range(held_out[b], held[b]):
            if 0 <= table[b, j] < nb:
                left[table[b, j]] -= 1
                given[b].append(table[b, j])
            else:
                err[b] |= DERR_BLOCK
    free = np.flatnonzero(left <= 0) if count_ok else np.zeros(0, np.int64)
    lost = count_ok and free_count + len(free) > nb
    for b in range(B):
        if err[b] & (DERR_CAPACITY | DERR_POOL):
            continue
        if any(left[x] < 0 for x in given[b]) or (lost and held_out[b] < held[b]):
            err[b] |= DERR_POOL
    count = free_count
    for x in free:
        if count < nb:
            pool[count] = x
            count += 1
    return dict(held=held_out, shares=np.maximum(left - 1, 0).astype(np.int32), pool=pool, count=count, err=err)


def compact(table, held, shares, free_blocks):
    B, max_blocks = table.shape
    nb = len(shares)
    err, live = np.zeros(B, np.int32), set()
    for b in range(B):
        if not 0 <= held[b] <= max_blocks:
            err[b] = DERR_CAPACITY
            continue
        ids = table[b, :held[b]]
        if any(not 0 <= x < nb for x in ids):
            err[b] = DERR_BLOCK
        live |= {int(x) for x in ids if 0 <= x < nb}
    n = len(live)
    movers, holes = sorted(x for x in live if x >= n), sorted(set(range(n)) - live)
    to = {x: x for x in live} | dict(zip(movers, holes))
    out, new = table.copy(), np.zeros(nb, np.int32)
    for x in live:
        new[to[x]] = shares[x]
    for b in range(B):
        if err[b] & DERR_CAPACITY:
            continue
        for j in range(held[b]):
            out[b, j] = to.get(int(table[b, j]), table[b, j])
    pool = free_blocks.copy()
    pool[:nb - n] = np.arange(nb - 1, n - 1, -1)
    src, dst = np.full(nb // 2, -1, np.int32), np.full(nb // 2, -1, np.int32)
    src[:len(movers)], dst[:len(movers)] = movers, holes
    return dict(table=out, shares=new, pool=pool, count=nb - n, copy_src=src, copy_dst=dst, copy_count=len(movers), err=err)


def copy_blocks(cache, copy_src, copy_dst, copy_rows=None, count=None):
    """(the cache [num_blocks, bs, ...] after the copies, the error of each)."""
    out, nb, bs = cache.copy(), cache.shape[0], cache.shape[1]
    n = len(copy_src) if count is None else min(max(count, 0), len(copy_src))
    err = np.zeros(len(copy_src), np.int32)
    for i in range(n):
        s, d = copy_src[i], copy_dst[i]
        if s < 0:
            continue
        if s >= nb or not 0 <= d < nb:
            err[i] = DERR_BLOCK
            continue
        r = bs if copy_rows is None else min(max(int(copy_rows[i]), 0), bs)
        out[d, :r] = cache[s, :r]
    return out, err


def prefix_attn(q, k_cache, v_cache, table, seq_lens, group_offsets, prefix_lens, scale):
    """fp64 attention over each sequence's keys in order; (out, lse, err)."""
    B, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    cap = table.shape[1] * bs
    out, lse, err = np.full((B, Hq, D), np.nan), np.full((B, Hq), np.nan), np.zeros(B, np.int32)
    off = np.asarray(group_offsets)
    if off[0] != 0 or off[-1] != B or (np.diff(off) < 0).any():
        return out, lse, np.full(B, DERR_SEQ, np.int32)
    for g, P in enumerate(prefix_lens):
        for b in range(off[g], off[g + 1]):
            L = int(seq_lens[b])
            if L < 0 or L > cap or P < 0 or P > L:
                err[b] = DERR_CAPACITY
                continue
            t = np.arange(L)
            ids = table[np.where(t < P, off[g], b), t // bs]
            if ((ids < 0) | (ids >= nb)).any():
                err[b] = DERR_BLOCK
                continue
            if L == 0:
                out[b], lse[b] = 0.0, -np.inf
                continue
            k, v = k_cache[ids, t % bs].astype(np.float64), v_cache[ids, t % bs].astype(np.float64)
            for h in range(Hq):
                z = k[:, h // (Hq // Hkv)] @ q[b, h].astype(np.float64) * scale
                m = z.max()
                w = np.exp(z - m)
                lse[b, h] = m + np.log(w.sum())
                out[b, h] = w @ v[:, h // (Hq // Hkv)] / w.sum()
    return out, lse, err


def logprobs(logits, tokens, temperature=1.0, top=0):
    T, V = logits.shape
    lp, ent, err = np.zeros(T), np.zeros(T), np.zeros(T, np.int32)
    ids, tops = np.full((T, top), -1, np.int32), np.zeros((T, top))
    for t in range(T):
        x = logits[t].astype(np.float64)
        if tokens[t] < 0:
            continue
        if tokens[t] >= V:
            err[t] = DERR_TOKEN
        elif np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
            err[t] = DERR_NONFINITE
        if err[t]:
            lp[t] = ent[t] = np.nan
            tops[t] = np.nan
            continue
        z = (x - x.max()) / temperature
        p = np.exp(z)
        logp = z - np.log(p.sum())
        lp[t] = logp[tokens[t]]
        some = p > 0
        ent[t] = -(np.exp(logp[some]) * logp[some]).sum()
        order = np.lexsort((np.arange(V), -(x + 0.0)))[:top]
        ids[t], tops[t] = order, logp[order]
    return dict(logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=tops, err=err)
