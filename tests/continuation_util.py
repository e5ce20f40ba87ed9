"""Inputs of the tests of the operators for several continuations of one prompt (numpy, seeded)."""
import numpy as np


def pages_state(r, B, bs, max_len, max_blocks=None, empty=0.4, shared=0.5, spare=0.3, free=20, extra=3):
    """A consistent state of B sequences: tables, held blocks, shares, the pool.  Some sequences are empty, some
    share their first blocks with an earlier one, some hold a block past their length."""
    L = r.integers(1, max_len + 1, B)
    L[r.random(B) < empty] = 0
    need = -(-L // bs)
    max_blocks = max_blocks or int(-(-max_len // bs)) + 3
    held = np.minimum(need + (L > 0) * (r.random(B) < spare), max_blocks)
    nb = int(held.sum()) + free + extra
    ids = list(r.permutation(nb))
    table, shares = r.integers(-3, nb + 3, (B, max_blocks)).astype(np.int32), np.zeros(nb, np.int32)
    for b in range(B):
        n = 0
        donors = [a for a in range(b) if L[a] > 0]
        if donors and L[b] and r.random() < shared:
            a = r.choice(donors)
            n = int(min(L[a] // bs, L[b] // bs))
            table[b, :n] = table[a, :n]
            shares[table[b, :n]] += 1
        for j in range(n, held[b]):
            table[b, j] = ids.pop()
    pool = np.full(nb, -7, np.int32)
    pool[:free] = [ids.pop() for _ in range(free)]
    return dict(seq_lens=L.astype(np.int32), table=table, held=held.astype(np.int32), shares=shares, free_blocks=pool, free_count=free)


def refs(table, held, nb):
    """How many held table entries refer to each block."""
    n = np.zeros(nb, np.int64)
    for b in range(len(held)):
        np.add.at(n, table[b, :held[b]], 1)
    return n


def fork_list(r, state, pad=2):
    """Forks of the non-empty sequences into all the empty ones, some places unused."""
    empty, used = np.flatnonzero(state["held"] == 0), np.flatnonzero(state["held"] > 0)
    F = len(empty) + pad
    src, dst = np.full(F, -1, np.int32), np.full(F, -1, np.int32)
    at = np.sort(r.permutation(F)[: len(empty)])
    if len(used):
        src[at], dst[at] = r.choice(used, len(empty)), r.permutation(empty)
    return src, dst


def prefix_case(r, members, prefix, suffix, Hq, Hkv, D, bs, cap=0, scale=None):
    """q, caches (as float32) and tables: group g has members[g] sequences that share prefix[g] keys; suffix: own
    keys of each sequence.  Slots outside the keys are NaN, and stale table entries hold anything."""
    G, B = len(members), int(sum(members))
    off = np.concatenate([[0], np.cumsum(members)]).astype(np.int32)
    of = np.repeat(np.arange(G), members)
    P = np.asarray(prefix, np.int64)[of] if B else np.zeros(0, np.int64)
    L = P + np.asarray(suffix, np.int64)
    first = np.arange(B) == off[of] if B else np.zeros(0, bool)
    mb = max(1, -(-max([cap] + list(L)) // bs))
    nb = int(sum(-(-L // bs) + 1)) + 2
    ids = list(r.permutation(nb))
    table = r.integers(-5, nb + 5, (B, mb)).astype(np.int32)
    q = r.standard_normal((B, Hq, D)).astype(np.float32)
    kc, vc = (np.full((nb, bs, Hkv, D), np.nan, np.float32) for _ in range(2))
    for b in range(B):
        # whole shared blocks are those of the first sequence; the others' entries there may hold anything
        lo = 0 if first[b] else int(P[b]) // bs
        for j in range(lo, -(-int(L[b]) // bs)):
            table[b, j] = ids.pop()
        for t in range(0 if first[b] else int(P[b]), int(L[b])):
            kc[table[b, t // bs], t % bs] = r.standard_normal((Hkv, D))
            vc[table[b, t // bs], t % bs] = r.standard_normal((Hkv, D))
    return dict(q=q, k_cache=kc, v_cache=vc, table=table, seq_lens=L.astype(np.int32), group_offsets=off,
                prefix_lens=np.asarray(prefix, np.int32), scale=scale or D ** -0.5)
