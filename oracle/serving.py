"""Plain fp64 oracle of the operators around the verification step: the slot plan, the
rotary K/V append and single-token attention.  Written from their definitions, one sequence
after the other, with no code shared with the library."""
from __future__ import annotations

import numpy as np

DERR_PARENT, DERR_BLOCK, DERR_CAPACITY, DERR_POOL = 1, 2, 4, 128


def plan_slots(seq_lens, new_lens, table, held, free_blocks, free_count, block_size, max_tokens, parent=None):
    """The plan with a list as the free stack: every surplus block pushed first, then every
    fresh one popped, sequence by sequence.  Returns a dict of the call's outputs."""
    B, max_blocks = table.shape
    num_blocks = len(free_blocks)
    table, pool = table.copy(), free_blocks.copy()
    count_ok = 0 <= free_count <= num_blocks
    stack = list(pool[:free_count]) if count_ok else []
    err = np.zeros(B, np.int32)
    n = np.maximum(new_lens.astype(np.int64), 0)
    L = np.maximum(seq_lens.astype(np.int64), 0)
    ends = np.cumsum(n)
    for b in range(B):
        if (seq_lens[b] < 0 or new_lens[b] < 0 or L[b] + n[b] > max_blocks * block_size or held[b] < 0
                or held[b] > max_blocks or (n[b] > 0 and ends[b] > max_tokens)):
            err[b] |= DERR_CAPACITY
        if parent is not None and n[b] > parent.shape[1]:
            err[b] |= DERR_PARENT
        if not count_ok:
            err[b] |= DERR_POOL
    want = -(-(L + n) // block_size)
    pushed = []
    live = [b for b in range(B) if err[b] == 0]
    pushes = 0
    for b in live:
        back = int(max(0, held[b] - want[b]))
        pushes += back
        if back and free_count + pushes > num_blocks:
            err[b] |= DERR_POOL
            continue
        for j in range(want[b], held[b]):
            stack.append(table[b, j])
            pushed.append((b, table[b, j]))
    out_held, total = held.copy(), L.astype(np.int32)
    dry = False
    for b in live:
        if err[b]:
            continue
        need = int(max(0, want[b] - held[b]))
        if need and (dry or need > len(stack)):
            dry = True
            err[b] |= DERR_POOL
            continue
        for j in range(held[b], want[b]):
            table[b, j] = stack.pop()
        out_held[b] = want[b]
        total[b] = L[b] + n[b]
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int32)
    ok = err == 0
    for b in range(B):
        if not ok[b]:
            continue
        for j in range(n[b]):
            t, i = int(L[b] + j), int(ends[b] - n[b] + j)
            block = int(table[b, t // block_size])
            if 0 <= block < num_blocks:
                slots[i] = block * block_size + t % block_size
            else:
                err[b] |= DERR_BLOCK
            depth = j
            if parent is not None:
                depth, x, seen = 0, j, 0
                while x > 0 and 0 <= parent[b, x] < x:
                    x, depth = int(parent[b, x]), depth + 1
                if x != 0 or parent[b, 0] != -1:
                    err[b] |= DERR_PARENT
                    depth = None
            positions[i] = -1 if depth is None else L[b] + depth
    if count_ok and len(stack) > free_count:
        pool[free_count:len(stack)] = stack[free_count:]
        left = set()
        for p in range(free_count, len(stack)):
            left.add(p)
        for k, (b, block) in enumerate(pushed):  # a returned id outside the cache, still on the stack
            if free_count + k in left and not 0 <= block < num_blocks:
                err[b] |= DERR_BLOCK
    offsets = np.concatenate([[0], ends]).astype(np.int32)
    return dict(table=table, held=out_held.astype(np.int32), pool=pool,
                count=len(stack) if count_ok else free_count, total=total, offsets=offsets, slots=slots,
                positions=positions, err=err)


def axis_of_pairs(sections, order):
    """Axis of each rotary pair: section after section, or the axes in turn while they last."""
    left, axes = list(sections), []
    if order == "blocks":
        for a, k in enumerate(left):
            axes += [a] * k
        return np.array(axes, int)
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                axes.append(a)
                left[a] -= 1
    return np.array(axes, int)


def rope(x, positions, inv_freq, sections, order="blocks", pairs="halves"):
    """x [T, H, D] turned, in fp64.  positions [axes, T]."""
    x = x.astype(np.float64)
    R = 2 * len(inv_freq)
    axes = axis_of_pairs(sections, order)
    out = x.copy()
    for i in range(R // 2):
        theta = positions[axes[i]].astype(np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
        a, b = (i, i + R // 2) if pairs == "halves" else (2 * i, 2 * i + 1)
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out


def decode_attn(q, k_cache, v_cache, table, seq_lens, scale):
    """out [B, Hq, D], lse [B, Hq], err [B] and mass [B, Hq, D] = sum_t p_t |v_t| (the size the
    rounding of the weights acts on), in fp64."""
    B, Hq, D = q.shape
    num_blocks, bs, Hkv, _ = k_cache.shape
    max_blocks = table.shape[1]
    G = Hq // Hkv
    out, mass = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, err = np.full((B, Hq), -np.inf), np.zeros(B, np.int32)
    for b in range(B):
        L = int(seq_lens[b])
        if L < 0 or L > max_blocks * bs:
            err[b] = DERR_CAPACITY
        elif L > 0:
            ids = table[b, : -(-L // bs)]
            if ((ids < 0) | (ids >= num_blocks)).any():
                err[b] = DERR_BLOCK
        if err[b]:
            out[b], mass[b], lse[b] = np.nan, np.nan, np.nan
            continue
        if L == 0:
            continue
        rows = k_cache[ids].reshape(-1, Hkv, D)[:L].astype(np.float64)
        vals = v_cache[ids].reshape(-1, Hkv, D)[:L].astype(np.float64)
        for h in range(Hq):
            with np.errstate(all="ignore"):
                s = scale * (rows[:, h // G] @ q[b, h].astype(np.float64))
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                out[b, h] = (w @ vals[:, h // G]) / total
                mass[b, h] = (w @ np.abs(vals[:, h // G])) / total
                lse[b, h] = m + np.log(total)
    return out, lse, err, mass
