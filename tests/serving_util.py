"""Inputs of the serving operators' tests (numpy, seeded)."""
import numpy as np


def plan_case(r, B, bs, max_len, max_new, ended=0.0, tree=None, pool="ample", pad=0, spare=0.3):
    """A consistent allocator state and the next step's lengths, as plan_slots' arguments."""
    L = r.integers(0, max_len + 1, B)
    n = r.integers(0, max_new + 1, B) if tree is None else np.full(B, tree)
    held = -(-L // bs) + (r.random(B) < spare) * r.integers(0, 4, B)
    gone = r.random(B) < ended
    L[gone], n[gone] = 0, 0
    max_blocks = max(1, -(-(max_len + max(max_new, tree or 0)) // bs) + 3)
    held = np.minimum(held, max_blocks)
    want = -(-(L + n) // bs)
    grow, back = int(np.maximum(want - held, 0).sum()), int(np.maximum(held - want, 0).sum())
    free = dict(ample=grow + 5, exact=max(0, grow - back), short=max(0, (grow * 2) // 3 - back))[pool]
    num_blocks = max(1, int(held.sum()) + free + 3)
    ids = r.permutation(num_blocks).astype(np.int32)
    table = r.integers(-3, num_blocks + 3, (B, max_blocks)).astype(np.int32)  # stale entries hold anything
    rows = np.arange(max_blocks)[None] < held[:, None]
    table[rows] = ids[: held.sum()]
    pool_arr = np.full(num_blocks, -7, np.int32)
    pool_arr[:free] = ids[held.sum(): held.sum() + free]
    c = dict(seq_lens=L.astype(np.int32), new_lens=n.astype(np.int32), table=table, held=held.astype(np.int32),
             free_blocks=pool_arr, free_count=free, block_size=bs, max_tokens=int(n.sum()) + pad)
    if tree is not None:
        par = np.maximum(np.arange(tree)[None] - 1 - r.integers(0, 5, (B, tree)), 0)
        par[:, 0] = -1
        c["parent"] = par.astype(np.int32)
    return c


def bf16_round(x):
    """float32 -> the nearest bfloat16, as float32 (ties to even; finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)
