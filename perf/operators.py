"""The serving operators around the paged cache: what is measured, and their plain forms.

Three operators, in the order in which a decoding program calls them each step:

  plan    block tables, slot maps and positions from request lengths (`kv_plan_slots`)
  rope    rotary positions of q and k, K/V rows written at their slots (`rope_kv_append`)
  decode  attention of one new token over the paged cache (`decode_attn`)

A case's lengths are spread evenly over its range and then dealt to the sequences by the
seed, so the work of a case is the same for every seed.
"""
import math

import numpy as np
import torch

own = False

POOL = 128  # seq_err bit: the pool has too few free blocks (the library's TSV_DERR_POOL)


# ------------------------------------------------------------------------------- the cases

def _plan(name, B, lo, hi, nlo, nhi, bs, cap, tree=False, finished=0, pad=0, pool="ample"):
    """lo..hi cached tokens, nlo..nhi new ones (`tree`: N = nhi draft nodes each), a table of `cap` slots,
    every `finished`-th sequence ended (its blocks go back), `pad` unused places of the slot map."""
    return dict(name=name, op="plan", B=B, lo=lo, hi=hi, nlo=nlo, nhi=nhi, bs=bs, cap=cap, tree=tree,
                finished=finished, pad=pad, pool=pool)


def _rope(name, T, Hq, Hkv, D, R, dtype, bs, axes="", pairs="halves", order="blocks", fused=True, far=8192, pad=0):
    """T token rows of Hq query and Hkv key/value heads; R rotated dimensions; `axes`: rotary pairs of each
    axis ("" = one axis); positions up to `far`; `fused`: q, k, v are parts of one projection's rows."""
    return dict(name=name, op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, dtype=dtype, bs=bs, axes=axes, pairs=pairs,
                order=order, fused=fused, far=far, pad=pad)


def _decode(name, B, Hq, Hkv, D, lo, hi, bs, dtype, cap=0):
    """One new token for each of B sequences over lo..hi keys; a table of `cap` slots (0: as many as needed)."""
    return dict(name=name, op="decode", B=B, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, bs=bs, dtype=dtype, cap=cap)


def listed():
    return [
        # a small batch verifying chains of 5 drafts: latency of one small launch
        _plan("plan_chain_b8", 8, 2048, 2048, 6, 6, 16, 8192, tree=True),
        # the large serving mix: 64 trees of 64 nodes, an eighth of the requests just ended
        _plan("plan_serving_b64", 64, 512, 32768, 64, 64, 16, 36864, tree=True, finished=8),
        # a prefill batch of many ragged prompts, the slot map padded to the captured size
        _plan("plan_prefill_b1000", 1000, 0, 7001, 1, 511, 16, 8192, finished=10, pad=777),
        # one new token for 8 sequences
        _rope("rope_step_b8", 8, 32, 8, 128, 128, "bf16", 16, fused=True),
        # the serving mix's 64 trees of 64 nodes, one projection's rows
        _rope("rope_tree_serving", 4096, 64, 8, 128, 128, "bf16", 16, far=32768),
        # a prompt of video patches: time, height and width, rows of an odd number, padded
        _rope("rope_video_axes", 20011, 32, 8, 128, 128, "bf16", 16, axes="16,24,24", far=100000, pad=101),
        # fp32, half of a small head rotated in neighbouring pairs
        _rope("rope_partial_f32", 777, 8, 2, 64, 32, "f32", 32, pairs="neighbours", fused=False),
        # the tiny fp32 shape: one sequence, latency
        _decode("decode_tiny_f32", 1, 8, 2, 64, 256, 256, 16, "f32"),
        # a draft or target step of a small batch
        _decode("decode_chain_b8", 8, 32, 8, 128, 2048, 2048, 16, "bf16"),
        # the large serving mix, ragged
        _decode("decode_serving_b64", 64, 64, 8, 128, 512, 32768, 16, "bf16", cap=36864),
        # two very long requests: few rows, a long axis
        _decode("decode_long_b2", 2, 64, 8, 128, 120001, 131071, 64, "bf16"),
        # fp32 caches of a middling ragged batch
        _decode("decode_ragged_f32_b13", 13, 32, 8, 128, 1, 9001, 16, "f32"),
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "rope", "rope", "decode", "decode"])
    bs = rng.choice([8, 16, 32, 64, 128])
    if op == "plan":
        B = between(1, 2000)
        tree = rng.random() < 0.5
        hi = between(1, 30000)
        nhi = between(1, 128 if tree else 600)
        nlo = nhi if rng.random() < 0.5 else between(1, nhi)
        c = _plan("", B, rng.randrange(hi + 1), hi, nlo, nhi, bs, hi + nhi + rng.randrange(1, 3 * bs), tree=tree,
                  finished=rng.choice([0, 0, 3, 7]), pad=rng.choice([0, 0, 1, 513]),
                  pool=rng.choice(["ample", "ample", "exact", "short"]))
        if B * c["cap"] // bs > 4000000:  # the table itself stays moderate
            c["B"] = max(1, 4000000 * bs // c["cap"])
    elif op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 5, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        R = rng.choice([D, D, D // 2, D - 16])
        n = rng.choice([1, 1, 2, 3, 4])
        cuts = sorted(rng.sample(range(1, R // 2), n - 1)) if n > 1 else []
        axes = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [R // 2])) if n > 1 else ""
        T = between(1, min(30000, 1200000 // (Hq + 2 * Hkv)))
        c = _rope("", T, Hq, Hkv, D, R, rng.choice(["bf16", "bf16", "f32"]), bs, axes=axes,
                  pairs=rng.choice(["halves", "neighbours"]), order=rng.choice(["blocks", "rounds"]),
                  fused=rng.random() < 0.7, far=between(1, 1000000), pad=rng.choice([0, 0, 1, 37]))
    else:
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hi = between(1, 100000)
        most = 900000000 // (Hkv * D * (2 if dtype == "bf16" else 4))  # keys in all
        B = min(between(1, 300), max(1, most // hi))
        hi = min(hi, most)
        c = _decode("", B, Hq, Hkv, D, rng.randrange(hi + 1), hi, bs, dtype, cap=rng.choice([0, 0, hi + 4097]))
    del c["name"]
    return c


# ------------------------------------------------------------------------- sizes and inputs

def _spread(lo, hi, n):
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi], np.int64)


def _plan_lengths(c):
    """Cached and new lengths before the seed deals them (ended sequences have none of either)."""
    L, n = _spread(c["lo"], c["hi"], c["B"]), _spread(c["nlo"], c["nhi"], c["B"])[::-1].copy()
    if c["finished"]:
        L[:: c["finished"]] = 0
        n[:: c["finished"]] = 0
    return L, n


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _prepare_plan(c, seed):
    r = np.random.default_rng(seed)
    B, bs, N = c["B"], c["bs"], c["nhi"]
    L, n = _plan_lengths(c)
    deal = r.permutation(B)
    L, n = L[deal], n[deal]
    # blocks held: those of the cached tokens, some left from a longer tree before; an ended
    # sequence still holds what it had
    max_blocks = -(-c["cap"] // bs)
    held = -(-L // bs) + (r.random(B) < 0.3) * r.integers(0, 1 + 64 // bs, B)
    held = np.where((L == 0) & (n == 0), r.integers(1, 2 + c["hi"] // bs, B), held)
    held = np.minimum(held, max_blocks)
    want = -(-(L + n) // bs)
    grow, back = np.maximum(want - held, 0).sum(), np.maximum(held - want, 0).sum()
    free = dict(ample=int(grow) + 64, exact=max(0, int(grow - back)), short=max(0, int(grow * 3 // 4 - back)))[c["pool"]]
    # the cache has room for every such deal; blocks neither held nor free belong to others
    num_blocks = int((-(-L // bs) - (-(n + bs) // bs)).sum()) + B * (64 // bs) + 64
    num_blocks += (B // c["finished"] + 1) * (2 + c["hi"] // bs) if c["finished"] else 0
    assert held.sum() + free <= num_blocks
    ids = r.permutation(num_blocks).astype(np.int32)
    table = np.full((B, max_blocks), -1, np.int32)
    row = np.arange(max_blocks)[None, :] < held[:, None]
    table[row] = ids[: int(held.sum())]
    pool = np.zeros(num_blocks, np.int32)
    pool[:free] = ids[int(held.sum()): int(held.sum()) + free]
    s = dict(seq_lens=_i32(L), new_lens=_i32(n), table=_i32(table), held=_i32(held), pool=_i32(pool),
             count=_i32(np.array([free])), parent=None, bs=bs)
    if c["tree"]:
        # random trees: each node below one of the few before it
        par = np.arange(N)[None, :] - 1 - r.integers(0, 4, (B, N))
        par = np.maximum(par, 0)
        par[:, 0] = -1
        s["parent"] = _i32(par)
    T = int(n.sum()) + c["pad"]
    T = max(T, 1)
    dev = dict(dtype=torch.int32, device="cuda")
    s.update(held_out=torch.empty(B, **dev), count_out=torch.empty(1, **dev), total=torch.empty(B, **dev),
             offsets=torch.empty(B + 1, **dev), slots=torch.empty(T, dtype=torch.int64, device="cuda"),
             positions=torch.empty(T, **dev), err=torch.empty(B, **dev))
    return s


def _sections(c):
    return [int(x) for x in c["axes"].split(",")] if c["axes"] else [c["R"] // 2]


def _axis_of_pair(c):
    """Which axis a rotary pair takes its position from: sections one after the other, or in rounds (every
    axis in turn while it has pairs left)."""
    sec = _sections(c)
    if c["order"] == "blocks":
        return np.repeat(np.arange(len(sec)), sec)
    left, out = list(sec), []
    while len(out) < c["R"] // 2:
        for a in range(len(sec)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return np.array(out)


def _prepare_rope(c, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    T, Hq, Hkv, D, bs = c["T"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    pad = min(c["pad"], T // 2)
    dt = _dtype(c)
    if c["fused"]:
        rows = _randn(g, (T, (Hq + 2 * Hkv) * D), dt)
        q = rows[:, : Hq * D].view(T, Hq, D)
        k = rows[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        v = rows[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    else:
        q, k, v = (_randn(g, (T, h, D), dt) for h in (Hq, Hkv, Hkv))
    nb = -(-T // bs)
    num_blocks = nb + nb // 4 + 2
    blocks = r.permutation(num_blocks - 1)[:nb].astype(np.int64)  # the last block stays free
    t = np.arange(T)
    slots = blocks[t // bs] * bs + t % bs
    slots[T - pad:] = -1
    A = len(_sections(c))
    start = r.integers(0, c["far"], A)
    pos = np.stack([(start[a] + t // (1 if a == 0 else 7 ** a)) % c["far"] for a in range(A)])
    pos[:, T - pad:] = -1
    inv = (10000.0 ** (-np.arange(c["R"] // 2) / (c["R"] // 2))).astype(np.float32)
    return dict(q=q, k=k, v=v, positions=_i32(pos), inv_freq=torch.from_numpy(inv).cuda(),
                k_cache=_randn(g, (num_blocks, bs, Hkv, D), dt), v_cache=_randn(g, (num_blocks, bs, Hkv, D), dt),
                slots=torch.from_numpy(slots).cuda(), axis=torch.from_numpy(_axis_of_pair(c)).cuda(),
                sections=_sections(c), order=c["order"], pairs=c["pairs"], q_out=torch.empty(T, Hq, D, dtype=dt, device="cuda"),
                err=torch.empty(T, dtype=torch.int32, device="cuda"))


def _prepare_decode(c, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    dt = _dtype(c)
    L = r.permutation(_spread(c["lo"], c["hi"], B))
    nb = -(-L // bs)
    max_blocks = max(1, -(-max(c["cap"], c["hi"]) // bs))
    num_blocks = int(nb.sum()) + 1
    table = np.full((B, max_blocks), -1, np.int32)
    table[np.arange(max_blocks)[None, :] < nb[:, None]] = r.permutation(num_blocks)[: int(nb.sum())]
    s = dict(q=_randn(g, (B, Hq, D), dt), k_cache=_randn(g, (num_blocks, bs, Hkv, D), dt),
             v_cache=_randn(g, (num_blocks, bs, Hkv, D), dt), table=_i32(table), seq_lens=_i32(L), scale=D ** -0.5,
             out=torch.empty(B, Hq, D, dtype=dt, device="cuda"), lse=torch.empty(B, Hq, device="cuda"),
             err=torch.empty(B, dtype=torch.int32, device="cuda"), longest=int(c["hi"]), ws=None)
    if own:
        import tree_speculative_decoding_03_gb300 as tsv
        n = tsv.decode_attn_workspace_size(B, Hq, Hkv, D, bs, max_blocks, tsv.TSV_BF16 if c["dtype"] == "bf16" else tsv.TSV_F32)
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    if own:
        import tree_speculative_decoding_03_gb300 as tsv
        tsv.load()
    s = dict(plan=_prepare_plan, rope=_prepare_rope, decode=_prepare_decode)[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return dict(plan=_plain_plan, rope=_plain_rope, decode=_plain_decode)[state["op"]](state)


def _own(s):
    import tree_speculative_decoding_03_gb300 as tsv
    if s["op"] == "plan":
        tsv.kv_plan_slots(s["seq_lens"], s["new_lens"], s["table"], s["held"], s["held_out"], s["pool"], s["count"],
                          s["count_out"], s["total"], s["offsets"], s["slots"], s["positions"], s["bs"], s["err"],
                          parent=s["parent"])
        return dict(table=s["table"], held=s["held_out"], pool=s["pool"], count=s["count_out"], total=s["total"],
                    offsets=s["offsets"], slots=s["slots"], positions=s["positions"], err=s["err"])
    if s["op"] == "rope":
        tsv.rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"],
                           s["slots"], s["err"], sections=s["sections"], order=s["order"], pairs=s["pairs"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"], err=s["err"])
    tsv.decode_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["out"], s["scale"],
                    workspace=s["ws"], seq_err=s["err"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"], err=s["err"])


def _plain_plan(s):
    bs, table, pool = s["bs"], s["table"], s["pool"]
    B, mb = table.shape
    L, n, h, count = s["seq_lens"].long(), s["new_lens"].long(), s["held"].long(), s["count"].long()
    want = (L + n + bs - 1) // bs
    grow, back = (want - h).clamp(min=0), (h - want).clamp(min=0)
    grow_end, back_end = grow.cumsum(0), back.cumsum(0)
    top = count + back_end[-1]  # blocks free once the surplus is back
    fits = (grow == 0) | (grow_end <= top)
    grow = torch.where(fits, grow, torch.zeros_like(grow))
    first = grow_end - (want - h).clamp(min=0)

    def stack(p):
        """Block at place p of the free stack: the pool's own, then the surplus in order of sequence."""
        item = (p - count).clamp(min=0)
        b = torch.searchsorted(back_end, item, right=True).clamp(max=B - 1)
        i = (want[b] + item - (back_end[b] - back[b])).clamp(0, mb - 1)
        return torch.where(p < count, pool[p.clamp(0, pool.numel() - 1)], table[b, i])

    j = torch.arange(mb, device=table.device)[None, :]
    fresh = (j >= h[:, None]) & (j < want[:, None]) & fits[:, None]
    new_table = torch.where(fresh, stack(top - 1 - (first[:, None] + j - h[:, None])), table)
    left = top - grow.sum()
    place = torch.arange(pool.numel(), device=table.device)
    new_pool = torch.where((place >= count) & (place < left), stack(place), pool)

    ends = n.cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends]).int()
    t = torch.arange(s["slots"].numel(), device=table.device)
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    i = t - (ends[b] - n[b])
    used = (t < ends[-1]) & fits[b]
    at = (L[b] + i).clamp(0, mb * bs - 1)
    slots = torch.where(used, new_table[b, at // bs].long() * bs + at % bs, torch.full_like(t, -1))
    depth = i
    if s["parent"] is not None:
        # each node's distance from the root, its ancestors followed in steps that double
        up = s["parent"].long()
        N = up.shape[1]
        far = (up >= 0).long()
        up = torch.where(up < 0, torch.zeros_like(up), up)
        for _ in range(max(1, (N - 1).bit_length())):
            far = far + far.gather(1, up)
            up = up.gather(1, up)
        depth = far[b, i.clamp(0, N - 1)]
    positions = torch.where(used, L[b] + depth, torch.full_like(t, -1)).int()
    held = torch.where(fits, want, h).int()
    total = torch.where(fits, L + n, L).int()
    err = torch.where(fits, torch.zeros_like(L), torch.full_like(L, POOL)).int()
    table.copy_(new_table)
    pool.copy_(new_pool)
    return dict(table=table, held=held, pool=pool, count=left.int(), total=total, offsets=offsets, slots=slots,
                positions=positions, err=err)


def _turn(x, cos, sin, R, halves):
    """The first R dimensions of each head rotated by its pairs' angles."""
    x = x.float()
    a, b = (x[..., : R // 2], x[..., R // 2: R]) if halves else (x[..., 0:R:2], x[..., 1:R:2])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([y, z], -1) if halves else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s):
    R = 2 * s["inv_freq"].numel()
    halves = s["pairs"] == "halves"
    used = s["slots"] >= 0
    angle = s["positions"].double()[s["axis"]].t() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    row = used[:, None, None]
    q = torch.where(row, _turn(s["q"], cos, sin, R, halves), 0.0).to(s["q"].dtype)
    kc, vc = s["k_cache"], s["v_cache"]
    Hkv, D = kc.shape[2:]
    kc, vc = kc.view(-1, Hkv, D), vc.view(-1, Hkv, D)
    # rows without a slot write the last row, which no sequence owns, with what it holds
    at = torch.where(used, s["slots"], torch.full_like(s["slots"], kc.shape[0] - 1))
    kc[at] = torch.where(row, _turn(s["k"], cos, sin, R, halves).to(kc.dtype), kc[-1])
    vc[at] = torch.where(row, s["v"], vc[-1])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], err=torch.zeros_like(s["slots"], dtype=torch.int32))


def _plain_decode(s):
    q, table, bs = s["q"], s["table"], s["k_cache"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    nb = max(1, -(-s["longest"] // bs))
    ids = table[:, :nb].clamp(min=0).long()
    keys = torch.arange(nb * bs, device=q.device)[None, :] < s["seq_lens"][:, None]  # [B, keys]
    k = s["k_cache"][ids].view(B, nb * bs, Hkv, D)
    qg = q.float().view(B, Hkv, Hq // Hkv, D)
    score = (qg @ k.permute(0, 2, 3, 1).float()) * s["scale"]  # [B, Hkv, G, keys]
    del k
    score = score.masked_fill(~keys[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][ids].view(B, nb * bs, Hkv, D).permute(0, 2, 1, 3).float()
    v = v.masked_fill(~keys[:, None, :, None], 0.0)
    empty = (s["seq_lens"] == 0)[:, None, None, None]
    out = torch.where(empty, 0.0, (p @ v) / total)
    lse = (top + total.log()).view(B, Hq)
    return dict(out=out.view(B, Hq, D).to(q.dtype), lse=lse, err=torch.zeros_like(s["seq_lens"]))


# ------------------------------------------------------------------------- what it has to do

def work(case):
    c = case
    if c["op"] == "plan":
        L, n = _plan_lengths(c)
        T, B, bs = int(n.sum()), c["B"], c["bs"]
        touched = int((-(-(L + n) // bs) - L // bs).sum())
        return dict(bytes=12 * (T + c["pad"]) + 32 * B + 8 * touched + (4 * B * c["nhi"] if c["tree"] else 0), flops=0)
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        T, D = c["T"], c["D"]
        T -= min(c["pad"], T // 2)
        A = len(_sections(c))
        return dict(bytes=2 * T * (c["Hq"] + 2 * c["Hkv"]) * D * e + c["T"] * (4 * A + 12),
                    flops=3 * T * (c["Hq"] + c["Hkv"]) * c["R"])
    L = int(_spread(c["lo"], c["hi"], c["B"]).sum())
    return dict(bytes=2 * L * c["Hkv"] * c["D"] * e + 2 * c["B"] * c["Hq"] * c["D"] * e + 4 * (L // c["bs"] + c["B"]),
                flops=4 * L * c["Hq"] * c["D"])


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return dict(plan=_exact_plan, rope=_exact_rope, decode=_exact_decode)[case["op"]](case, s)


def _exact_plan(c, s):
    """A free list that is pushed to and popped from, one sequence after the other."""
    bs = s["bs"]
    L, n, held = (s[k].cpu().numpy().astype(np.int64) for k in ("seq_lens", "new_lens", "held"))
    table, pool = s["table"].cpu().numpy().copy(), s["pool"].cpu().numpy().copy()
    free = pool[: int(s["count"])].tolist()
    parent = None if s["parent"] is None else s["parent"].cpu().numpy()
    want = -(-(L + n) // bs)
    for b in range(len(L)):
        free += table[b, want[b]:held[b]].tolist()
    T = s["slots"].numel()
    slots, positions = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    offsets = np.concatenate([[0], np.cumsum(n)])
    err, new_held, total, exhausted = np.zeros(len(L), np.int32), want.copy(), L + n, False
    for b in range(len(L)):
        need = max(0, want[b] - held[b])
        exhausted = exhausted or need > len(free)
        if exhausted and need:
            err[b], new_held[b], total[b] = POOL, held[b], L[b]
            continue
        for j in range(held[b], want[b]):
            table[b, j] = free.pop()
        at = np.arange(L[b], L[b] + n[b])
        where = slice(offsets[b], offsets[b] + n[b])
        slots[where] = table[b, at // bs].astype(np.int64) * bs + at % bs
        deep = np.arange(n[b])
        if parent is not None:
            deep = np.zeros(n[b], np.int64)
            for i in range(1, n[b]):
                deep[i] = deep[parent[b, i]] + 1
        positions[where] = L[b] + deep
    old = int(s["count"])
    if len(free) > old:
        pool[old:len(free)] = free[old:]
    t = torch.from_numpy
    return dict(table=t(table), held=t(new_held.astype(np.int32)), pool=t(pool), count=torch.tensor([len(free)], dtype=torch.int32),
                total=t(total.astype(np.int32)), offsets=t(offsets.astype(np.int32)), slots=t(slots), positions=t(positions), err=t(err))


def _exact_rope(c, s):
    """Each pair as a complex number times e^(i * position * frequency)."""
    R, T = c["R"], c["T"]
    axis = _axis_of_pair(c)
    pos = s["positions"].cpu().numpy().astype(np.float64)
    inv = s["inv_freq"].cpu().numpy().astype(np.float64)
    turn = torch.from_numpy(np.exp(1j * (pos[axis].T * inv))).cuda()[:, None, :]

    def rotate(x):
        x = x.double()
        if c["pairs"] == "halves":
            z = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2: R].contiguous()) * turn
            return torch.cat([z.real, z.imag, x[..., R:]], -1)
        z = torch.view_as_complex(x[..., :R].reshape(T, -1, R // 2, 2)) * turn
        return torch.cat([torch.view_as_real(z).reshape(T, -1, R), x[..., R:]], -1)

    slots = s["slots"].cpu().numpy()
    rows = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q[rows] = rotate(s["q"])[rows]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    Hkv, D = kc.shape[2:]
    to = s["slots"][rows]
    kc.view(-1, Hkv, D)[to] = rotate(s["k"])[rows]
    vc.view(-1, Hkv, D)[to] = s["v"].double()[rows]
    return dict(q=q, k_cache=kc, v_cache=vc, err=None)


def _exact_decode(c, s):
    """One sequence after the other, its keys gathered in order."""
    B, Hq, D = s["q"].shape
    Hkv, bs = c["Hkv"], c["bs"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["seq_lens"].tolist()
    for b, L in enumerate(lens):
        if L == 0:
            continue
        ids = s["table"][b, : -(-L // bs)].long()
        k = s["k_cache"][ids].reshape(-1, Hkv, D)[:L].double()
        v = s["v_cache"][ids].reshape(-1, Hkv, D)[:L].double()
        q = s["q"][b].double().view(Hkv, Hq // Hkv, D)
        z = torch.einsum("hgd,lhd->hgl", q, k) * s["scale"]
        lse[b] = torch.logsumexp(z, -1).reshape(Hq)
        out[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), v).reshape(Hq, D)
    return dict(out=out, lse=lse, err=None)
