"""Operators for several continuations of one prompt (samples, beams) on the paged cache: what is
measured, and their plain forms.

  pages     sequences forked on shared blocks, blocks released by reference, the cache compacted,
            block contents copied (`kv_fork_seqs`, `kv_release_seqs`, `kv_compact_blocks`, `kv_copy_blocks`)
  prefix    attention of one new token for groups of sequences that share a prefix (`prefix_decode_attn`)
  logprobs  log probabilities of given tokens, entropy and top alternatives (`token_logprobs`)

A case's lengths are spread evenly over its range and then dealt to the sequences by the
seed, so the work of a case is the same for every seed.
"""
import math

import numpy as np
import torch

own = False

POOL = 128  # error bit: too few free blocks (the library's TSV_DERR_POOL)


# ------------------------------------------------------------------------------- the cases

def _fork(name, requests, copies, lo, hi, Hkv, D, bs, dtype, cap, pad=0, pool="ample"):
    """`copies` new sequences from each of `requests` of lo..hi tokens, and one layer's rows of the copied blocks;
    a table of `cap` slots, `pad` unused places of the fork list."""
    return dict(name=name, op="pages", kind="fork", requests=requests, copies=copies, lo=lo, hi=hi, Hkv=Hkv, D=D, bs=bs, dtype=dtype,
                cap=cap, pad=pad, pool=pool)


def _release(name, requests, copies, lo, hi, bs, cap, left):
    """`requests` groups of 1 + `copies` sequences on shared blocks, of which all but `left` a group end."""
    return dict(name=name, op="pages", kind="release", requests=requests, copies=copies, lo=lo, hi=hi, bs=bs, cap=cap, left=left)


def _compact(name, B, lo, hi, Hkv, D, bs, dtype, cap, free, scattered):
    """B sequences of lo..hi tokens in a cache with `free` percent free blocks, `scattered` percent of the blocks that
    can have to move doing so."""
    return dict(name=name, op="pages", kind="compact", B=B, lo=lo, hi=hi, Hkv=Hkv, D=D, bs=bs, dtype=dtype, cap=cap, free=free,
                scattered=scattered)


def _prefix(name, groups, mlo, mhi, plo, phi, slo, shi, Hq, Hkv, D, bs, dtype, cap=0):
    """`groups` of mlo..mhi sequences that share plo..phi keys, with slo..shi keys of their own (the new token's among them)."""
    return dict(name=name, op="prefix", groups=groups, mlo=mlo, mhi=mhi, plo=plo, phi=phi, slo=slo, shi=shi, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                dtype=dtype, cap=cap)


def _logprobs(name, T, V, top, dtype, temperature=1.0, entropy=True, extra=0, pad=0, masked=0):
    """T rows of V logits, `extra` elements between rows, `pad` rows without a token, `masked` percent of the vocabulary at -inf."""
    return dict(name=name, op="logprobs", T=T, V=V, top=top, dtype=dtype, temperature=temperature, entropy=entropy, extra=extra, pad=pad,
                masked=masked)


def listed():
    return [
        # eight samples of one prompt: latency
        _fork("fork_samples_b8", 1, 7, 2053, 2053, 8, 128, 16, "bf16", 8192),
        # a serving batch whose 64 requests go on as eight beams each, the list padded to a captured size
        _fork("fork_beams_b512", 64, 7, 512, 8191, 8, 128, 16, "bf16", 36864, pad=3),
        # the same batch when all but one or two beams of each request are dropped
        _release("release_beams_b512", 64, 7, 512, 8191, 16, 36864, 2),
        # a half-empty cache put together at its low end
        _compact("compact_cache", 40, 1, 1999, 8, 128, 16, "bf16", 8192, 48, 90),
        # eight samples of one prompt, a few tokens in: latency
        _prefix("prefix_samples_b8", 1, 8, 8, 2048, 2048, 1, 64, 32, 8, 128, 16, "bf16"),
        # a long common document under a serving batch
        _prefix("prefix_serving_b64", 1, 64, 64, 32768, 32768, 1, 512, 64, 8, 128, 16, "bf16", cap=36864),
        # ragged groups of ragged prompts
        _prefix("prefix_groups_ragged", 24, 1, 16, 0, 8191, 1, 999, 32, 8, 64, 32, "bf16"),
        # the fp32 shape
        _prefix("prefix_small_f32", 2, 3, 4, 256, 777, 1, 33, 8, 2, 64, 16, "f32"),
        # a step of a small batch with the alternatives a client asks for: latency
        _logprobs("logprobs_step_b8", 8, 128256, 20, "f32"),
        # a prompt scored, the vocabulary of the large serving mix
        _logprobs("logprobs_prompt_2000", 2000, 128256, 5, "bf16", pad=17),
        # beams: 16 alternatives of 512 rows at a temperature, rows of odd length
        _logprobs("logprobs_beams_v32k", 512, 32001, 16, "f32", temperature=0.75, extra=2, masked=10),
        # one row of a small vocabulary, no alternatives
        _logprobs("logprobs_tiny", 1, 1000, 0, "f32", entropy=False),
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["pages", "pages", "prefix", "prefix", "logprobs", "logprobs"])
    bs = rng.choice([8, 16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "pages":
        kind = rng.choice(["fork", "release", "compact"])
        hi = between(1, 16000)
        lo = rng.randrange(hi + 1)
        cap = hi + rng.randrange(1, 5000)
        most = 160000000 // (Hkv * D * (1 if dtype == "bf16" else 2))  # tokens in the cache
        if kind == "compact":
            c = _compact("", min(between(1, 600), max(1, most // (3 * hi))), min(lo, hi), hi, Hkv, D, bs, dtype, cap, rng.randrange(1, 70),
                         rng.randrange(0, 101))
        else:
            copies = between(1, 16)
            requests = min(between(1, 300), max(1, most // (2 * hi)), max(1, 4000000 * bs // (cap * (copies + 1))))
            if kind == "fork":
                c = _fork("", requests, copies, lo, hi, Hkv, D, bs, dtype, cap, pad=rng.choice([0, 0, 1, 9]),
                          pool=rng.choice(["ample", "ample", "exact", "short"]))
            else:
                c = _release("", requests, copies, lo, hi, bs, cap, rng.randrange(copies + 2))
    elif op == "prefix":
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 8])
        e = 1 if dtype == "bf16" else 4
        groups = between(1, 40)
        mhi = min(between(1, 100), max(1, 256 // groups))
        phi = between(1, 60000)
        shi = between(1, 4000)
        most = 110000000 // (Hkv * D * e * mhi * groups)  # keys of a sequence that the case can afford
        phi, shi = max(1, min(phi, most)), max(1, min(shi, most))
        phi = max(1, min(phi, 60000 * 8 // (Hq * e)))
        c = _prefix("", groups, rng.randrange(1, mhi + 1), mhi, rng.randrange(phi + 1), phi, rng.randrange(1, shi + 1), shi, Hq, Hkv, D, bs,
                    dtype, cap=rng.choice([0, 0, phi + shi + 4097]))
    else:
        V = between(50, 150000)
        T = between(1, min(4000, max(1, 128256 * 2000 // (V * (1 if dtype == "bf16" else 2)))))
        c = _logprobs("", T, V, rng.choice([0, 1, 5, 20, 32]), dtype, temperature=rng.choice([1.0, 1.0, 0.5, 0.75, 1.5]),
                      entropy=rng.random() < 0.7, extra=rng.choice([0, 0, 1, 8, 100]), pad=rng.choice([0, 0, min(T - 1, 3)]),
                      masked=rng.choice([0, 0, 30]))
    del c["name"]
    return c


# ------------------------------------------------------------------------- sizes and inputs

def _spread(lo, hi, n):
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi], np.int64)


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


def _empty(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="cuda")


def _caches(c, seed, num_blocks):
    g = _gen(seed)
    shape = (num_blocks, c["bs"], c["Hkv"], c["D"])
    return dict(k_cache=_randn(g, shape, _dtype(c)), v_cache=_randn(g, shape, _dtype(c)))


def _prepare_fork(c, seed):
    r = np.random.default_rng(seed)
    R, C, bs = c["requests"], c["copies"], c["bs"]
    B, mb = R * (C + 1), -(-c["cap"] // bs)
    L = np.zeros(B, np.int64)
    rows = r.permutation(B)
    src, dst = rows[:R], rows[R:]
    L[src] = r.permutation(_spread(c["lo"], c["hi"], R))
    held = -(-L // bs)
    of = np.repeat(np.arange(R), C)
    need = int((L[src][of] % bs > 0).sum())
    free = dict(ample=need + 40, exact=need, short=need * 3 // 4)[c["pool"]]
    num_blocks = int(held.sum()) + free + 1  # the last block is nobody's
    ids = r.permutation(num_blocks - 1)
    table = np.full((B, mb), -1, np.int32)
    table[np.arange(mb)[None, :] < held[:, None]] = ids[: held.sum()]
    pool = np.zeros(num_blocks, np.int32)
    pool[:free] = ids[held.sum():]
    shares = np.zeros(num_blocks, np.int32)
    F = R * C + c["pad"]
    fs, fd = np.full(F, -1, np.int64), np.full(F, -1, np.int64)
    at = np.sort(r.permutation(F)[: R * C])
    fs[at], fd[at] = src[of], dst
    s = dict(fork_src=_i32(fs), fork_dst=_i32(fd), lens=_i32(L), lens_out=_empty(B), table=_i32(table), held=_i32(held), held_out=_empty(B),
             shares=_i32(shares), shares_out=_empty(num_blocks), pool=_i32(pool), count=_i32([free]), count_out=_empty(1),
             copy_src=_empty(F), copy_dst=_empty(F), copy_rows=_empty(F), err=_empty(F), copy_err=_empty(F), bs=bs)
    s.update(_caches(c, seed, num_blocks))
    return s


def _prepare_release(c, seed):
    r = np.random.default_rng(seed)
    R, C, bs = c["requests"], c["copies"], c["bs"]
    B, mb = R * (C + 1), -(-c["cap"] // bs)
    L = r.permutation(_spread(c["lo"], c["hi"], R))
    rows = r.permutation(B).reshape(R, C + 1)
    full, held1 = L // bs, -(-L // bs)
    num_blocks = int((held1 + C * (held1 - full)).sum()) + 50
    ids = r.permutation(num_blocks)
    used = 0
    table, held, keep = np.full((B, mb), -1, np.int32), np.zeros(B, np.int64), np.zeros(B, np.int64)
    shares = np.zeros(num_blocks, np.int32)
    for i in range(R):
        shared = ids[used: used + full[i]]
        used += full[i]
        shares[shared] = C
        table[rows[i], : full[i]] = shared
        if held1[i] > full[i]:
            table[rows[i], full[i]] = ids[used: used + C + 1]
            used += C + 1
        held[rows[i]] = held1[i]
        keep[rows[i][: c["left"]]] = L[i]
    pool = np.zeros(num_blocks, np.int32)
    pool[: num_blocks - used] = ids[used:]
    return dict(keep=_i32(keep), table=_i32(table), held=_i32(held), held_out=_empty(B), shares=_i32(shares), shares_out=_empty(num_blocks),
                pool=_i32(pool), count=_i32([num_blocks - used]), count_out=_empty(1), err=_empty(B), bs=bs)


def _compact_sizes(c):
    """Lengths, blocks held, live blocks, all blocks, blocks that move."""
    L = _spread(c["lo"], c["hi"], c["B"])
    held = -(-L // c["bs"])
    shared = np.zeros(c["B"], np.int64)
    shared[1::2] = np.minimum(held[1::2], held[: c["B"] - 1: 2]) // 2
    n = int((held - shared).sum())
    nb = max(n * 100 // (100 - c["free"]), n) + 2
    return L, held, shared, n, nb, min(n, nb - n) * c["scattered"] // 100


def _prepare_compact(c, seed):
    r = np.random.default_rng(seed)
    B, mb = c["B"], -(-c["cap"] // c["bs"])
    _, held, shared, n, nb, moves = _compact_sizes(c)
    low = r.permutation(n)[: n - moves]
    high = n + r.permutation(nb - 1 - n)[:moves]  # (the last block stays out of it)
    ids = r.permutation(np.concatenate([low, high])).astype(np.int32)
    table, shares, used = np.full((B, mb), -1, np.int32), np.zeros(nb, np.int32), 0
    for b in range(B):
        s, h = int(shared[b]), int(held[b])
        if s:
            table[b, :s] = table[b - 1, :s]
            shares[table[b, :s]] += 1
        table[b, s:h] = ids[used: used + h - s]
        used += h - s
    deal = r.permutation(B)
    s = dict(table=_i32(table[deal]), table_out=_empty(B, mb), held=_i32(held[deal]), shares=_i32(shares), shares_out=_empty(nb),
             pool=_empty(nb).fill_(-1), count_out=_empty(1), copy_src=_empty(nb // 2), copy_dst=_empty(nb // 2), copy_count=_empty(1),
             err=_empty(B), copy_err=_empty(nb // 2), bs=c["bs"], ws=None)
    s.update(_caches(c, seed, nb))
    if own:
        import tree_speculative_decoding_03_gb300 as tsv
        s["ws"] = torch.empty(tsv.kv_compact_workspace_size(nb), dtype=torch.uint8, device="cuda")
    return s


def _prefix_sizes(c):
    """Members and prefix of each group, keys of their own of each sequence."""
    members = _spread(c["mlo"], c["mhi"], c["groups"])
    return members, _spread(c["plo"], c["phi"], c["groups"])[::-1], _spread(c["slo"], c["shi"], int(members.sum()))


def _prepare_prefix(c, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    Hq, Hkv, D, bs, dt = c["Hq"], c["Hkv"], c["D"], c["bs"], _dtype(c)
    members, P, S = _prefix_sizes(c)
    B, G = int(members.sum()), c["groups"]
    deal = r.permutation(G)
    members, P, S = members[deal], P[deal], r.permutation(S)
    of = np.repeat(np.arange(G), members)
    offsets = np.concatenate([[0], np.cumsum(members)])
    L = P[of] + S
    nb, full = -(-L // bs), P[of] // bs
    first = np.arange(B) == offsets[of]
    mb = -(-max(c["cap"], c["phi"] + c["shi"]) // bs)
    own_blocks = nb - np.where(first, 0, full)
    num_blocks = int(own_blocks.sum()) + 1
    ids = r.permutation(num_blocks).astype(np.int32)
    table = np.full((B, mb), -1, np.int32)
    j = np.arange(mb)[None, :]
    table[(j < nb[:, None]) & (first[:, None] | (j >= full[:, None]))] = ids[: own_blocks.sum()]
    table = np.where(j < full[:, None], table[offsets[of]], table)
    s = dict(q=_randn(g, (B, Hq, D), dt), k_cache=_randn(g, (num_blocks, bs, Hkv, D), dt), v_cache=_randn(g, (num_blocks, bs, Hkv, D), dt),
             table=_i32(table), seq_lens=_i32(L), offsets=_i32(offsets), prefix_lens=_i32(P), group=_i32(of), scale=D ** -0.5,
             out=torch.empty(B, Hq, D, dtype=dt, device="cuda"), lse=torch.empty(B, Hq, device="cuda"), err=_empty(B),
             longest=int(c["phi"] + c["shi"]), ws=None)
    if own:
        import tree_speculative_decoding_03_gb300 as tsv
        n = tsv.prefix_decode_attn_workspace_size(B, G, Hq, Hkv, D, bs, mb, tsv.TSV_BF16 if c["dtype"] == "bf16" else tsv.TSV_F32)
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_logprobs(c, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    T, V, dt = c["T"], c["V"], _dtype(c)
    logits = (2.5 * torch.randn(T, V + c["extra"], generator=g, device="cuda")).to(dt)
    if c["masked"]:
        logits[:, torch.rand(V + c["extra"], generator=g, device="cuda") * 100 < c["masked"]] = -math.inf
        logits[:, 0] = 0.5  # something is left
    tokens = r.integers(0, V, T)
    tokens[T - c["pad"]:] = -1
    f32 = dict(dtype=torch.float32, device="cuda")
    n = c["top"]
    return dict(logits=logits[:, :V], tokens=_i32(tokens), temperature=c["temperature"], logprobs=torch.empty(T, **f32),
                entropy=torch.empty(T, **f32) if c["entropy"] else None, top_ids=_empty(T, n) if n else None,
                top_logprobs=torch.empty(T, n, **f32) if n else None, err=_empty(T), top=n)


def prepare(case, seed):
    if own:
        import tree_speculative_decoding_03_gb300 as tsv
        tsv.load()
    kind = case.get("kind", case["op"])
    s = dict(fork=_prepare_fork, release=_prepare_release, compact=_prepare_compact, prefix=_prepare_prefix,
             logprobs=_prepare_logprobs)[kind](case, seed)
    s["kind"] = kind
    return s


# ------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return dict(fork=_plain_fork, release=_plain_release, compact=_plain_compact, prefix=_plain_prefix,
                logprobs=_plain_logprobs)[state["kind"]](state)


def _own(s):
    import tree_speculative_decoding_03_gb300 as tsv
    if s["kind"] == "fork":
        tsv.kv_fork_seqs(s["fork_src"], s["fork_dst"], s["lens"], s["lens_out"], s["table"], s["held"], s["held_out"], s["shares"],
                         s["shares_out"], s["pool"], s["count"], s["count_out"], s["copy_src"], s["copy_dst"], s["copy_rows"], s["bs"],
                         s["err"])
        tsv.kv_copy_blocks(s["k_cache"], s["v_cache"], s["copy_src"], s["copy_dst"], s["copy_err"], copy_rows=s["copy_rows"])
        return _fork_outputs(s)
    if s["kind"] == "release":
        tsv.kv_release_seqs(s["keep"], s["table"], s["held"], s["held_out"], s["shares"], s["shares_out"], s["pool"], s["count"],
                            s["count_out"], s["bs"], s["err"])
        return _release_outputs(s)
    if s["kind"] == "compact":
        tsv.kv_compact_blocks(s["table"], s["table_out"], s["held"], s["shares"], s["shares_out"], s["pool"], s["count_out"], s["copy_src"],
                              s["copy_dst"], s["copy_count"], s["err"], workspace=s["ws"])
        tsv.kv_copy_blocks(s["k_cache"], s["v_cache"], s["copy_src"], s["copy_dst"], s["copy_err"], copy_count=s["copy_count"])
        return _compact_outputs(s)
    if s["kind"] == "prefix":
        tsv.prefix_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["offsets"], s["prefix_lens"], s["out"],
                               s["scale"], workspace=s["ws"], seq_err=s["err"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"], err=s["err"])
    tsv.token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["err"], temperature=s["temperature"], entropy=s["entropy"],
                       top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return _logprobs_outputs(s)


def _fork_outputs(s):
    return {k: s[k] for k in ("lens_out", "table", "held_out", "shares_out", "count_out", "copy_src", "copy_dst", "copy_rows", "err", "k_cache",
                              "v_cache")}


def _release_outputs(s):
    return {k: s[k] for k in ("held_out", "shares_out", "pool", "count_out", "err")}


def _compact_outputs(s):
    return {k: s[k] for k in ("table_out", "shares_out", "pool", "count_out", "copy_src", "copy_dst", "copy_count", "err", "k_cache", "v_cache")}


def _logprobs_outputs(s):
    return {k: s[k] for k in ("logprobs", "entropy", "top_ids", "top_logprobs", "err") if s[k] is not None}


def _plain_fork(s):
    bs, table, pool, count = s["bs"], s["table"], s["pool"].long(), s["count"].long()
    B, mb = table.shape
    last = s["k_cache"].shape[0] - 1
    used = s["fork_src"] >= 0
    src = torch.where(used, s["fork_src"], 0).long()
    L = torch.where(used, s["lens"].long()[src], 0)
    full, rest = L // bs, L % bs
    need = (rest > 0).long()
    taken = need.cumsum(0)
    ok = used & ((need == 0) | (taken <= count))
    fresh = pool[(count - taken).clamp(min=0)]
    j = torch.arange(mb, device=table.device)[None, :]
    rows = table[src].long()
    # rows that are not written go to a row of their own behind the batch
    dst = torch.where(ok, s["fork_dst"].long(), B)
    more = torch.cat([table.long(), torch.zeros_like(table[:1]).long()])
    row = torch.where(j < full[:, None], rows, torch.where((j == full[:, None]) & (rest > 0)[:, None], fresh[:, None], more[dst]))
    more[dst] = row
    table.copy_(more[:B])
    refs = torch.where((j < full[:, None]) & ok[:, None], rows, last + 1)
    shares = torch.cat([s["shares"], s["shares"][:1]])
    shares = shares.index_add(0, refs.view(-1), torch.ones_like(refs.view(-1), dtype=torch.int32))
    s["shares_out"].copy_(shares[:-1])
    zero = torch.zeros_like(s["lens"][:1])
    held, lens = torch.cat([s["held"], zero]), torch.cat([s["lens"], zero])
    held[dst], lens[dst] = (full + need).int(), L.int()
    s["held_out"].copy_(held[:B])
    s["lens_out"].copy_(lens[:B])
    copies = ok & (rest > 0)
    s["count_out"].copy_(count - copies.sum())
    from_ = torch.where(copies, rows.gather(1, full.clamp(max=mb - 1)[:, None])[:, 0], -1)
    s["copy_src"].copy_(from_)
    s["copy_dst"].copy_(torch.where(copies, fresh, -1))
    s["copy_rows"].copy_(torch.where(copies, rest, 0))
    s["err"].copy_(torch.where(used & ~ok, POOL, 0))
    # the copied rows; those past the filled ones copy the last block's onto themselves
    r = torch.arange(bs, device=table.device)[None, :]
    take = copies[:, None] & (r < rest[:, None])
    to = torch.where(take, fresh[:, None] * bs + r, last * bs).view(-1)
    fr = torch.where(take, from_[:, None] * bs + r, last * bs).view(-1)
    k, v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    k[to] = k[fr]
    v[to] = v[fr]
    return _fork_outputs(s)


def _plain_release(s):
    bs, table, pool = s["bs"], s["table"], s["pool"]
    B, mb = table.shape
    nb = pool.numel()
    stay = torch.minimum((s["keep"] + bs - 1) // bs, s["held"])
    j = torch.arange(mb, device=table.device)[None, :]
    gone = (j >= stay[:, None]) & (j < s["held"][:, None])
    ids = torch.where(gone, table, nb).view(-1).long()
    shares = torch.cat([s["shares"], s["shares"][:1]]).index_add(0, ids, torch.full_like(ids, -1, dtype=torch.int32))[:-1]
    free = shares < 0
    place = torch.where(free, s["count"] + free.cumsum(0) - 1, nb)
    more = torch.cat([pool, pool[:1]])
    more[place] = torch.arange(nb, device=table.device, dtype=torch.int32)
    pool.copy_(more[:-1])
    s["shares_out"].copy_(shares.clamp(min=0))
    s["held_out"].copy_(stay)
    s["count_out"].copy_(s["count"] + free.sum())
    s["err"].zero_()
    return _release_outputs(s)


def _plain_compact(s):
    table = s["table"].long()
    mb, nb, half = table.shape[1], s["shares"].numel(), s["copy_src"].numel()
    ids = torch.arange(nb, device=table.device)
    mine = torch.arange(mb, device=table.device)[None, :] < s["held"][:, None]
    live = torch.zeros(nb + 1, dtype=torch.bool, device=table.device)
    live[torch.where(mine, table, nb).view(-1)] = True
    live = live[:-1]
    n = live.sum()
    high, hole = live & (ids >= n), ~live & (ids < n)
    src = torch.full((half + 1,), -1, dtype=torch.long, device=table.device)
    dst = src.clone()
    src[torch.where(high, high.cumsum(0) - 1, half)] = ids
    dst[torch.where(hole, hole.cumsum(0) - 1, half)] = ids
    moves = high.sum()
    k = torch.arange(half + 1, device=table.device) < moves
    src, dst = torch.where(k, src, -1), torch.where(k, dst, -1)
    # places past the moves write the last block, which is never a destination
    a, b = torch.where(k, src, nb - 1), torch.where(k, dst, nb - 1)
    to = ids.clone()
    to[a] = torch.where(k, dst, to[nb - 1])
    shares = torch.where(live, s["shares"], 0)
    moved = shares.clone()
    moved[b] = torch.where(k, shares[a], shares[nb - 1])
    s["shares_out"].copy_(torch.where(ids < n, moved, 0))
    s["table_out"].copy_(torch.where(mine, to[table.clamp(min=0)], table))
    s["pool"].copy_(torch.where(ids < nb - n, nb - 1 - ids, -1))
    s["count_out"].copy_(nb - n)
    s["copy_src"].copy_(src[:-1])
    s["copy_dst"].copy_(dst[:-1])
    s["copy_count"].copy_(moves)
    s["err"].zero_()
    s["k_cache"][b] = s["k_cache"][a]
    s["v_cache"][b] = s["v_cache"][a]
    return _compact_outputs(s)


def _plain_prefix(s):
    q, bs = s["q"], s["k_cache"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    t = torch.arange(s["longest"], device=q.device)[None, :]
    keys = t < s["seq_lens"][:, None]
    group = s["group"].long()
    first, prefix = s["offsets"].long()[group], s["prefix_lens"][group]
    row = torch.where(t < prefix[:, None], first[:, None], torch.arange(B, device=q.device)[:, None])
    at = (s["table"][row, t // bs].long().clamp(min=0) * bs + t % bs).view(-1)
    k = s["k_cache"].view(-1, Hkv, D)[at].view(B, -1, Hkv, D)
    qg = q.float().view(B, Hkv, Hq // Hkv, D)
    score = (qg @ k.permute(0, 2, 3, 1).float()) * s["scale"]
    del k
    score = score.masked_fill(~keys[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"].view(-1, Hkv, D)[at].view(B, -1, Hkv, D).permute(0, 2, 1, 3).float()
    v = v.masked_fill(~keys[:, None, :, None], 0.0)
    out = (p @ v) / total
    return dict(out=out.view(B, Hq, D).to(q.dtype), lse=(top + total.log()).view(B, Hq), err=torch.zeros_like(s["seq_lens"]))


def _plain_logprobs(s):
    x = s["logits"].float()
    T, V = x.shape
    used = (s["tokens"] >= 0)[:, None]
    top = x.amax(-1, keepdim=True)
    d = (x - top) / s["temperature"]
    p = d.exp()
    total = p.sum(-1, keepdim=True)
    log = total.log()
    picked = d.gather(1, s["tokens"].clamp(min=0).long()[:, None]) - log
    s["logprobs"].copy_(torch.where(used, picked, 0.0)[:, 0])
    if s["entropy"] is not None:
        h = log - (p * d.clamp(min=-1e30)).sum(-1, keepdim=True) / total
        s["entropy"].copy_(torch.where(used, h, 0.0)[:, 0])
    if s["top"]:
        # distinct keys: the value's bits in an order of whole numbers, then the lower index first
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * 2 ** 20 + (2 ** 20 - 1 - torch.arange(V, device=x.device))
        ids = 2 ** 20 - 1 - key.topk(s["top"], -1).values % 2 ** 20
        s["top_ids"].copy_(torch.where(used, ids, -1))
        s["top_logprobs"].copy_(torch.where(used, d.gather(1, ids) - log, 0.0))
    s["err"].zero_()
    return _logprobs_outputs(s)


# ------------------------------------------------------------------------- what it has to do

def work(case):
    c = case
    if c["op"] == "logprobs":
        e, rows = 2 if c["dtype"] == "bf16" else 4, c["T"] - c["pad"]
        return dict(bytes=rows * c["V"] * e + c["T"] * (12 + 4 * c["entropy"] + 8 * c["top"]), flops=6 * rows * c["V"])
    if c["op"] == "prefix":
        e = 2 if c["dtype"] == "bf16" else 4
        members, P, S = _prefix_sizes(c)
        B, row = int(members.sum()), c["Hkv"] * c["D"] * e
        keys = int(P.sum() + S.sum())
        return dict(bytes=2 * keys * row + 2 * B * c["Hq"] * c["D"] * e + 4 * B * c["Hq"] + 4 * (keys // c["bs"] + B),
                    flops=4 * int((members * P).sum() + S.sum()) * c["Hq"] * c["D"])
    bs = c["bs"]
    if c["kind"] == "compact":
        _, held, _, _, nb, moves = _compact_sizes(c)
        block = bs * c["Hkv"] * c["D"] * (2 if c["dtype"] == "bf16" else 4)
        return dict(bytes=moves * (4 * block + 8) + 8 * int(held.sum()) + 12 * nb, flops=0)
    L, C = _spread(c["lo"], c["hi"], c["requests"]), c["copies"]
    blocks = int((-(-L // bs)).sum())
    if c["kind"] == "release":
        return dict(bytes=4 * blocks * (C + 1 - min(C + 1, c["left"])) + 12 * blocks + 16 * c["requests"] * (C + 1), flops=0)
    row = c["Hkv"] * c["D"] * (2 if c["dtype"] == "bf16" else 4)
    return dict(bytes=C * int((L % bs).sum()) * row * 4 + 4 * blocks * (C + 1) + 8 * blocks + 24 * c["requests"] * C, flops=0)


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return dict(fork=_exact_fork, release=_exact_release, compact=_exact_compact, prefix=_exact_prefix,
                    logprobs=_exact_logprobs)[s["kind"]](case, s)


def _host(s, *names):
    return [s[n].cpu().numpy().copy() for n in names]


def _exact_fork(c, s):
    """One fork after the other, the free blocks a list."""
    bs = s["bs"]
    table, held, lens, shares, pool, fs, fd = _host(s, "table", "held", "lens", "shares", "pool", "fork_src", "fork_dst")
    free, F = pool[: int(s["count"])].tolist(), len(fs)
    lists = np.full((3, F), -1, np.int32)
    lists[2] = 0
    err, dry = np.zeros(F, np.int32), False
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for i in range(F):
        if fs[i] < 0:
            continue
        a, b = fs[i], fd[i]
        full, rest = divmod(int(lens[a]), bs)
        if rest:
            if dry or not free:
                dry, err[i] = True, POOL
                continue
            fresh = free.pop()
            lists[:, i] = table[a, full], fresh, rest
            k[fresh, :rest] = k[int(table[a, full]), :rest]
            v[fresh, :rest] = v[int(table[a, full]), :rest]
            table[b, full] = fresh
        table[b, :full] = table[a, :full]
        shares[table[a, :full]] += 1
        held[b], lens[b] = full + (rest > 0), lens[a]
    t = torch.from_numpy
    return dict(lens_out=t(lens), table=t(table), held_out=t(held), shares_out=t(shares), count_out=torch.tensor([len(free)], dtype=torch.int32),
                copy_src=t(lists[0]), copy_dst=t(lists[1]), copy_rows=t(lists[2]), err=t(err), k_cache=k, v_cache=v)


def _exact_release(c, s):
    bs = s["bs"]
    keep, table, held, shares, pool = _host(s, "keep", "table", "held", "shares", "pool")
    count, out, left = int(s["count"]), held.copy(), shares.astype(np.int64) + 1
    for b in range(len(held)):
        out[b] = min(held[b], -(-int(keep[b]) // bs))
        np.subtract.at(left, table[b, out[b]: held[b]], 1)
    ended = np.flatnonzero(left == 0)
    pool[count: count + len(ended)] = ended
    t = torch.from_numpy
    return dict(held_out=t(out), shares_out=t(np.maximum(left - 1, 0).astype(np.int32)), pool=t(pool),
                count_out=torch.tensor([count + len(ended)], dtype=torch.int32), err=torch.zeros(len(held), dtype=torch.int32))


def _exact_compact(c, s):
    table, held, shares, pool = _host(s, "table", "held", "shares", "pool")
    nb, half = len(shares), s["copy_src"].numel()
    live = sorted({int(x) for b in range(len(held)) for x in table[b, : held[b]]})
    n, in_use = len(live), set(live)
    src, dst = [x for x in live if x >= n], [x for x in range(n) if x not in in_use]
    to = dict(zip(live, live))
    to.update(zip(src, dst))
    new = np.zeros(nb, np.int32)
    for x in live:
        new[to[x]] = shares[x]
    out = table.copy()
    for b in range(len(held)):
        out[b, : held[b]] = [to[int(x)] for x in table[b, : held[b]]]
    pool[: nb - n] = np.arange(nb - 1, n - 1, -1)
    lists = np.full((2, half), -1, np.int32)
    lists[0, : len(src)], lists[1, : len(src)] = src, dst
    k, v = s["k_cache"].double(), s["v_cache"].double()
    if src:
        k[dst], v[dst] = k[src], v[src]
    t = torch.from_numpy
    return dict(table_out=t(out), shares_out=t(new), pool=t(pool), count_out=torch.tensor([nb - n], dtype=torch.int32), copy_src=t(lists[0]),
                copy_dst=t(lists[1]), copy_count=torch.tensor([len(src)], dtype=torch.int32), err=torch.zeros(len(held), dtype=torch.int32),
                k_cache=k, v_cache=v)


def _exact_prefix(c, s):
    """One sequence after the other, its keys gathered in order."""
    B, Hq, D = s["q"].shape
    Hkv, bs = c["Hkv"], c["bs"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, dtype=torch.float64, device="cuda")
    lens, offsets, shared = s["seq_lens"].tolist(), s["offsets"].tolist(), s["prefix_lens"].tolist()
    table = s["table"].cpu().numpy()
    for g in range(len(shared)):
        for b in range(offsets[g], offsets[g + 1]):
            t = np.arange(lens[b])
            row = np.where(t < shared[g], offsets[g], b)
            at = torch.from_numpy(table[row, t // bs].astype(np.int64) * bs + t % bs).cuda()
            k, v = (s[n].view(-1, Hkv, D)[at].double() for n in ("k_cache", "v_cache"))
            z = torch.einsum("hgd,lhd->hgl", s["q"][b].double().view(Hkv, Hq // Hkv, D), k) * s["scale"]
            lse[b] = torch.logsumexp(z, -1).reshape(Hq)
            out[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), v).reshape(Hq, D)
    return dict(out=out, lse=lse, err=None)


def _exact_logprobs(c, s):
    tokens = s["tokens"].tolist()
    T, n = len(tokens), c["top"]
    f64 = dict(dtype=torch.float64, device="cuda")
    picked, entropy, tops = torch.zeros(T, **f64), torch.zeros(T, **f64), torch.zeros(T, n, **f64)
    ids = torch.full((T, n), -1, dtype=torch.int32, device="cuda")
    for t in range(T):
        if tokens[t] < 0:
            continue
        x = s["logits"][t].double()
        logp = torch.log_softmax(x / c["temperature"], 0)
        picked[t] = logp[tokens[t]]
        entropy[t] = torch.special.entr(logp.exp()).sum()
        if n:
            order = torch.sort(x, descending=True, stable=True).indices[:n]
            ids[t], tops[t] = order.int(), logp[order]
    out = dict(logprobs=picked, err=None)
    if c["entropy"]:
        out["entropy"] = entropy
    if n:
        out.update(top_ids=ids, top_logprobs=tops)
    return out
