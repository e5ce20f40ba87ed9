"""What the operators for several continuations refuse, answered on the host: by the C entries (the fake
pointers below would fault if anything reached a device) and by the binding's checks."""
import re

import pytest
import torch

import tree_speculative_decoding_03_gb300 as tsv

P, A, M = None, 4096, 4104  # null, 16-byte aligned, misaligned


@pytest.fixture(scope="module")
def lib():
    tsv.build()
    return tsv.load()


TABLE = [(dict(B=-1), 1), (dict(mb=0), 1), (dict(nb=0), 1), (dict(B=8193), 2), (dict(mb=1 << 27), 2), (dict(nb=(1 << 30) + 1), 2)]
BLOCKS = [(dict(bs=12), 2), (dict(bs=4), 2), (dict(bs=256), 2)]


def _fork(lib, ptrs=None, F=3, B=4, bs=16, mb=8, nb=64, err=A):
    return lib.tsv_kv_fork_seqs(*([A] * 15 if ptrs is None else ptrs), F, B, bs, mb, nb, err, P)


@pytest.mark.parametrize("kw,status", TABLE + BLOCKS + [(dict(F=-1), 1), (dict(F=8193), 2), (dict(err=P), 1)])
def test_fork_refusals(lib, kw, status):
    assert _fork(lib, **kw) == status and lib.tsv_last_error()


def test_fork_null_arrays(lib):
    for i in range(15):
        p = [A] * 15
        p[i] = P
        assert _fork(lib, p) == tsv.TSV_ERR_ARG, i


def _release(lib, ptrs=None, B=4, bs=16, mb=8, nb=64, err=A):
    return lib.tsv_kv_release_seqs(*([A] * 9 if ptrs is None else ptrs), B, bs, mb, nb, err, P)


@pytest.mark.parametrize("kw,status", TABLE + BLOCKS + [(dict(err=P), 1)])
def test_release_refusals(lib, kw, status):
    assert _release(lib, **kw) == status and lib.tsv_last_error()


def test_release_null_arrays(lib):
    for i in range(9):
        p = [A] * 9
        p[i] = P
        assert _release(lib, p) == tsv.TSV_ERR_ARG, i


def _compact(lib, ptrs=None, B=4, mb=8, nb=64, ws=A, wsb=256, err=A):
    return lib.tsv_kv_compact_blocks(*([A] * 10 if ptrs is None else ptrs), B, mb, nb, ws, wsb, err, P)


@pytest.mark.parametrize("kw,status", TABLE[:4] + [(dict(mb=(1 << 27) + 1), 2), TABLE[5], (dict(ws=P), 1), (dict(wsb=255), 1), (dict(ws=A + 2), 1), (dict(err=P), 1)])
def test_compact_refusals(lib, kw, status):
    assert _compact(lib, **kw) == status and lib.tsv_last_error()


def test_compact_null_arrays_and_workspace(lib):
    for i in range(10):
        p = [A] * 10
        p[i] = P
        assert _compact(lib, p) == tsv.TSV_ERR_ARG, i
    assert tsv.kv_compact_workspace_size(64) == 256 and tsv.kv_compact_workspace_size(0) == 0


def _copy(lib, kc=A, vc=A, src=A, dst=A, rows=P, count=P, n=3, Hkv=2, D=64, bs=16, nb=64, dt=0, err=A):
    return lib.tsv_kv_copy_blocks(kc, vc, src, dst, rows, count, n, Hkv, D, bs, nb, dt, err, P)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(n=(1 << 30) + 1), 2), (dict(Hkv=0), 1), (dict(D=96), 2), (dict(bs=24), 2), (dict(nb=0), 1), (dict(dt=2), 1),
    (dict(Hkv=1 << 23), 2), (dict(kc=P), 1), (dict(vc=P), 1), (dict(src=P), 1), (dict(dst=P), 1), (dict(err=P), 1), (dict(kc=M), 1),
    (dict(vc=M), 1)])
def test_copy_refusals(lib, kw, status):
    assert _copy(lib, **kw) == status and lib.tsv_last_error()


def test_copy_of_nothing(lib):
    assert _copy(lib, n=0, kc=P, vc=P, src=P, dst=P, err=P) == tsv.TSV_OK


def _prefix(lib, q=A, kc=A, vc=A, bt=A, sl=A, off=A, pre=A, out=A, lse=P, B=2, G=1, Hq=8, Hkv=2, D=64, bs=16, mb=4096, nb=8, scale=0.125,
            dt=0, ws=A, wsb=1 << 32, err=A):
    return lib.tsv_prefix_decode_attn(q, kc, vc, bt, sl, off, pre, out, lse, B, G, Hq, Hkv, D, bs, mb, nb, scale, dt, ws, wsb, err, P)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(G=-1), 1), (dict(G=0), 1), (dict(B=8193), 2), (dict(G=8193), 2), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=9), 1),
    (dict(B=8192, Hq=4096), 2), (dict(nb=(1 << 26) + 1), 2), (dict(D=96), 2), (dict(bs=48), 2), (dict(mb=0), 1), (dict(nb=0), 1), (dict(mb=1 << 27), 2), (dict(dt=2), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=3e38), 1),
    (dict(q=M), 1), (dict(out=M), 1), (dict(kc=M), 1), (dict(vc=M), 1), (dict(q=P), 1), (dict(bt=P), 1), (dict(sl=P), 1), (dict(off=P), 1),
    (dict(pre=P), 1), (dict(out=P), 1), (dict(err=P), 1), (dict(ws=P), 1), (dict(wsb=16), 1), (dict(ws=M), 1)])
def test_prefix_refusals(lib, kw, status):
    assert _prefix(lib, **kw) == status and lib.tsv_last_error()


def test_prefix_workspace_query(lib):
    assert _prefix(lib, B=0, G=0, q=P, out=P, ws=P, wsb=0) == tsv.TSV_OK
    size = tsv.prefix_decode_attn_workspace_size
    assert size(2, 1, 8, 2, 96, 16, 4, tsv.TSV_BF16) == 0 and size(0, 1, 8, 2, 64, 16, 4, tsv.TSV_BF16) == 0
    for dt in (tsv.TSV_BF16, tsv.TSV_F32):
        need = size(64, 3, 8, 2, 64, 16, 4096, dt)
        assert 0 < size(1, 1, 8, 2, 64, 16, 4096, dt) <= need
        assert _prefix(lib, B=64, G=3, dt=dt, wsb=need - 1) == tsv.TSV_ERR_ARG


def _logp(lib, x=A, stride=100, tok=A, T=3, V=100, temp=1.0, top=5, dt=1, lp=A, ent=P, ids=A, tops=A, err=A):
    return lib.tsv_token_logprobs(x, stride, tok, T, V, temp, top, dt, lp, ent, ids, tops, err, P)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(top=-1), 1), (dict(T=(1 << 27) + 1), 2), (dict(V=(1 << 30) + 1, stride=1 << 31), 2), (dict(top=33), 2),
    (dict(V=4, stride=4), 1), (dict(dt=2), 1), (dict(stride=99), 1), (dict(temp=0.0), 1), (dict(temp=-1.0), 1), (dict(temp=float("nan")), 1),
    (dict(temp=float("inf")), 1), (dict(temp=1e-39), 1), (dict(x=P), 1), (dict(tok=P), 1), (dict(lp=P), 1), (dict(ids=P), 1), (dict(tops=P), 1),
    (dict(err=P), 1), (dict(x=A + 2), 1), (dict(x=A + 1, dt=0), 1)])
def test_logprobs_refusals(lib, kw, status):
    assert _logp(lib, **kw) == status and lib.tsv_last_error()


def test_logprobs_of_nothing(lib):
    assert _logp(lib, T=0, x=P, tok=P, lp=P, ids=P, tops=P, err=P) == tsv.TSV_OK


def test_error_bit_matches_the_header():
    m = re.search(r"TSV_DERR_SEQ\s*=\s*(\d+)", open(tsv.HEADER).read())
    assert int(m.group(1)) == tsv.TSV_DERR_SEQ


def _each(call, ok, changes, match=None):
    for kw in changes:
        with pytest.raises(ValueError, match=match):
            call(**{**ok, **kw})
    with pytest.raises(ValueError, match="CUDA device"):  # CPU tensors
        call(**ok)


def test_binding_refuses_wrong_shapes_and_types():
    def i32(*n):
        return torch.zeros(*n, dtype=torch.int32)

    B, mb, nb, F = 3, 4, 9, 2
    per_seq = {n: i32(B) for n in ("seq_lens", "seq_lens_out", "blocks_held", "blocks_held_out")}
    per_block = {n: i32(nb) for n in ("shares", "shares_out", "free_blocks")}
    one = {n: i32(1) for n in ("free_count", "free_count_out")}
    per_fork = {n: i32(F) for n in ("fork_src", "fork_dst", "copy_src", "copy_dst", "copy_rows", "fork_err")}
    ok = dict(**per_seq, **per_block, **one, **per_fork, block_table=i32(B, mb), block_size=16)
    wrong = [{n: i32(t.numel() + 1)} for d in (per_seq, per_block, one, per_fork) for n, t in d.items()]
    wrong += [{n: t.long()} for d in (per_seq, per_block, one, per_fork) for n, t in d.items()]
    wrong += [dict(block_table=i32(mb, B).t()), dict(block_table=i32(B)), dict(shares=None)]
    _each(tsv.kv_fork_seqs, ok, wrong)

    ok = dict(keep_lens=i32(B), block_table=i32(B, mb), blocks_held=i32(B), blocks_held_out=i32(B), **per_block, **one, block_size=16,
              seq_err=i32(B))
    _each(tsv.kv_release_seqs, ok, [{n: i32(t.numel() + 1)} for n, t in ok.items() if n not in ("block_table", "block_size")] +
          [dict(block_table=i32(B + 1, mb)), dict(seq_err=torch.zeros(B))])

    ok = dict(block_table=i32(B, mb), block_table_out=i32(B, mb), blocks_held=i32(B), **per_block, free_count_out=i32(1), copy_src=i32(nb // 2),
              copy_dst=i32(nb // 2), copy_count=i32(1), seq_err=i32(B), workspace=torch.zeros(4 * nb, dtype=torch.uint8))
    _each(tsv.kv_compact_blocks, ok, [dict(copy_src=i32(nb)), dict(copy_dst=i32(3)), dict(block_table_out=i32(B, mb + 1)), dict(seq_err=i32(2)),
                                      dict(workspace=None), dict(workspace=torch.zeros(8, 8).t()), dict(copy_count=i32(2))])

    kc, vc = torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 64)
    ok = dict(k_cache=kc, v_cache=vc, copy_src=i32(F), copy_dst=i32(F), copy_err=i32(F))
    _each(tsv.kv_copy_blocks, ok, [dict(v_cache=vc.bfloat16()), dict(v_cache=vc[:2]), dict(k_cache=kc.double(), v_cache=vc.double()),
                                   dict(copy_dst=i32(3)), dict(copy_err=i32(1)), dict(copy_rows=i32(3)), dict(copy_count=i32(2)),
                                   dict(k_cache=kc[:, :8], v_cache=vc[:, :8]), dict(copy_src=i32(F).long())])

    q, out = torch.zeros(B, 8, 64), torch.zeros(B, 8, 64)
    ok = dict(q=q, k_cache=kc, v_cache=vc, block_table=i32(B, mb), seq_lens=i32(B), group_offsets=i32(3), prefix_lens=i32(2), out=out, scale=0.1,
              workspace=torch.zeros(64, dtype=torch.uint8), seq_err=i32(B))
    _each(tsv.prefix_decode_attn, ok, [dict(group_offsets=i32(2)), dict(prefix_lens=i32(2).long()), dict(prefix_lens=i32(3)), dict(out=out[:1]),
                                       dict(out=out.bfloat16()), dict(k_cache=kc.double()), dict(block_table=i32(B + 1, mb)), dict(seq_err=None),
                                       dict(lse=torch.zeros(B, 7)), dict(seq_lens=i32(B + 1)), dict(q=q.transpose(0, 1)),
                                       dict(workspace=torch.zeros(8, 8).t())])

    T, V = 5, 40
    x = torch.zeros(T, V)
    ok = dict(logits=x, tokens=i32(T), logprobs=torch.zeros(T), tok_err=i32(T), top_ids=i32(T, 3), top_logprobs=torch.zeros(T, 3))
    _each(tsv.token_logprobs, ok, [dict(logits=x.double()), dict(logits=torch.zeros(V, T).t()), dict(tokens=i32(T).long()), dict(tokens=i32(4)),
                                   dict(logprobs=torch.zeros(T).bfloat16()), dict(tok_err=i32(4)), dict(entropy=torch.zeros(4)),
                                   dict(top_ids=None), dict(top_logprobs=None), dict(top_logprobs=torch.zeros(T, 4)), dict(top_ids=i32(T))])
