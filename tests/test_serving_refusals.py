"""What the serving operators refuse, answered on the host: by the C entries (the fake
pointers below would fault if anything reached a device) and by the binding's checks."""
import ctypes

import pytest
import torch

import tree_speculative_decoding_03_gb300 as tsv

P, A, M = None, 4096, 4104  # null, 16-byte aligned, misaligned


@pytest.fixture(scope="module")
def lib():
    tsv.build()
    return tsv.load()


def _plan(lib, ptrs=None, B=4, N=8, bs=16, mb=8, nb=64, mt=32, parent=P, err=A):
    p = [A] * 13 if ptrs is None else list(ptrs)
    p[2] = parent
    return lib.tsv_kv_plan_slots(*p, B, N, bs, mb, nb, mt, err, P)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(mb=0), 1), (dict(nb=0), 1), (dict(mt=-1), 1), (dict(B=8193), 2), (dict(bs=12), 2),
    (dict(bs=4), 2), (dict(bs=256), 2), (dict(mb=1 << 27), 2), (dict(mt=(1 << 30) + 1), 2), (dict(nb=(1 << 30) + 1), 2),
    (dict(parent=A, N=0), 1), (dict(parent=A, N=129), 2), (dict(err=P), 1)])
def test_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status
    assert lib.tsv_last_error()


def test_plan_null_arrays(lib):
    for i in [0, 1] + list(range(3, 13)):
        p = [A] * 13
        p[i] = P
        assert _plan(lib, p) == tsv.TSV_ERR_ARG, i
    assert _plan(lib, [P] * 13, B=0) == tsv.TSV_OK


def _rope(lib, q=A, k=A, v=A, qo=A, kc=A, vc=A, pos=A, T=4, Hq=8, Hkv=2, D=64, qs=None, ks=None, vs=None, qos=None,
          bs=16, nb=8, dt=0, opts=None, err=A):
    qs, ks, vs, qos = (d if x is None else x for x, d in ((qs, Hq * D), (ks, Hkv * D), (vs, Hkv * D), (qos, Hq * D)))
    return lib.tsv_rope_kv_append(q, k, v, pos, A, qo, kc, vc, A, T, Hq, Hkv, D, qs, ks, vs, qos, bs, nb, dt,
                                  None if opts is None else ctypes.byref(opts), err, P)


def _opts(R=64, nei=0, axes=1, rounds=0, sec=(32, 0, 0, 0)):
    return tsv.RopeOptions(R, nei, axes, rounds, (ctypes.c_int * 4)(*sec))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(D=96), 2), (dict(bs=24), 2), (dict(nb=0), 1), (dict(dt=3), 1),
    (dict(q=M, qo=A + 64), 1), (dict(k=M), 1), (dict(v=M), 1), (dict(qo=M), 1), (dict(kc=M), 1), (dict(vc=M), 1),
    (dict(pos=P), 1), (dict(err=P), 1), (dict(qs=8 * 64 - 8), 1), (dict(ks=2 * 64 + 4), 1), (dict(vs=64), 1),
    (dict(qos=8 * 64 + 1), 1), (dict(qs=8 * 64 + 64), 1),  # in place with another stride
    (dict(opts=_opts(R=8, sec=(4, 0, 0, 0))), 2), (dict(opts=_opts(R=24, sec=(12, 0, 0, 0))), 2),
    (dict(opts=_opts(R=80, sec=(40, 0, 0, 0))), 2), (dict(opts=_opts(nei=2)), 1), (dict(opts=_opts(rounds=-1)), 1),
    (dict(opts=_opts(axes=0)), 1), (dict(opts=_opts(axes=5)), 1), (dict(opts=_opts(sec=(31, 0, 0, 0))), 1),
    (dict(opts=_opts(axes=2, sec=(33, -1, 0, 0))), 1), (dict(opts=_opts(axes=1, sec=(16, 16, 0, 0))), 1)])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert lib.tsv_last_error()


def test_rope_empty_batch(lib):
    assert _rope(lib, q=P, k=P, v=P, qo=P, kc=P, vc=P, pos=P, T=0, err=P) == tsv.TSV_OK


def _decode(lib, q=A, kc=A, vc=A, bt=A, sl=A, out=A, lse=P, B=2, Hq=8, Hkv=2, D=64, bs=16, mb=4096, nb=8, scale=0.125, dt=0,
            ws=A, wsb=1 << 30, err=A):
    return lib.tsv_decode_attn(q, kc, vc, bt, sl, out, lse, B, Hq, Hkv, D, bs, mb, nb, scale, dt, ws, wsb, err, P)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=9), 1), (dict(B=1 << 28), 2), (dict(D=96), 2), (dict(D=256), 2), (dict(bs=48), 2),
    (dict(mb=0), 1), (dict(nb=0), 1), (dict(mb=1 << 27), 2), (dict(dt=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=M), 1), (dict(out=M), 1), (dict(kc=M), 1),
    (dict(vc=M), 1), (dict(q=P), 1), (dict(bt=P), 1), (dict(sl=P), 1), (dict(err=P), 1), (dict(ws=P), 1), (dict(wsb=16), 1),
    (dict(ws=M), 1)])
def test_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status
    assert lib.tsv_last_error()


def test_decode_workspace_query(lib):
    assert _decode(lib, B=0, q=P, out=P, ws=P, wsb=0) == tsv.TSV_OK
    assert tsv.decode_attn_workspace_size(2, 8, 2, 96, 16, 4, tsv.TSV_BF16) == 0
    assert tsv.decode_attn_workspace_size(0, 8, 2, 64, 16, 4, tsv.TSV_BF16) == 0
    small, large = (tsv.decode_attn_workspace_size(B, 8, 2, 64, 16, 4096, tsv.TSV_BF16) for B in (1, 64))
    assert 0 < small <= large


def test_binding_refuses_wrong_shapes_and_types():
    i32 = dict(dtype=torch.int32)
    q, out = torch.zeros(2, 8, 64), torch.zeros(2, 8, 64)
    kc, vc = torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 64)
    bt, sl, err = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    ok = dict(q=q, k_cache=kc, v_cache=vc, block_table=bt, seq_lens=sl, out=out, scale=0.1, seq_err=err)
    for k, bad in (("out", out[:1]), ("out", out.bfloat16()), ("v_cache", vc[:2]), ("k_cache", kc.double()),
                   ("block_table", bt.long()), ("block_table", bt[:1]), ("seq_lens", sl[:1]), ("seq_lens", sl.long()),
                   ("seq_err", None), ("seq_err", err[:1]), ("lse", torch.zeros(2, 7)), ("q", q.transpose(0, 1)),
                   ("block_table", torch.zeros(4, 2, **i32).t()), ("workspace", torch.zeros(8, 8).t())):
        with pytest.raises((ValueError, tsv.TsvError)):
            tsv.decode_attn(**{**ok, k: bad})
    with pytest.raises(ValueError, match="CUDA device"):  # CPU tensors
        tsv.decode_attn(**ok)

    T = 5
    pos, inv, slots, terr = torch.zeros(T, **i32), torch.zeros(32), torch.zeros(T, dtype=torch.int64), torch.zeros(T, **i32)
    k, v, q, qo = torch.zeros(T, 2, 64), torch.zeros(T, 2, 64), torch.zeros(T, 8, 64), torch.zeros(T, 8, 64)
    ok = dict(q=q, k=k, v=v, positions=pos, inv_freq=inv, q_out=qo, k_cache=kc, v_cache=vc, slot_map=slots, tok_err=terr)
    for kw in (dict(k=k[:4]), dict(v=v.bfloat16()), dict(q_out=qo[:, :4]), dict(q=torch.zeros(T, 64, 8).transpose(1, 2)),
               dict(positions=pos.long()), dict(positions=torch.zeros(2, T, **i32)), dict(slot_map=slots.int()),
               dict(slot_map=slots[:4]), dict(tok_err=terr[:1]), dict(inv_freq=inv.double()), dict(order="x"), dict(pairs="x"),
               dict(sections=[16, 16]), dict(positions=torch.zeros(5, T, **i32), sections=[8, 8, 8, 4, 4]),
               dict(k_cache=kc[:, :8]), dict(k=torch.zeros(T, 64, 2).transpose(1, 2))):
        with pytest.raises(ValueError):
            tsv.rope_kv_append(**{**ok, **kw})
    with pytest.raises(ValueError, match="CUDA device"):
        tsv.rope_kv_append(**ok)

    B = 2
    names = ["seq_lens", "new_lens", "blocks_held", "blocks_held_out", "total_lens", "seq_err"]
    ok = {n: torch.zeros(B, **i32) for n in names}
    ok.update(block_table=bt, free_blocks=torch.zeros(9, **i32), free_count=torch.zeros(1, **i32),
              free_count_out=torch.zeros(1, **i32), token_offsets=torch.zeros(B + 1, **i32), slot_map=slots, positions=pos,
              block_size=16)
    for kw in [{n: torch.zeros(B + 1, **i32)} for n in names] + [{n: torch.zeros(B, dtype=torch.int64)} for n in names] + [
            dict(token_offsets=torch.zeros(B, **i32)), dict(positions=pos[:3]), dict(slot_map=pos), dict(free_count=torch.zeros(2, **i32)),
            dict(free_blocks=torch.zeros(9)), dict(parent=torch.zeros(3, 5, **i32)), dict(parent=torch.zeros(2, 5)),
            dict(block_table=bt.t().contiguous().t())]:
        with pytest.raises(ValueError):
            tsv.kv_plan_slots(**{**ok, **kw})
    with pytest.raises(ValueError, match="CUDA device"):
        tsv.kv_plan_slots(**ok)


def test_pool_error_bit_matches_the_header():
    import re
    m = re.search(r"TSV_DERR_POOL\s*=\s*(\d+)", open(tsv.HEADER).read())
    assert int(m.group(1)) == tsv.TSV_DERR_POOL
