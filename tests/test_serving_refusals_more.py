"""More of what the serving operators refuse on the host (fake pointers: nothing reaches a device)."""
import pytest
import torch

import test_serving_refusals as refusals
import tree_speculative_decoding_03_gb300 as tsv
from test_serving_refusals import A, P, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("given", [7, 8, 10, 11, 12])
def test_plan_of_an_empty_batch_needs_all_of_its_arrays_or_none(lib, given):  # noqa: F811
    p = [P] * 13
    p[given] = A
    assert refusals._plan(lib, p, B=0) == tsv.TSV_ERR_ARG
    p = [P if i in (0, 1, 2, 3, 4, 5, 6, 9) else A for i in range(13)]
    p[given] = P
    assert refusals._plan(lib, p, B=0, err=P) == tsv.TSV_ERR_ARG


@pytest.mark.parametrize("D,most", [(64, 1 << 22), (128, 1 << 21)])
def test_rows_past_32_bit_offsets(lib, D, most):  # noqa: F811
    # a token's row of 2^28 elements is the largest: in-row offsets of the kernels have 32 bits
    for dt in (tsv.TSV_BF16, tsv.TSV_F32):
        for Hkv in (1, most + 1):
            assert refusals._decode(lib, B=1, Hq=most + 1, Hkv=Hkv, D=D, dt=dt, wsb=1 << 60) == tsv.TSV_ERR_UNSUPPORTED
        for kw in (dict(Hq=most + 1), dict(Hkv=most + 1), dict(Hq=2 ** 31 - 1, Hkv=2 ** 31 - 1)):
            assert refusals._rope(lib, qo=A + 64, D=D, dt=dt, **kw) == tsv.TSV_ERR_UNSUPPORTED, kw
    assert tsv.decode_attn_workspace_size(1, most, most, D, 16, 4, tsv.TSV_BF16) > 0
    assert tsv.decode_attn_workspace_size(1, most + 1, 1, D, 16, 4, tsv.TSV_BF16) == 0


def test_a_scale_that_overflows_in_base_two(lib):  # noqa: F811
    # scale * log2(e) has to be finite too: infinity times a score of 0 would be NaN
    for scale in (2.4e38, 3.4e38):
        assert refusals._decode(lib, scale=scale) == tsv.TSV_ERR_ARG


# What the compiled binding refuses, told apart by its message: every tensor below is on the CPU, which is
# refused last, so a check that were missing would show as that refusal instead.
I32 = dict(dtype=torch.int32)


def refused(f, message, ok, **kw):
    with pytest.raises(ValueError) as e:
        f(**{**ok, **kw})
    assert message in str(e.value) and "CUDA device" not in str(e.value), (kw.keys(), str(e.value))


def last_refusal(f, ok):
    with pytest.raises(ValueError, match="CUDA device"):
        f(**ok)


def _decode_args():
    return dict(q=torch.zeros(2, 8, 64), k_cache=torch.zeros(4, 16, 2, 64), v_cache=torch.zeros(4, 16, 2, 64), block_table=torch.zeros(2, 4, **I32),
                seq_lens=torch.zeros(2, **I32), out=torch.zeros(2, 8, 64), scale=0.1, seq_err=torch.zeros(2, **I32), lse=torch.zeros(2, 8),
                workspace=torch.zeros(64, dtype=torch.uint8))


def _rope_args():
    T = 5
    return dict(q=torch.zeros(T, 8, 64), k=torch.zeros(T, 2, 64), v=torch.zeros(T, 2, 64), positions=torch.zeros(T, **I32), inv_freq=torch.zeros(32),
                q_out=torch.zeros(T, 8, 64), k_cache=torch.zeros(4, 16, 2, 64), v_cache=torch.zeros(4, 16, 2, 64),
                slot_map=torch.zeros(T, dtype=torch.int64), tok_err=torch.zeros(T, **I32))


def _plan_args():
    B, T = 3, 7
    ok = {n: torch.zeros(B, **I32) for n in ("seq_lens", "new_lens", "blocks_held", "blocks_held_out", "total_lens", "seq_err")}
    ok.update(block_table=torch.zeros(B, 4, **I32), free_blocks=torch.zeros(9, **I32), free_count=torch.zeros(1, **I32),
              free_count_out=torch.zeros(1, **I32), token_offsets=torch.zeros(B + 1, **I32), slot_map=torch.zeros(T, dtype=torch.int64),
              positions=torch.zeros(T, **I32), block_size=16, parent=torch.zeros(B, 5, **I32))
    return ok


def wrong_forms(t, kinds):
    """Tensors like t that differ in one property each: "type", "shape", "rank", "strides"."""
    other = {torch.float32: torch.float64, torch.int32: torch.int64, torch.int64: torch.int32, torch.uint8: torch.int8}[t.dtype]
    forms = dict(type=t.to(other), shape=torch.cat([t, t[:1]]), rank=t[None],
                 strides=torch.stack([t, t], -1)[..., 0])  # every second element of another tensor
    return [forms[k] for k in kinds]


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "block_table", "seq_lens", "out", "seq_err", "lse"])
@pytest.mark.parametrize("kind", ["type", "shape", "rank", "strides"])
def test_decode_arguments(lib, name, kind):  # noqa: F811
    ok = _decode_args()
    last_refusal(tsv.decode_attn, ok)
    if (name, kind) == ("k_cache", "shape"):
        refused(tsv.decode_attn, "v_cache must be", ok, k_cache=torch.zeros(5, 16, 2, 64))  # the caches differ
        return
    refused(tsv.decode_attn, f"{name} must ", ok, **{name: wrong_forms(ok[name], [kind])[0]})


def test_decode_other_arguments(lib):  # noqa: F811
    ok = _decode_args()
    for q in (ok["q"][0], ok["q"][None]):
        refused(tsv.decode_attn, "q must have 3 dimensions", ok, q=q)
    refused(tsv.decode_attn, "q must be", ok, q=wrong_forms(ok["q"], ["strides"])[0])
    refused(tsv.decode_attn, "q must be", ok, q=ok["q"].transpose(0, 1))
    refused(tsv.decode_attn, "unsupported dtype", ok, q=ok["q"].half())
    refused(tsv.decode_attn, "out must be", ok, out=ok["out"].bfloat16())
    refused(tsv.decode_attn, "k_cache must be", ok, k_cache=torch.zeros(4, 16, 2, 128))  # another head size
    refused(tsv.decode_attn, "workspace must be contiguous", ok, workspace=torch.zeros(8, 8).t())
    for n in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "out", "seq_err"):
        refused(tsv.decode_attn, f"{n} must be a torch tensor", ok, **{n: None})
    for n in ("workspace", "lse"):
        refused(tsv.decode_attn, f"{n} must be a torch tensor", ok, **{n: 3})
    with pytest.raises(TypeError):
        tsv.decode_attn(**{**ok, "scale": "x"})


@pytest.mark.parametrize("name", ["v_cache", "positions", "inv_freq", "slot_map", "tok_err"])
@pytest.mark.parametrize("kind", ["type", "shape", "strides"])
def test_rope_arguments(lib, name, kind):  # noqa: F811
    ok = _rope_args()
    last_refusal(tsv.rope_kv_append, ok)
    if (name, kind) == ("inv_freq", "shape"):
        return  # its size is the rotary one: checked by the library
    refused(tsv.rope_kv_append, f"{name} must be", ok, **{name: wrong_forms(ok[name], [kind])[0]})


@pytest.mark.parametrize("name", ["q", "k", "v", "q_out"])
def test_rope_rows(lib, name):  # noqa: F811
    ok = _rope_args()
    t = ok[name]
    T, H, D = t.shape
    rows = torch.zeros(T, 3 * H, D)
    last_refusal(tsv.rope_kv_append, {**ok, name: rows[:, :H]})  # strided tokens are taken
    message = f"{name} must be"
    if name != "q":  # q gives the sizes and the type
        refused(tsv.rope_kv_append, message, ok, **{name: torch.zeros(T + 1, H, D)})
        refused(tsv.rope_kv_append, message, ok, **{name: torch.zeros(T, H + 1, D)})
        refused(tsv.rope_kv_append, message, ok, **{name: t.bfloat16()})
        refused(tsv.rope_kv_append, message, ok, **{name: t[0]})
    refused(tsv.rope_kv_append, message, ok, **{name: torch.zeros(T, D, H).transpose(1, 2)})  # elements apart
    refused(tsv.rope_kv_append, message, ok, **{name: torch.zeros(T, 2 * H * D).as_strided((T, H, D), (2 * H * D, D, 2))})
    refused(tsv.rope_kv_append, message, ok, **{name: rows[:, ::3]})  # heads apart
    refused(tsv.rope_kv_append, message, ok, **{name: torch.zeros(H, T, D).transpose(0, 1)})


def test_rope_other_arguments(lib):  # noqa: F811
    ok, T = _rope_args(), 5
    refused(tsv.rope_kv_append, "q must have 3 dimensions", ok, q=ok["q"][0])
    refused(tsv.rope_kv_append, "unsupported dtype", ok, q=ok["q"].half())
    refused(tsv.rope_kv_append, "k_cache must have 4 dimensions", ok, k_cache=ok["k_cache"][0])
    refused(tsv.rope_kv_append, "k_cache must be", ok, k_cache=ok["k_cache"].bfloat16())
    refused(tsv.rope_kv_append, "k_cache must be", ok, k_cache=wrong_forms(ok["k_cache"], ["strides"])[0])
    refused(tsv.rope_kv_append, "k must be", ok, k_cache=torch.zeros(4, 16, 3, 64))  # other heads than k
    refused(tsv.rope_kv_append, "v_cache must be", ok, v_cache=ok["v_cache"][:, :8])
    refused(tsv.rope_kv_append, "inv_freq must have 1 dimensions", ok, inv_freq=ok["inv_freq"][None])
    refused(tsv.rope_kv_append, "positions must be [T] or [axes, T]", ok, positions=torch.zeros(1, 1, T, **I32))
    refused(tsv.rope_kv_append, "several position axes need their sections", ok, positions=torch.zeros(2, T, **I32))
    refused(tsv.rope_kv_append, "2 sections for 1 position axes", ok, sections=[16, 16])
    refused(tsv.rope_kv_append, "5 sections for 5 position axes", ok, positions=torch.zeros(5, T, **I32), sections=[8, 8, 8, 4, 4])
    refused(tsv.rope_kv_append, "a section must hold", ok, positions=torch.zeros(2, T, **I32), sections=[-1, 33])
    refused(tsv.rope_kv_append, "a section must hold", ok, positions=torch.zeros(2, T, **I32), sections=[2 ** 40, 0])
    refused(tsv.rope_kv_append, "order must be", ok, order="x")
    refused(tsv.rope_kv_append, "pairs", ok, pairs="x")
    for n in ok:
        refused(tsv.rope_kv_append, f"{n} must be a torch tensor", ok, **{n: None})


@pytest.mark.parametrize("name", ["seq_lens", "new_lens", "blocks_held", "blocks_held_out", "total_lens", "seq_err", "block_table", "free_blocks",
                                  "free_count", "free_count_out", "token_offsets", "slot_map", "positions", "parent"])
@pytest.mark.parametrize("kind", ["type", "shape", "rank", "strides", "none"])
def test_plan_arguments(lib, name, kind):  # noqa: F811
    ok = _plan_args()
    last_refusal(tsv.kv_plan_slots, ok)
    if kind == "none":
        if name == "parent":
            last_refusal(tsv.kv_plan_slots, {**ok, "parent": None})
        else:
            refused(tsv.kv_plan_slots, f"{name} must be a torch tensor", ok, **{name: None})
        return
    bad = wrong_forms(ok[name], [kind])[0]
    if kind == "shape" and name == "free_blocks":
        last_refusal(tsv.kv_plan_slots, {**ok, name: bad})  # any number of blocks
    elif kind == "strides" and ok[name].numel() == 1:
        last_refusal(tsv.kv_plan_slots, {**ok, name: bad})  # one element has no strides
    elif kind == "shape" and name in ("slot_map", "block_table"):
        with pytest.raises(ValueError, match="must be a contiguous"):  # the other arrays' sizes follow from it
            tsv.kv_plan_slots(**{**ok, name: bad})
    else:
        refused(tsv.kv_plan_slots, f"{name} must ", ok, **{name: bad})
