"""More of what the serving operators refuse on the host (fake pointers: nothing reaches a device)."""
import pytest

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
