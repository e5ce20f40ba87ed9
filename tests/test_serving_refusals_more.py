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
