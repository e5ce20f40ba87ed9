"""The "hooks" test build: what a wait of the tree attention kernel that runs out takes with it.  A CTA goes through many short
sequences; from the one in which a wait gives up to its last, none is complete, and all of them are told."""
import numpy as np
import pytest

import oracle
import tree_speculative_decoding_03_gb300 as tsv
import workloads as W
from gpu_util import run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks_lib():
    tsv.build(variant="hooks")
    lib = tsv.load("hooks")
    tsv.use_variant("hooks")
    yield lib
    lib.tsv_test_set_stall(0)
    tsv.use_variant(None)


@pytest.mark.parametrize("D,N,Hq", [(64, 8, 4), (128, 60, 4)])  # one and two 128-row tiles
def test_every_sequence_that_a_stalled_cta_loses_is_told(hooks_lib, D, N, Hq):
    w = W.CONFIGS[3].replace(B=1500, Hq=Hq, Hkv=1, D=D, prefix=(0, 120), N=N, depth=6, V=64, seed=7)
    inp = W.generate(w)
    assert hooks_lib.tsv_test_set_stall(1) == 0
    _, err = run_attn(inp)
    assert (err == tsv.TSV_DERR_TIMEOUT).all(), (err != tsv.TSV_DERR_TIMEOUT).sum()  # every CTA's first tile stalls
    assert hooks_lib.tsv_test_set_stall(0) == 0
    got, err = run_attn(inp)
    assert not err.any()
    want, _ = oracle.tree_verify_attn(inp)
    assert np.abs(got - want).max() <= 2e-2
