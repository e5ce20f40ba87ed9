"""Token log probabilities on a GPU that cannot hold a cluster of eight: the "hooks" test build treats clusters above a given
size as not resident, and the smaller cluster or the single CTA of a row gives the same."""
import numpy as np
import pytest
import torch

import test_gpu_logprobs as logprobs
import tree_speculative_decoding_03_gb300 as tsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def hooks_lib():
    tsv.build(variant="hooks")
    lib = tsv.load("hooks")
    tsv.use_variant("hooks")
    yield lib
    lib.tsv_test_set_logprobs_cluster(8)
    tsv.use_variant(None)


@pytest.mark.parametrize("most", [8, 7, 4, 2, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_smaller_clusters(hooks_lib, most, dtype):
    hooks_lib.tsv_test_set_logprobs_cluster(most)
    for T, V, top, temp, extra in ((1, 32000, 5, 1.0, 0), (2, 128256, 20, 1.0, 3), (9, 128256, 1, 1.3, 8), (30, 32001, 16, 0.75, 5), (60, 20000, 0, 1.0, 0)):
        r = np.random.default_rng(V + T)
        x = torch.from_numpy((3 * r.standard_normal((T, V + extra))).astype(np.float32)).to(dtype).cuda()[:, :V]
        tok = r.integers(0, V, T)
        for entropy in (True, False):
            logprobs.check(x, tok, logprobs.run(x, tok, temp, top, entropy), temp, top)
