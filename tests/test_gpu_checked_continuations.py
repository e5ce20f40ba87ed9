"""The operators for several continuations in the checked test build (every global access through a computed
index is compared with its buffer's extent first): small cases give the oracle's results, and no check fails."""
import numpy as np
import pytest
import torch

import continuation_util as U
import test_gpu_logprobs as logprobs
import test_gpu_pages as pages
import test_gpu_prefix_attn as prefix
import tree_speculative_decoding_03_gb300 as tsv
from oracle import continuations as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked_lib():
    tsv.build(variant="checked")
    tsv.use_variant("checked")
    yield tsv.load("checked")
    tsv.use_variant(None)


@pytest.mark.parametrize("B,bs,max_len,kw", [(3, 16, 40, {}), (40, 8, 300, dict(extra=9000)), (40, 8, 90, dict(max_blocks=2000)),
                                             (30, 128, 900, dict(free=0, extra=0))])
def test_pages(B, bs, max_len, kw):
    r = np.random.default_rng(B)
    s = U.pages_state(r, B, bs, max_len, **kw)
    src, dst = U.fork_list(r, s)
    pages.same(pages.run_fork(s, src, dst, bs), C.fork(src, dst, block_size=bs, **pages.args(s)))
    keep = pages.releases(r, s, bs)
    a = pages.args(s)
    del a["seq_lens"]
    pages.same(pages.run_release(s, keep, bs), C.release(keep, block_size=bs, **a))
    pages.same(pages.run_compact(s), C.compact(s["table"], s["held"], s["shares"], s["free_blocks"]))


def test_copy():
    pages.test_copy(torch.bfloat16, 3, 64, 128, 20, 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("i", [0, 3, 5, 6, 8, 10, 12])
def test_prefix(dtype, i):
    for cap in (0, 40000):
        c = prefix.rounded(U.prefix_case(np.random.default_rng(i), *prefix.CASES[i], cap=cap), dtype)
        d = prefix.on_device(c, dtype)
        tsv.prefix_decode_attn(**d)
        prefix.check(c, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs(dtype):
    logprobs.test_against_the_oracle(dtype, 7, 4097, 32, 1.0, 3)
    logprobs.test_rows_at_every_alignment(dtype)
