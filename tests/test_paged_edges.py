"""Paged cache operators at the ends of their ranges."""
import pytest
import torch

import attention_forward_17_b200 as fa
from paged_utils import Problem

HINT = pytest.mark.parametrize("hint", [1, None], ids=["rows", "tiles"])      # which kernel takes long sequences


def with_hint(pr, hint):
    return fa.KVBatch(pr.batch.cu, pr.batch.kv_len, pr.batch.table, pr.tokens, hint)


# ------------------------------------------------------------------ queries and keys of zeros
@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("news,kvs,window", [([1], [64], 0), ([200], [300], 0), ([60, 1, 129], [60, 9, 129], 0),
                                             ([300], [400], 50)])
def test_queries_of_zeros_over_small_keys(cuda_device, hint, news, kvs, window):
    # every score is 0: the mean of the visible rows of V, and the logarithm of their number
    pr = Problem(news, kvs, heads=2, group=2, fp8=True, seed=60)
    pr.q.zero_()
    for x, by in (("k", -40), ("v", 0)):
        pr.gpu[x + "e"] += by
        pr.dense[x] = [r * 2.0 ** by for r in pr.dense[x]]
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint), window=window, sinks=3)
    torch.cuda.synchronize()
    pr.check(got, window, 3, what="zeros")


@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,kv", [(1, 1), (1, 40), (100, 100), (300, 333)])
def test_all_zeros_through_an_e4m3_cache(cuda_device, hint, d, n, kv):
    # what a server sends to warm up; also rows of a mixed batch
    c = fa.KVCache.empty(30, 2, 16, d, torch.float8_e4m3fn)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = fa.KVBatch(torch.tensor([0, n], **i32), torch.tensor([kv], **i32), torch.randperm(30, device="cuda").int().view(1, 30),
                   n, hint)
    whole = fa.KVBatch(torch.tensor([0, kv], **i32), b.kv_len, b.table, kv, kv)
    z = torch.zeros(kv, 2, d, dtype=torch.bfloat16, device="cuda")
    fa.kv_append(c, whole, z, z)
    o, lse = fa.paged_attention(torch.zeros(n, 8, d, dtype=torch.bfloat16, device="cuda"), c, b)
    torch.cuda.synchronize()
    want = torch.log(torch.arange(kv - n + 1, kv + 1, dtype=torch.float64)).unsqueeze(1)
    assert (o == 0).all()
    # LSE = ln 2 (m + log2 l): V's rows have the scale 2^-63, so |m| and log2 l are up to 80 while
    # the sum is small; l is exact, its logarithm good to 2^-22 of itself, and each rounds by 2^-24
    assert ((lse.double().cpu() - want).abs() <= 80 * (2.0 ** -22 + 2 * 2.0 ** -24)).all()
