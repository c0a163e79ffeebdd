"""What the paged attention leaves behind when a device-side wait ran out of time, without one: rows
whose CTA gave up say so in LSE, whether one CTA has them or several."""
import pytest
import torch

import attention_forward_17_b200 as fa
from paged_utils import Problem


def test_arguments_are_checked():
    f = fa.lib.fa_selftest_paged_attn_abandoned
    assert f(None, 0, 0, None, 0, 0, None, 1, None, None, 0, 0, 1.0, None, 0, None, None) == fa.FA_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("news,kvs,heads", [
    ([1, 1], [200, 30], 2),                    # whole items of the row kernel
    ([1, 2], [30000, 500], 1),                 # items of the row kernel cut into parts and joined
    ([600], [3000], 1),                        # the tile kernel, cut and whole items
    ([300, 1, 1], [900, 4000, 20], 2),         # both kernels and the common join
])
def test_rows_of_an_abandoned_call_are_marked(cuda_device, fp8, news, kvs, heads):
    pr = Problem(news, kvs, heads=heads, group=4, page=64, fp8=fp8, seed=70, pad_rows=1)
    q = pr.q.cuda()
    _, lse = fa.selftest_paged_attention_abandoned(q, pr.cache, pr.batch)
    torch.cuda.synchronize()
    assert torch.isnan(lse[:-1]).all()
    # the next call is as ever
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fa.paged_attention(q, pr.cache, pr.batch, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    pr.check(got, what="after an abandoned call")
