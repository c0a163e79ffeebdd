"""Paged cache operators at the ends of their ranges."""
import ctypes

import pytest
import torch

import attention_forward_17_b200 as fa
from attention_forward_17_b200 import _binding as bnd
from paged_utils import Problem

HINT = pytest.mark.parametrize("hint", [1, None], ids=["rows", "tiles"])      # which kernel takes long sequences


def with_hint(pr, hint):
    return fa.KVBatch(pr.batch.cu, pr.batch.kv_len, pr.batch.table, pr.tokens, hint)


# ------------------------------------------------------------------ sizes (no GPU needed)
def test_the_largest_number_of_tokens():
    # a missing pointer is found after the sizes
    def codes(tokens):
        c = bnd._CacheStruct(None, None, None, None, 4, 1, 16, 64, 1024, 1024, 64, fa.FA_KV_BF16, None)
        b = bnd._BatchStruct(64, 128, 256, 2, tokens, 4, 4, 2)
        cr, br = ctypes.addressof(c), ctypes.addressof(b)
        return (fa.lib.fa_kv_append(cr, br, 16, 16, 64, 64, None, None), fa.lib.fa_kv_read(cr, br, 16, 16, 64, 64, None, None),
                fa.lib.fa_paged_attn(16, 64, 64, 16, 64, 64, 16, 1, cr, br, 0, 0, 1.0, 16, 0, None, None))
    assert codes(2 ** 30) == (fa.FA_ERR_NULL,) * 3
    assert codes(2 ** 30 + 1) == (fa.FA_ERR_SHAPE,) * 3
    text = open(bnd.HEADER).read()
    assert "tokens 0 .. 2^30 (" in text


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



# ------------------------------------------------------------------ rows that a query does not see
def rescale(pr, x, s, p, by):
    """Row p of sequence s times 2^by, in the cache's scales and in the 64-bit values."""
    pg, row = int(pr.table[s, p // pr.page]), p % pr.page
    pr.gpu[x + "e"][pg, :, row] += by
    assert (pr.gpu[x + "e"][pg, :, row].int() - by == pr.cpu[x][1][pg, :, row].cuda().int()).all()
    pr.dense[x][s][p] *= 2.0 ** by


def reference(pr, news, kvs):
    """The same problem with other lengths, and no GPU side."""
    c = Problem.__new__(Problem)
    c.__dict__.update(pr.__dict__)
    c.news, c.kvs = news, kvs
    c.dense = {x: [r[:t].clone() for r, t in zip(pr.dense[x], kvs)] for x in "kv"}
    return c


def compare(c, got, rows, by, window=0, sinks=0, what="", least=0.0):
    """Packed rows `rows` of got against the 64-bit form of c, where rows of V lie up to 2^by apart.

    Beside the bounds of attention(): LSE = ln 2 (m + log2 l), where m and -log2 l hold V's exponent (up to
    |by| + 16) and cancel; the logarithm is good to 2^-22 of itself and each rounds by 2^-24.  A tile's scales may
    differ by 2^8 before each key is taken by its own: weights are then f16 numbers that start at 2^0
    instead of 2^8, of steps of 2^-24 at the least, so each is off by another 2^-25 of the sum."""
    o, lse, bo, bl = c.attention(None, window, sinks)
    bl = bl + (abs(by) + 16) * (2.0 ** -22 + 2 * 2.0 ** -24)
    bo += least
    for s, t in enumerate(c.kvs):
        r0, r1 = int(c.cu[s]), int(c.cu[s + 1])
        bo[r0:r1] += t * 2.0 ** -25 * max(c.dense["v"][s].abs().max().item(), 0.0)
    go, gl = got[0].double().cpu()[rows], got[1].double().cpu()[rows]
    assert torch.isfinite(go).all(), what
    eo, el = (go - o[rows]).abs() - bo[rows], (gl - lse[rows]).abs() - bl[rows]
    assert (eo <= 0).all(), f"{what}: O off by {eo.max().item():.3e} more than its bound, {(eo > 0).sum().item()} of {eo.numel()}"
    assert (el <= 0).all(), f"{what}: LSE off by {el.max().item():.3e} more than its bound"


@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("x", ["k", "v"])
@pytest.mark.parametrize("by", [6, 9, 12, 13, 20, 24, 32, 60])
@pytest.mark.parametrize("d", [64, 128])
def test_a_later_row_of_any_size_changes_nothing(cuda_device, hint, x, by, d):
    # a row in the middle of a tile; the rows before it must come out as if it were not there
    pr = Problem([200, 70], [200, 300], heads=2, group=2, d=d, fp8=True, page=32, seed=61)
    rescale(pr, x, 0, 100, by)
    rescale(pr, x, 1, 260, by)
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint))
    torch.cuda.synchronize()
    c = reference(pr, [200, 70], [200, 300])
    for s, p in ((0, 100), (1, 260)):
        for y in "kv":
            c.dense[y][s][p] = 0.0
    before = torch.tensor(list(range(100)) + list(range(200, 230)))
    compare(c, got, before, 0, what="rows before")
    if x == "v":
        compare(pr, got, torch.arange(270), by, what="all rows")


@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("by", [12, 24, 32, 60])
def test_a_row_before_the_window_of_any_size_changes_nothing(cuda_device, hint, by):
    pr = Problem([300], [400], heads=1, group=2, fp8=True, page=16, seed=62)
    rescale(pr, "v", 0, 120, by)
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint), window=64, sinks=5)
    torch.cuda.synchronize()
    c = reference(pr, [300], [400])
    c.dense["v"][0][120] = 0.0
    rows = torch.tensor([i for i in range(300) if not 120 <= 100 + i < 120 + 64])
    compare(c, got, rows, 0, 64, 5, what="rows that do not see it")


@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("by", [-12, -21, -30, -50])
def test_small_rows_beside_large_ones(cuda_device, hint, by):
    # the first row sees the small one alone, the second that and a large one
    pr = Problem([90], [90], heads=2, group=2, fp8=True, page=16, seed=63)
    for x in "kv":
        rescale(pr, x, 0, 0, by)
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint))
    torch.cuda.synchronize()
    compare(pr, got, torch.arange(90), by, what="all rows")
    v = pr.dense["v"][0][0].repeat_interleave(2, 0)
    # one key: O is its row of V, which bf16 holds exactly
    assert torch.equal(got[0][0].double().cpu(), v)


@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("x", ["k", "v"])
def test_rows_at_the_lowest_scale(cuda_device, hint, x):
    # they may count as zeros: 448 * 2^-63 < 2^-54 of O; of a score, nothing
    pr = Problem([140, 1], [140, 70], heads=2, group=2, fp8=True, page=16, seed=65)
    for s, p in ((0, 0), (0, 77), (0, 139), (1, 3), (1, 69)):
        pg, row = int(pr.table[s, p // 16]), p % 16
        for h in range(2):
            by = 64 - int(pr.cpu[x][1][pg, h, row])
            pr.gpu[x + "e"][pg, h, row] = 64
            pr.dense[x][s][p, h] *= 2.0 ** by
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint))
    torch.cuda.synchronize()
    compare(pr, got, torch.arange(141), 63, what="lowest scale", least=2.0 ** -54)



@pytest.mark.gpu
@HINT
@pytest.mark.parametrize("news,kvs", [([1], [70]), ([1], [20000]), ([140], [140]), ([70, 1, 1], [700, 300, 20])])
def test_large_values_beside_zeros(cuda_device, hint, news, kvs):
    # the documented ends of V's range: magnitudes just below 2^48, and rows of zeros that keep their weight
    pr = Problem(news, kvs, heads=1, group=2, fp8=True, page=64, seed=67)
    for s, t in enumerate(kvs):
        for p0 in range(0, t, 64):
            pg, n = int(pr.table[s, p0 // 64]), min(64, t - p0)
            pr.gpu["ve"][pg, :, :n] += 45
            pr.gpu["v"].view(torch.uint8)[pg, :, 1:n:2] = 0
            pr.gpu["ve"][pg, :, 1:n:2] = 64
        pr.dense["v"][s] *= 2.0 ** 45
        pr.dense["v"][s][1::2] = 0.0
        assert pr.dense["v"][s].abs().max() < 2.0 ** 48
    got = fa.paged_attention(pr.q.cuda(), pr.cache, with_hint(pr, hint))
    torch.cuda.synchronize()
    compare(pr, got, torch.arange(sum(news)), 108, what="large V")


# ------------------------------------------------------------------ rows before the first sequence
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("skip", [1, 3, 130])
def test_packed_rows_before_the_first_sequence(cuda_device, fp8, heads, skip):
    # some sequences of a larger batch: cu does not start at 0
    pr = Problem([40, 0, 1, 90], [50, 7, 1, 200], heads=heads, d=64, page=16, fp8=fp8, seed=64, garbage=0)
    T = pr.tokens + skip
    cu = pr.batch.cu + skip
    b = fa.KVBatch(cu, pr.batch.kv_len, pr.batch.table, T, 90)
    new = {x: torch.cat([torch.full((skip, heads, 64), float("nan"), dtype=torch.bfloat16), pr.new[x]]).cuda() for x in "kv"}
    other = Problem([40, 0, 1, 90], [50, 7, 1, 200], heads=heads, d=64, page=16, fp8=fp8, seed=64, garbage=0)
    fa.kv_append(other.cache, other.batch, other.new["k"].cuda(), other.new["v"].cuda())
    fa.kv_append(pr.cache, b, new["k"], new["v"])
    got = [torch.full((T, heads, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.kv_read(pr.cache, b, *got)
    q = torch.cat([torch.full((skip, 2 * heads, 64), float("nan"), dtype=torch.bfloat16), pr.q]).cuda()
    out, lse = torch.full_like(q, 5.0), torch.full((T, 2 * heads), 5.0, device="cuda")
    fa.paged_attention(q, pr.cache, b, out=out, lse=lse)
    want = fa.kv_read(other.cache, other.batch)
    o2, l2 = fa.paged_attention(pr.q.cuda(), other.cache, other.batch)
    torch.cuda.synchronize()
    for x, g, w in zip("kv", got, want):
        assert torch.equal(pr.gpu[x].view(torch.uint8), other.gpu[x].view(torch.uint8)), x
        assert (g[:skip] == 5.0).all() and torch.equal(g[skip:], w)
    assert (out[:skip] == 5.0).all() and (lse[:skip] == 5.0).all()
    assert torch.equal(out[skip:], o2) and torch.equal(lse[skip:], l2)


# ------------------------------------------------------------------ handles
@pytest.mark.gpu
def test_handles_do_not_take_other_tensors(cuda_device):
    # the kernels would go on reading the old ones
    pr = Problem([1, 3], [40, 70], fp8=True, seed=66)
    for handle, names in ((pr.cache, ("k", "v", "k_exp", "v_exp", "heads", "d", "device")),
                          (pr.batch, ("cu", "kv_len", "table", "tokens", "device"))):
        for name in names:
            with pytest.raises(AttributeError, match=name):
                setattr(handle, name, getattr(handle, name))
        with pytest.raises(AttributeError):
            handle.other = 1
    pr.batch.kv_len.copy_(torch.tensor([30, 60]))       # written in place: read by the next call
    pr.dense = {x: [r[:t] for r, t in zip(pr.dense[x], (30, 60))] for x in "kv"}
    pr.kvs = [30, 60]
    pr.check(pr.run(), what="other lengths")
