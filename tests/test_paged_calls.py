"""Calls of the paged cache operators that their documentation allows: strided packed tensors, nothing to
do, nonsense in the lengths, a first call under capture, a server's loop."""
import math
import os
import subprocess
import sys

import pytest
import torch

import attention_forward_17_b200 as fa
from paged_utils import Problem

FP8 = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@FP8
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["slices of one projection", "heads first"])
def test_append_and_read_of_strided_tensors(cuda_device, fp8, heads, d, form):
    lens = dict(news=[33, 1, 7], kvs=[40, 9, 7], heads=heads, d=d, fp8=fp8, garbage=0, seed=80, pad_rows=2)
    a, b = Problem(**lens), Problem(**lens)
    T = a.tokens
    fa.kv_append(a.cache, a.batch, a.new["k"].cuda(), a.new["v"].cuda())

    def wide(fill):
        if form == "heads first":
            w = torch.full((2, heads, T, d + 8), fill, dtype=torch.bfloat16, device="cuda")
            return w, [w[i, :, :, :d].transpose(0, 1) for i in range(2)]
        w = torch.full((T, 2 * heads + 3, d), fill, dtype=torch.bfloat16, device="cuda")
        return w, [w[:, i * heads + 1:(i + 1) * heads + 1] for i in range(2)]
    w, (k, v) = wide(float("nan"))
    k.copy_(a.new["k"])
    v.copy_(a.new["v"])
    fa.kv_append(b.cache, b.batch, k, v)
    w, (k, v) = wide(3.0)
    fa.kv_read(b.cache, b.batch, k, v)
    want = fa.kv_read(a.cache, a.batch)
    torch.cuda.synchronize()
    for x in ("k", "v", "ke", "ve"):
        if a.gpu[x] is not None:
            assert same_bits(a.gpu[x], b.gpu[x]), x
    n = T - 2
    assert torch.equal(k[:n], want[0][:n]) and torch.equal(v[:n], want[1][:n])
    k[:n], v[:n] = 3.0, 3.0
    assert (w == 3.0).all()                                  # padding rows and all that lies between


def guarded(shape, dtype, fill, pad=4096):
    """A tensor inside a larger buffer of `fill`, and a check that the rest still is."""
    n = math.prod(shape)
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")

    def intact():
        return bool((buf[:pad] == fill).all() and (buf[n + pad:] == fill).all())
    return buf[pad:pad + n].view(shape), intact


@FP8
@pytest.mark.parametrize("hint", [1, 40, 400], ids=["rows", "both", "tiles"])
@pytest.mark.parametrize("cu,kv", [
    ([0, 9, 3, 5], [30, 30, 30]), ([-5, 2, 400, 401], [30, 30, 30]), ([0, 2, 4, 150], [2 ** 31 - 1, -7, 300]),
    ([4, 4, 0, 150], [5, 5, 2 ** 31 - 1]), ([149, 149, 149, 149], [1, 2, 3]), ([0, -1, -1, -2 ** 31], [9, 9, 9]),
    ([0, 100, 150, 150], [-(2 ** 31), 50, 0]),
])
def test_nonsense_lengths_write_nothing_outside(cuda_device, fp8, hint, cu, kv):
    pr = Problem([60, 30, 60], [60, 300, 90], heads=2, group=2, d=64, page=16, fp8=fp8, garbage=0, seed=81)
    T = pr.tokens
    b = fa.KVBatch(torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(kv, dtype=torch.int32, device="cuda"),
                   pr.batch.table, T, hint)
    out, out_ok = guarded((T, 4, 64), torch.bfloat16, 7.0)
    lse, lse_ok = guarded((T, 4), torch.float32, 7.0)
    ws, ws_ok = guarded((fa.paged_attention_workspace(pr.cache, b, 4),), torch.uint8, 7)
    k, k_ok = guarded((T, 2, 64), torch.bfloat16, 7.0)
    v, v_ok = guarded((T, 2, 64), torch.bfloat16, 7.0)
    out.fill_(9.0), lse.fill_(9.0), k.fill_(9.0), v.fill_(9.0)
    cache = [t.clone() for t in pr.gpu.values() if t is not None]
    fa.paged_attention(pr.q.cuda(), pr.cache, b, out=out, lse=lse, workspace=ws)
    fa.kv_read(pr.cache, b, k, v)
    torch.cuda.synchronize()
    assert out_ok() and lse_ok() and ws_ok() and k_ok() and v_ok()
    assert all(same_bits(a, t) for a, t in zip(cache, [t for t in pr.gpu.values() if t is not None]))
    # rows that belong to no sequence stay (offsets clamped to the rows there are)
    c = [min(max(x, 0), T) for x in cu]
    mine = torch.zeros(T, dtype=torch.bool)
    for s in range(3):
        mine[c[s]:c[s + 1]] = True
    assert (out.cpu()[~mine] == 9.0).all() and (lse.cpu()[~mine] == 9.0).all()


@FP8
def test_nothing_to_do(cuda_device, fp8):
    pr = Problem([2], [20], fp8=fp8, seed=82)
    i32 = dict(dtype=torch.int32, device="cuda")
    for seqs, tokens in ((0, 0), (0, 3), (2, 0)):
        b = fa.KVBatch(torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32), torch.zeros(seqs, 4, **i32), tokens)
        k = torch.full((tokens, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        q = torch.full((tokens, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        out, lse = q.clone(), torch.full((tokens, 4), 3.0, device="cuda")
        fa.kv_append(pr.cache, b, k, k)
        fa.kv_read(pr.cache, b, k, k.clone())
        assert fa.paged_attention_workspace(pr.cache, b, 4) == 0
        fa.paged_attention(q, pr.cache, b, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (k == 3.0).all() and (out == 3.0).all() and (lse == 3.0).all()
    # an empty page table holds no position: rows without a key, and without a place
    b = fa.KVBatch(torch.tensor([0, 2], **i32), torch.tensor([0], **i32), torch.zeros(1, 0, **i32), 2, 2)
    o, lse = fa.paged_attention(pr.q.cuda(), pr.cache, b)
    k, v = fa.kv_read(pr.cache, b)
    torch.cuda.synchronize()
    assert (o == 0).all() and torch.isneginf(lse).all() and (k == 0).all() and (v == 0).all()


def test_first_call_of_a_process_is_captured(cuda_device):
    code = """
import torch
from paged_utils import Problem
import attention_forward_17_b200 as fa
for news in ([1, 1], [90, 1]):
    pr = Problem(news, [300, 40], heads=2, group=4, page=16, seed=83)
    q, k, v = pr.q.cuda(), pr.new["k"].cuda(), pr.new["v"].cuda()
    for s, n in enumerate(news):
        for x, t in (("k", k), ("v", v)):
            pr.dense[x][s][pr.kvs[s] - n:] = t[int(pr.cu[s]):int(pr.cu[s + 1])].double().cpu()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fa.kv_append(pr.cache, pr.batch, k, v)
        got = fa.paged_attention(q, pr.cache, pr.batch)
        kr, vr = fa.kv_read(pr.cache, pr.batch)
    g.replay()
    torch.cuda.synchronize()
    pr.check(got, what="captured")
    assert torch.equal(kr, k) and torch.equal(vr, v)
print("captured")
"""
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@FP8
@pytest.mark.parametrize("d", [64, 128])
def test_a_servers_loop_to_its_bound(cuda_device, fp8, d):
    # two prompts in chunks beside single tokens, each step appended and attended to, against the 64-bit form of
    # every step with its own elementwise bound
    H, G, page = 2, 4, 16
    end = [150, 90]
    whole = Problem([0, 0], end, heads=H, group=G, d=d, page=page, fp8=fp8, seed=84, garbage=0)
    dense = {x: [r.clone() for r in whole.dense[x]] for x in "kv"}
    g = torch.Generator().manual_seed(85)
    new = {x: [torch.randn(t, H, d, generator=g).bfloat16() for t in end] for x in "kv"}
    at = [0, 0]
    for step in ([70, 0], [1, 64], [60, 1], [1, 1], [18, 24]):
        n0, n1 = step
        kvs = [at[0] + n0, at[1] + n1]
        T = n0 + n1
        cu = torch.tensor([0, n0, T], dtype=torch.int32)
        b = fa.KVBatch(cu.cuda(), torch.tensor(kvs, dtype=torch.int32, device="cuda"), whole.batch.table, T, max(step))
        rows = {x: torch.cat([new[x][s][at[s]:kvs[s]] for s in range(2)]) for x in "kv"}
        fa.kv_append(whole.cache, b, rows["k"].cuda(), rows["v"].cuda())
        back = dict(zip("kv", fa.kv_read(whole.cache, b)))
        q = torch.randn(T, H * G, d, generator=g).bfloat16()
        got = fa.paged_attention(q.cuda(), whole.cache, b)
        torch.cuda.synchronize()
        for x in "kv":
            held = back[x].double().cpu()
            if fp8:                                          # 4 significant bits: half a step is 2^-4 of the value, or
                scale = rows[x].double().abs().amax(-1, keepdim=True) / 448 * 2           # 2^-10 of at most this scale
                assert ((held - rows[x].double()).abs() <= 2.0 ** -4 * rows[x].double().abs() + 2.0 ** -10 * scale).all()
            else:
                assert torch.equal(back[x].cpu(), rows[x])
            for s in range(2):
                dense[x][s][at[s]:kvs[s]] = held[int(cu[s]):int(cu[s + 1])]
        c = Problem.__new__(Problem)
        c.__dict__.update(whole.__dict__)
        c.news, c.kvs, c.cu, c.tokens, c.q = step, kvs, cu, T, q
        c.dense = {x: [dense[x][s][:kvs[s]] for s in range(2)] for x in "kv"}
        c.check(got, what=f"step {step} at {at}")
        at = kvs
