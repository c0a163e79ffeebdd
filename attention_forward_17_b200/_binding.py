"""ctypes binding of libfa_b200.so (include/fa.h).

Argument marshalling only: every step of the attention forward pass (and of
the row softmax, GEMM, vector-add and paged cache entry points) runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or the device is not
sm_100, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "fa.h")
LIB_PATH = os.path.join(HERE, "libfa_b200.so")

FA_OK = 0
FA_ERR_NULL = -1
FA_ERR_SHAPE = -2
FA_ERR_HEADDIM = -3
FA_ERR_ALIGN = -4
FA_ERR_SCALE = -5
FA_ERR_CUDA = -6
FA_ERR_TIMEOUT = -7
FA_ERR_ARCH = -8
FA_ERR_ARG = -9
FA_ERR_PAGE = -10

FA_GEMM_PLAIN, FA_GEMM_BIAS, FA_GEMM_BIAS_GELU = 0, 1, 2
FA_KV_BF16, FA_KV_E4M3 = 0, 1
FA_KV_PREPARED_BYTES = 1024

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_exp", _vp), ("v_exp", _vp), ("pages", _i64), ("heads", _i64),
                ("page_size", _i64), ("d", _i64), ("page_stride", _i64), ("head_stride", _i64),
                ("row_stride", _i64), ("type", _i64), ("prepared", _vp)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("cu", _vp), ("kv_len", _vp), ("table", _vp), ("seqs", _i64), ("tokens", _i64),
                ("table_width", _i64), ("table_stride", _i64), ("max_new", _i64)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str = "fa_fwd"):
        self.status = status
        super().__init__(f"{where} failed with status {status}: {strerror(status)}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python attention_forward_17_b200/build.py` "
            "(there is no non-CUDA fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int,
                           ctypes.c_float, _vp]
    lib.fa_fwd.restype = ctypes.c_int
    lib.fa_fwd_status.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int,
                                  ctypes.c_float, _vp, _vp]
    lib.fa_fwd_status.restype = ctypes.c_int
    lib.fa_fwd_host.argtypes = [_vp] * 10 + [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_float,
                                            _vp]
    lib.fa_fwd_host.restype = ctypes.c_int
    lib.fa_selftest_wait_timeout.argtypes = [_vp, _i64, ctypes.c_int, _vp]
    lib.fa_selftest_wait_timeout.restype = ctypes.c_int
    lib.fa_row_softmax.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_float, _vp]
    lib.fa_row_softmax.restype = ctypes.c_int
    lib.fa_row_softmax_launches.argtypes = [_i64, _i64]
    lib.fa_row_softmax_launches.restype = ctypes.c_int
    lib.fa_fwd_schedule.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int,
                                    ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp, _vp]
    lib.fa_fwd_schedule.restype = ctypes.c_int
    lib.fa_fwd_rescale_stats.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                         ctypes.c_int, ctypes.c_float, ctypes.c_int, _vp, _vp]
    lib.fa_fwd_rescale_stats.restype = ctypes.c_int
    lib.fa_schedule_count.argtypes = []
    lib.fa_schedule_count.restype = ctypes.c_int
    lib.fa_schedule_info.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.fa_schedule_info.restype = ctypes.c_int
    lib.fa_fwd_pick_schedule.argtypes = [_i64, _i64, ctypes.c_int, _vp, _vp]
    lib.fa_fwd_pick_schedule.restype = ctypes.c_int
    lib.fa_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp, _vp]
    lib.fa_gemm.restype = ctypes.c_int
    lib.fa_gemm_launches.argtypes = [_i64, _i64, _i64]
    lib.fa_gemm_launches.restype = ctypes.c_int
    lib.fa_vector_add.argtypes = [_vp, _vp, _vp, _i64, _vp]
    lib.fa_vector_add.restype = ctypes.c_int
    lib.fa_vector_add_launches.argtypes = [_i64]
    lib.fa_vector_add_launches.restype = ctypes.c_int
    lib.fa_kv_prepare.argtypes = [_vp, _vp]
    lib.fa_kv_prepare.restype = ctypes.c_int
    lib.fa_kv_append.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp]
    lib.fa_kv_append.restype = ctypes.c_int
    lib.fa_kv_read.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp]
    lib.fa_kv_read.restype = ctypes.c_int
    lib.fa_paged_attn.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64,
                                  ctypes.c_float, _vp, _i64, _vp, _vp]
    lib.fa_paged_attn.restype = ctypes.c_int
    lib.fa_selftest_paged_attn_abandoned.argtypes = lib.fa_paged_attn.argtypes
    lib.fa_selftest_paged_attn_abandoned.restype = ctypes.c_int
    lib.fa_paged_attn_workspace.argtypes = [_vp, _vp, _i64]
    lib.fa_paged_attn_workspace.restype = _i64
    lib.fa_fwd_launches.argtypes = [_i64, _i64, _i64, _i64]
    lib.fa_fwd_launches.restype = ctypes.c_int
    lib.fa_strerror.argtypes = [ctypes.c_int]
    lib.fa_strerror.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = ctypes.c_int
    return lib


lib = _load()


def header_functions() -> list[str]:
    """Names of the functions include/fa.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(fa_\w+)\s*\(", text, flags=re.M)


def strerror(status: int) -> str:
    return lib.fa_strerror(int(status)).decode()


def version() -> tuple[int, int]:
    v = lib.fa_version()
    return v >> 16, v & 0xFFFF


def launches_per_call(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_fwd_launches(B, H, N, d))


def _check_qkv(q, k, v):
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, H, N, d], got shape {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.shape == k.shape == v.shape):
        raise ValueError(f"q, k, v shapes differ: {tuple(q.shape)} {tuple(k.shape)} {tuple(v.shape)}")
    if not (q.device == k.device == v.device) or q.device.type != "cuda":
        raise ValueError("q, k, v must be on the same CUDA device")


def schedules() -> list[dict]:
    """Every compiled schedule of the attention kernel: id, d, emu_every, kv_slots,
    persistent, algorithm, smem_bytes, key_tile."""
    out = []
    for i in range(lib.fa_schedule_count()):
        vals = [ctypes.c_int() for _ in range(7)]
        rc = lib.fa_schedule_info(i, *[ctypes.byref(x) for x in vals])
        if rc != FA_OK:
            raise FaError(rc, "fa_schedule_info")
        out.append(dict(id=i, d=vals[0].value, emu_every=vals[1].value, kv_slots=vals[2].value,
                        persistent=vals[3].value, algorithm=vals[4].value,
                        smem_bytes=vals[5].value, key_tile=vals[6].value))
    return out


def pick_schedule(N: int, d: int, causal: bool) -> tuple[int, int]:
    """(schedule id, causal group) that fa_fwd uses for this problem."""
    sid, grp = ctypes.c_int(), ctypes.c_int()
    rc = lib.fa_fwd_pick_schedule(N, d, int(bool(causal)), ctypes.byref(sid), ctypes.byref(grp))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_pick_schedule")
    return sid.value, grp.value


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
           stream=None, status=None, schedule: int | None = None, causal_group: int | None = None):
    """O, LSE = attention forward of bf16 [B, H, N, d] CUDA tensors.

    ``out`` (bf16 [B,H,N,d]) and ``lse`` (fp32 [B,H,N]) are allocated when not
    given.  Runs on ``stream`` (a torch.cuda.Stream) or the current stream.
    ``status`` may be an int32 CUDA tensor with one element; it then receives
    FA_ERR_TIMEOUT should a device-side wait run out of time.  ``schedule``
    (an id from ``schedules()``) and ``causal_group`` override the table's
    choice.
    """
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like q")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    s = (stream if stream is not None else torch.cuda.current_stream(q.device)).cuda_stream
    with torch.cuda.device(q.device):
        if schedule is not None or causal_group is not None:
            rc = lib.fa_fwd_schedule(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                     -1 if schedule is None else int(schedule),
                                     0 if causal_group is None else int(causal_group),
                                     status.data_ptr() if status is not None else None, s)
        elif status is None:
            rc = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr(), B, H, N, d, int(bool(causal)), float(scale), s)
        else:
            rc = lib.fa_fwd_status(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                   lse.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                   status.data_ptr(), s)
    if rc != FA_OK:
        raise FaError(rc)
    return out, lse


def rescale_stats(q, k, v, causal: bool = False, scale: float | None = None,
                  schedule: int | None = None):
    """Runs the forward pass once with the rescale counters on; returns
    (O, LSE, warp_steps_rescaled, row_steps_rescaled, warp_steps_total): how many
    (warp, key tile) steps and (row, key tile) steps rescaled the output
    accumulator, and the number of (warp, key tile) steps the two-query-tile
    kernel executed.  Only that kernel counts (other schedules report zeros)."""
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    counts = torch.zeros(2, dtype=torch.int64, device=q.device)
    s = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        rc = lib.fa_fwd_rescale_stats(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                      lse.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                      -1 if schedule is None else int(schedule),
                                      counts.data_ptr(), s)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_rescale_stats")
    torch.cuda.synchronize(q.device)
    # (warp, key tile) steps of the two-query-tile kernel: 4 warps per query tile,
    # key tiles up to the diagonal under the mask
    nq, nk = (N + 127) // 128, (N + 127) // 128
    steps = sum(min(nk, t + 1) if causal else nk for t in range(nq))
    return out, lse, int(counts[0].item()), int(counts[1].item()), 4 * B * H * steps


def fa_fwd_host(q_h, k_h, v_h, o_h, lse_h, q_d, k_d, v_d, o_d, lse_d, causal: bool = False,
                scale: float | None = None, stream=None):
    """Host-to-host attention forward through caller-provided device buffers.

    All arguments are torch tensors: the ``*_h`` ones on the CPU (pinned for
    asynchronous copies), the ``*_d`` ones on the GPU.  Enqueues H2D copies,
    the kernel and D2H copies on ``stream`` and returns without waiting.
    """
    import torch
    _check_qkv(q_d, k_d, v_d)
    B, H, N, d = q_d.shape
    for t in (q_h, k_h, v_h, o_h):
        if t.shape != q_d.shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("host q/k/v/o must be contiguous bf16 tensors shaped like q_d")
    if tuple(lse_h.shape) != (B, H, N) or lse_h.dtype != torch.float32:
        raise ValueError("lse_h must be fp32 [B, H, N]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    s = (stream if stream is not None else torch.cuda.current_stream(q_d.device)).cuda_stream
    with torch.cuda.device(q_d.device):
        rc = lib.fa_fwd_host(q_h.data_ptr(), k_h.data_ptr(), v_h.data_ptr(), o_h.data_ptr(),
                             lse_h.data_ptr(), q_d.data_ptr(), k_d.data_ptr(), v_d.data_ptr(),
                             o_d.data_ptr(), lse_d.data_ptr(), B, H, N, d, int(bool(causal)),
                             float(scale), s)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_host")


def selftest_wait_timeout(status, limit_us: int, arrive: bool = False, stream=None):
    """Run the bounded-wait self-test kernel; `status` is an int32 CUDA tensor (one element)."""
    import torch
    s = (stream if stream is not None else torch.cuda.current_stream(status.device)).cuda_stream
    with torch.cuda.device(status.device):
        rc = lib.fa_selftest_wait_timeout(status.data_ptr(), int(limit_us), int(bool(arrive)), s)
    if rc != FA_OK:
        raise FaError(rc, "fa_selftest_wait_timeout")


def row_softmax(x, scale: float = 1.0, out=None, stream=None):
    """y = softmax(scale * x) over the last dimension of a contiguous bf16 CUDA tensor."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.device.type != "cuda":
        raise TypeError("x must be a bfloat16 CUDA tensor")
    if not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be contiguous with at least one dimension")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if out is None:
        out = torch.empty_like(x)
    if out.shape != x.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like x")
    s = (stream if stream is not None else torch.cuda.current_stream(x.device)).cuda_stream
    with torch.cuda.device(x.device):
        rc = lib.fa_row_softmax(x.data_ptr(), out.data_ptr(), rows, cols, float(scale), s)
    if rc != FA_OK:
        raise FaError(rc, "fa_row_softmax")
    return out


def gemm(a, b, bias=None, epilogue: int = FA_GEMM_BIAS_GELU, out=None, stream=None, status=None):
    """C = epilogue(A @ B) for contiguous bf16 CUDA tensors A [M, K], B [K, N], bias [N].

    ``epilogue`` is FA_GEMM_PLAIN, FA_GEMM_BIAS or FA_GEMM_BIAS_GELU (exact erf
    GELU).  ``out`` (bf16 [M, N]) is allocated when not given.  ``status`` may
    be an int32 CUDA tensor with one element (receives FA_ERR_TIMEOUT).
    """
    import torch
    for name, t in (("a", a), ("b", b)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device.type != "cuda":
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D tensor")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(a.shape)} @ {tuple(b.shape)}")
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (N,)
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous bf16 [N] tensor")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [M, N] tensor")
    s = (stream if stream is not None else torch.cuda.current_stream(a.device)).cuda_stream
    with torch.cuda.device(a.device):
        rc = lib.fa_gemm(a.data_ptr() if K else None, b.data_ptr() if K else None,
                         bias.data_ptr() if bias is not None else None, out.data_ptr(), M, N, K,
                         int(epilogue), status.data_ptr() if status is not None else None, s)
    if rc != FA_OK:
        raise FaError(rc, "fa_gemm")
    return out


def vector_add(x, y, out=None, stream=None):
    """z = x + y for contiguous fp32 CUDA tensors of equal shape."""
    import torch
    for name, t in (("x", x), ("y", y)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device.type != "cuda":
            raise TypeError(f"{name} must be a float32 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if x.shape != y.shape:
        raise ValueError("x and y shapes differ")
    if out is None:
        out = torch.empty_like(x)
    if out.shape != x.shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 tensor shaped like x")
    s = (stream if stream is not None else torch.cuda.current_stream(x.device)).cuda_stream
    with torch.cuda.device(x.device):
        rc = lib.fa_vector_add(x.data_ptr(), y.data_ptr(), out.data_ptr(), x.numel(), s)
    if rc != FA_OK:
        raise FaError(rc, "fa_vector_add")
    return out


_torch = None


def _need_torch():
    """torch, imported once: an import statement in each of a call's functions costs as much as its checks."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _fixed(name):
    """A read-only attribute: handles hold addresses, so a tensor set later would not be the one in use."""
    return property(operator.attrgetter("_" + name))


class KVCache:
    """The paged keys and values of one layer (a handle; the tensors stay the caller's, and are the same for its life).

    ``k`` and ``v`` are CUDA tensors [pages, heads, page_size, d] of equal shape and strides, bf16 or
    float8_e4m3fn, unit stride along d, any order of the other dimensions (pass
    ``x.transpose(1, 2)`` of a [pages, page_size, heads, d] tensor).  An e4m3 cache also needs
    ``k_exp`` and ``v_exp``, contiguous uint8 [pages, heads, page_size]: a row's scale is 2^(e - 127).
    page_size is 16, 32, 64, 128 or 256, d 64 or 128.
    """
    __slots__ = ("_k", "_v", "_k_exp", "_v_exp", "_device", "_heads", "_d", "_struct", "_ref", "_index", "_prepared")
    k, v, k_exp, v_exp, device, heads, d = map(_fixed, ("k", "v", "k_exp", "v_exp", "device", "heads", "d"))

    def __init__(self, k, v, k_exp=None, v_exp=None):
        torch = _need_torch()
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
                raise TypeError(f"{name} must be bfloat16 or float8_e4m3fn, got {t.dtype}")
            if t.dim() != 4:
                raise ValueError(f"{name} must be [pages, heads, page_size, d], got shape {tuple(t.shape)}")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError(f"{name} must have unit stride along d")
        if k.dtype != v.dtype or k.shape != v.shape or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must have the same type, shape, strides and device")
        fp8 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_exp", k_exp), ("v_exp", v_exp)):
            if not fp8:
                if t is not None:
                    raise ValueError(f"{name} belongs to an e4m3 cache only")
            elif (not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.shape != k.shape[:3]
                  or not t.is_contiguous() or t.device != k.device):
                raise ValueError(f"{name} must be a contiguous uint8 [pages, heads, page_size] tensor on the cache's device")
        self._k, self._v, self._k_exp, self._v_exp = k, v, k_exp, v_exp
        self._device, self._heads, self._d, self._index = k.device, k.shape[1], k.shape[3], k.device.index
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_exp.data_ptr() if fp8 else None,
                                    v_exp.data_ptr() if fp8 else None, *k.shape, *k.stride()[:3],
                                    FA_KV_E4M3 if fp8 else FA_KV_BF16, None)
        self._ref = ctypes.addressof(self._struct)
        # kept with the handle, whose tensors do not change
        self._prepared = ctypes.create_string_buffer(FA_KV_PREPARED_BYTES)
        rc = lib.fa_kv_prepare(self._ref, ctypes.addressof(self._prepared))
        if rc != FA_OK:
            raise FaError(rc, "fa_kv_prepare")
        self._struct.prepared = ctypes.addressof(self._prepared)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, d: int, dtype=None, device="cuda"):
        """A new cache of zeros (bf16 unless ``dtype`` is torch.float8_e4m3fn)."""
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        k, v = (torch.zeros(pages, heads, page_size, d, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        ke, ve = (torch.full((pages, heads, page_size), 127, dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, ke, ve)


class KVBatch:
    """The sequences of one step (a handle, used for every layer of the step; its tensors may be written, not replaced).

    ``cu`` int32 [seqs + 1]: rows cu[s] .. cu[s+1]-1 of the packed tensors are the last of the
    ``kv_len[s]`` (int32 [seqs]) tokens of sequence s; ``table`` int32 [seqs, width]: the pages of each
    sequence in order.  All contiguous (table: rows may be strided) on one CUDA device, read
    when the kernels run.  ``tokens`` is the number of rows of the packed tensors; rows before cu[0] and
    from cu[seqs] on are padding.  ``max_new`` is the largest number of new tokens of a sequence if known:
    it chooses the kernels, which round in different places; any value gives right results.
    """
    __slots__ = ("_cu", "_kv_len", "_table", "_tokens", "_device", "_struct", "_ref", "_sizes")
    cu, kv_len, table, tokens, device = map(_fixed, ("cu", "kv_len", "table", "tokens", "device"))

    def __init__(self, cu, kv_len, table, tokens: int, max_new: int | None = None):
        torch = _need_torch()
        for name, t, dim in (("cu", cu, 1), ("kv_len", kv_len, 1), ("table", table, 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device.type != "cuda":
                raise TypeError(f"{name} must be an int32 CUDA tensor")
            if t.dim() != dim:
                raise ValueError(f"{name} must have {dim} dimension(s)")
            if t.device != cu.device:
                raise ValueError("cu, kv_len and table must be on the same device")
        seqs = kv_len.shape[0]
        if cu.shape[0] != seqs + 1 or table.shape[0] != seqs:
            raise ValueError(f"cu must have {seqs + 1} entries and table {seqs} rows")
        if not cu.is_contiguous() or not kv_len.is_contiguous() or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("cu and kv_len must be contiguous, and the rows of table")
        if tokens < 0 or (max_new is not None and max_new < 0):
            raise ValueError("tokens and max_new must not be negative")
        self._cu, self._kv_len, self._table, self._tokens, self._device = cu, kv_len, table, int(tokens), cu.device
        width = table.shape[1]
        self._struct = _BatchStruct(cu.data_ptr(), kv_len.data_ptr(), table.data_ptr(), seqs, self._tokens, width,
                                    table.stride(0) if seqs > 1 else width,
                                    self._tokens if max_new is None else int(max_new))
        self._ref = ctypes.addressof(self._struct)
        self._sizes = {}            # workspace bytes by (heads_q, heads, d), sizes only


def _packed(name, t, tokens, heads, d, device):
    """(address, token stride, head stride) of a bf16 [tokens, heads, d] tensor."""
    if not isinstance(t, _torch.Tensor) or t.dtype != _torch.bfloat16 or t.device != device:
        raise TypeError(f"{name} must be a bfloat16 tensor on {device}")
    if t.shape != (tokens, heads, d):
        raise ValueError(f"{name} must be [tokens, heads, d] = {(tokens, heads, d)}, got {tuple(t.shape)}")
    ts, hs, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have unit stride along d")
    return t.data_ptr(), ts, hs


def _pair(cache, batch):
    if not isinstance(cache, KVCache) or not isinstance(batch, KVBatch):
        raise TypeError("cache must be a KVCache and batch a KVBatch")
    if batch._device != cache._device:
        raise ValueError("cache and batch must be on the same device")


def _call(index, f, *args):
    """f(*args) with device `index` current."""
    if _torch.cuda.current_device() == index:
        return f(*args)
    with _torch.cuda.device(index):
        return f(*args)


def _status_ptr(status, device):
    if status is None:
        return None
    if not isinstance(status, _torch.Tensor) or status.dtype != _torch.int32 or status.device != device or status.numel() < 1:
        raise TypeError(f"status must be an int32 tensor with one element on {device}")
    return status.data_ptr()


def _raw_stream(index):
    """Handle of the current stream of a device."""
    get = getattr(_torch._C, "_cuda_getCurrentRawStream", None)      # a tenth of the public call's time
    return get(index) if get is not None else _torch.cuda.current_stream(index).cuda_stream


def _stream(stream, index):
    return stream.cuda_stream if stream is not None else _raw_stream(index)


def _on(stream, f, *args, **kw):
    """f(*args), which allocates, with `stream` current: memory from the pool of the stream it is used on."""
    if stream is None:
        return f(*args, **kw)
    with _torch.cuda.stream(stream):
        return f(*args, **kw)


def kv_append(cache, batch, k, v, stream=None, status=None):
    """Write the new tokens' keys and values, bf16 [tokens, heads, d], into the cache's pages.

    Token and head strides are free (positive multiples of 8 elements, the same for k and v).  An e4m3 cache
    stores each row divided by the smallest power of two that brings it within +-448.  No two
    rows may have the same place.  ``status`` (int32 CUDA tensor) receives FA_ERR_PAGE if a row's
    page lies outside the cache (that row is not written).  As in the other calls, tensors used on a ``stream``
    that is not their own have to live until it is done with them (``Tensor.record_stream``).
    """
    _pair(cache, batch)
    kp, ts, hs = _packed("k", k, batch._tokens, cache._heads, cache._d, cache._device)
    vp, ts2, hs2 = _packed("v", v, batch._tokens, cache._heads, cache._d, cache._device)
    if (ts, hs) != (ts2, hs2):
        raise ValueError("k and v must have the same strides")
    rc = _call(cache._index, lib.fa_kv_append, cache._ref, batch._ref, kp, vp, ts, hs,
               _status_ptr(status, cache._device), _stream(stream, cache._index))
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_append")


def kv_read(cache, batch, out_k=None, out_v=None, stream=None, status=None):
    """Read the batch's rows back from the cache: (k, v), bf16 [tokens, heads, d].

    ``out_k`` and ``out_v`` (equal strides) are allocated when not given; padding rows are left
    as they are.  To read sequences whole pass a batch with n_s = kv_len[s].
    """
    _pair(cache, batch)
    if (out_k is None) != (out_v is None):
        raise ValueError("give both out_k and out_v or neither")
    if out_k is None:
        out_k = _on(stream, _torch.empty, batch._tokens, cache._heads, cache._d, dtype=_torch.bfloat16, device=cache._device)
        out_v = _on(stream, _torch.empty_like, out_k)
    kp, ts, hs = _packed("out_k", out_k, batch._tokens, cache._heads, cache._d, cache._device)
    vp, ts2, hs2 = _packed("out_v", out_v, batch._tokens, cache._heads, cache._d, cache._device)
    if (ts, hs) != (ts2, hs2):
        raise ValueError("out_k and out_v must have the same strides")
    rc = _call(cache._index, lib.fa_kv_read, cache._ref, batch._ref, kp, vp, ts, hs,
               _status_ptr(status, cache._device), _stream(stream, cache._index))
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_read")
    return out_k, out_v


def paged_attention_workspace(cache, batch, heads_q: int) -> int:
    """Bytes of workspace paged_attention needs for this cache and batch."""
    _pair(cache, batch)
    key = (heads_q, cache._heads, cache._d)
    n = batch._sizes.get(key)
    if n is None:
        n = _call(cache._index, lib.fa_paged_attn_workspace, cache._ref, batch._ref, heads_q)
        if n < 0:
            raise FaError(n, "fa_paged_attn_workspace")
        batch._sizes[key] = n
    return n


def paged_attention(q, cache, batch, scale: float | None = None, window: int = 0, sinks: int = 0, out=None,
                    lse=None, workspace=None, stream=None, status=None):
    """O, LSE = attention of the new tokens q, bf16 [tokens, heads_q, d], over the cached ones.

    heads_q is a multiple of the cache's heads; query head h reads key head h // (heads_q / heads).
    The row at position p sees keys j <= p, under a ``window`` > 0 only those with p - j < window
    or j < ``sinks``; the new tokens' own keys are expected in the cache (``kv_append``).  ``out``
    (bf16 of q's shape, own strides, no memory of q's), ``lse`` (fp32 [tokens, heads_q]) and ``workspace`` (uint8,
    paged_attention_workspace() elements; one for each call that may run at the same time) are
    allocated when not given, on the stream the call runs on.  Rows that see no key get 0 and
    -inf; padding rows are left as they are.  ``status`` (int32 CUDA tensor) receives FA_ERR_PAGE
    or FA_ERR_TIMEOUT.
    """
    _pair(cache, batch)
    if not isinstance(q, _torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [tokens, heads_q, d] tensor")
    heads_q, device = q.shape[1], cache._device
    qp, qts, qhs = _packed("q", q, batch._tokens, heads_q, cache._d, device)
    if scale is None:
        scale = 1.0 / math.sqrt(cache._d)
    bytes_ = paged_attention_workspace(cache, batch, heads_q)
    if out is None:
        out = _on(stream, _torch.empty_like, q)
    if lse is None:
        lse = _on(stream, _torch.empty, batch._tokens, heads_q, dtype=_torch.float32, device=device)
    if workspace is None:
        workspace = _on(stream, _torch.empty, bytes_, dtype=_torch.uint8, device=device)
    op, ots, ohs = _packed("out", out, batch._tokens, heads_q, cache._d, device)
    if lse.dtype != _torch.float32 or lse.shape != (batch._tokens, heads_q) or not lse.is_contiguous() or lse.device != device:
        raise ValueError("lse must be a contiguous fp32 [tokens, heads_q] tensor on the cache's device")
    if workspace.dtype != _torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    rc = _call(cache._index, lib.fa_paged_attn, qp, qts, qhs, op, ots, ohs, lse.data_ptr(), heads_q, cache._ref,
               batch._ref, int(window), int(sinks), float(scale), workspace.data_ptr(), workspace.numel(),
               _status_ptr(status, device), _stream(stream, cache._index))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_attn")
    return out, lse


def selftest_paged_attention_abandoned(q, cache, batch, window: int = 0, sinks: int = 0):
    """paged_attention as it goes on when a device-side wait has run out of time: LSE is NaN."""
    _pair(cache, batch)
    heads_q, device = q.shape[1], cache._device
    qp, qts, qhs = _packed("q", q, batch._tokens, heads_q, cache._d, device)
    out = _torch.empty_like(q)
    lse = _torch.empty(batch._tokens, heads_q, dtype=_torch.float32, device=device)
    workspace = _torch.empty(paged_attention_workspace(cache, batch, heads_q), dtype=_torch.uint8, device=device)
    op, ots, ohs = _packed("out", out, batch._tokens, heads_q, cache._d, device)
    rc = _call(cache._index, lib.fa_selftest_paged_attn_abandoned, qp, qts, qhs, op, ots, ohs, lse.data_ptr(), heads_q,
               cache._ref, batch._ref, int(window), int(sinks), 1.0 / math.sqrt(cache._d), workspace.data_ptr(),
               workspace.numel(), None, _raw_stream(cache._index))
    if rc != FA_OK:
        raise FaError(rc, "fa_selftest_paged_attn_abandoned")
    return out, lse
