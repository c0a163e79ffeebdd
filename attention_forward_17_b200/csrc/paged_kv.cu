// Paged key/value cache: writing new tokens (fa_kv_append) and reading rows
// back (fa_kv_read), for sm_100a.
//
// An e4m3 row is stored as x / 2^b with the power of two 2^b in one byte (its
// exponent field).  2^b is the smallest with max |x| <= 448 * 2^b: with
// max |x| = f 2^E, f in [1, 2), that is b = E - 8 when f <= 1.75 (448 = 1.75 2^8)
// and E - 7 otherwise, read off the bf16 exponent and fraction bits.  Scaling by
// it is exact in fp32, so the one rounding is the conversion to e4m3.  The byte is
// kept within 64 .. 253: rows below 2^-54 (zeros among them) take 2^-63, so that the
// reciprocals of the scales can be summed by the attention without overflow.
//
// Both kernels move bytes and compute almost nothing: they are bound by HBM for
// prompts (2 d bytes dense and d + 1 cached per row) and by latency for single
// tokens.  A lane has 8 values of a row (16 dense bytes, so that a warp's accesses
// are whole lines on both sides), d / 8 lanes a row.  A warp takes a token (2 or 4 when
// they have few heads) and moves four groups of its heads' rows of K and of V at a
// time: eight independent loads a lane, at offsets that K and V share, since
// the instructions spent on addresses are what kept simpler forms from HBM's rate.
// Appending loads the new rows before it looks the page up, so the two latencies
// overlap.  Finding a token's sequence is one load for up to 32 sequences (the
// warp searches cu 32 ways at once), and blocks take neighbouring tokens, so that most need
// no search and no look into the page table.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_common.cuh"

namespace fa {
namespace paged {
namespace {

constexpr int kThreads = 128;

struct KvParams {
    Batch b;
    uint8_t* cache[2];        // k, v
    uint8_t* exps[2];
    uint8_t* dense[2];        // bf16
    int64_t page_stride, head_stride, row_stride;      // bytes
    int64_t token_stride, dense_head_stride;           // bytes
    int heads;
    int64_t items, per_block;
    int* status;
};

// The sequence that owns packed row t (cu[s] <= t < cu[s+1]), or seqs if none:
// the number of s with cu[s+1] <= t, found by the whole warp, 32 ways a step.
__device__ __forceinline__ int find_seq(const Batch& b, int t, int lane) {
    int lo = 0, hi = b.seqs;                       // the answer lies in [lo, hi]
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;           // last entry of the stretch before `at`
        const bool below = at + step <= hi && __ldg(b.cu + at + step) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        lo += c * step;
        hi = min(hi, lo + step);
    }
    const int s = lo + lane;
    const bool below = s < hi && __ldg(b.cu + s + 1) <= t;
    return lo + __popc(__ballot_sync(0xffffffffu, below));
}

// Where packed rows live, for a warp that asks for rising t: the sequence is looked up when
// t leaves the last one, the page when the position leaves the last one.
struct Cursor {
    int end = -1, off = 0;               // rows below `end` sit at position t + off
    int at = -1, page = -1;              // the last page: its place in the table, its id
    bool padding = false;
    const int32_t* table = nullptr;

    // The page of row t, and the row within it; -1 without a place, -2 when t is padding.
    __device__ __forceinline__ int place(const Batch& b, int t, int lane, int& row, int* status) {
        if (t >= end) {
            const int s = find_seq(b, t, lane);
            padding = s >= b.seqs;
            end = 0x7fffffff;
            if (!padding) {
                const Seq q = load_seq(b, s);
                padding = t < q.row0;            // before the first sequence (or if cu decreases)
                end = padding ? q.row0 : q.row0 + max(q.n, 1);
                off = q.kv - q.n - q.row0;
                table = b.table + s * b.table_stride;
                at = -1;
            }
        }
        if (padding) return -2;
        const int p = t + off;
        if (p < 0) return -1;
        row = p & ((1 << b.page_log2) - 1);
        if (p >> b.page_log2 != at) {
            at = p >> b.page_log2;
            page = at < b.table_width ? __ldg(table + at) : -1;
            if (page < 0 || page >= b.pages) {
                if (lane == 0) report_page(status);
                page = -1;
            }
        }
        return page;
    }
};

// Largest magnitude bits (the order of magnitudes is that of their bits) of 8 bf16.
__device__ __forceinline__ uint32_t top_bits(const uint4& a) {
    constexpr uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
    return max(m & 0xffffu, m >> 16);
}
// The same of the finite ones only.
__device__ __forceinline__ uint32_t top_finite(const uint4& a) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        if (h < 0x7f80u) top = max(top, h);
    }
    return top;
}
__device__ __forceinline__ uint2 ld_global_nc_v2(const void* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two bf16 of w, times `inv`, as two e4m3.  The saturating conversion turns
// an infinity into +-448; a NaN becomes e4m3's NaN.
__device__ __forceinline__ uint32_t quantise2(uint32_t w, float inv) {
    return e4m3x2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
}

// Two e4m3 (low 16 bits of w) times 2^k as a bf16 pair, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t w, float scale) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
    float a, c;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(a), "=f"(c)
        : "r"(h));
    return pack_bf16x2(a * scale, c * scale);
}

// T tokens and 4 / T groups of heads at a time.
template <int D, bool FP8, bool APPEND, int T>
__global__ void __launch_bounds__(kThreads, APPEND ? 6 : 5) kv_kernel(const __grid_constant__ KvParams p) {
    constexpr int kLanes = D / 8;                      // lanes of one row
    constexpr int kRows = 32 / kLanes;                 // heads of one group
    constexpr int kGroups = 4 / T;
    constexpr int kItem = FP8 ? 8 : 16;                // cached bytes of a lane
    const int lane = threadIdx.x & 31;
    const int sub = lane % kLanes, in_group = lane / kLanes;
    Cursor cursor;
    // the block's items are neighbours, taken by its warps in turn
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_block;
    const int64_t stop = min(first + p.per_block, p.items);
    for (int64_t item = first + (threadIdx.x >> 5); item < stop; item += kThreads / 32) {
        const int t0 = static_cast<int>(item) * T;
        int page[T], row[T];
        bool known = false;
        for (int h0 = 0; h0 < p.heads; h0 += kRows * kGroups) {
            uint4 x[2][4];                             // k, v: dense values, or the cached bits
            int64_t off[4];
            bool on[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int h = h0 + (u % kGroups) * kRows + in_group, t = t0 + u / kGroups;
                on[u] = h < p.heads && t < p.b.tokens;
                off[u] = t * p.token_stride + h * p.dense_head_stride + sub * 16;
                if constexpr (APPEND) {
                    if (on[u]) {
                        x[0][u] = ld_global_nc_v4(p.dense[0] + off[u]);
                        x[1][u] = ld_global_nc_v4(p.dense[1] + off[u]);
                    }
                }
            }
            if (!known) {
                known = true;
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    page[i] = -2;
                    row[i] = 0;
                    if (t0 + i < p.b.tokens) page[i] = cursor.place(p.b, t0 + i, lane, row[i], p.status);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int h = h0 + (u % kGroups) * kRows + in_group, i = u / kGroups;
                const int64_t at = page[i] * p.page_stride + h * p.head_stride + row[i] * p.row_stride + sub * kItem;
                const int64_t e_at = ((static_cast<int64_t>(page[i]) * p.heads + h) << p.b.page_log2) + row[i];
                const bool has = on[u] && page[i] >= 0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if constexpr (!APPEND) {
                        x[w][u] = make_uint4(0u, 0u, 0u, 0u);
                        if (has) {
                            if constexpr (FP8) {
                                const uint2 c = ld_global_nc_v2(p.cache[w] + at);
                                x[w][u] = make_uint4(c.x, c.y, __ldg(p.exps[w] + e_at), 0u);
                            } else {
                                x[w][u] = ld_global_nc_v4(p.cache[w] + at);
                            }
                        }
                    } else if constexpr (!FP8) {
                        if (has) *reinterpret_cast<uint4*>(p.cache[w] + at) = x[w][u];
                    } else {
                        uint32_t top = has ? top_bits(x[w][u]) : 0u;
                        if (top >= 0x7f80u) top = top_finite(x[w][u]);
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        // exponent field of the scale: 2^b with b = E - 8 (+ 1 above 1.75 2^E)
                        const int field = static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 96u ? 1 : 0);
                        const int e = min(max(field, 64), 253);
                        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                        if (has) {
                            *reinterpret_cast<uint2*>(p.cache[w] + at) =
                                make_uint2(quantise2(x[w][u].x, inv) | quantise2(x[w][u].y, inv) << 16,
                                           quantise2(x[w][u].z, inv) | quantise2(x[w][u].w, inv) << 16);
                            if (sub == 0) p.exps[w][e_at] = static_cast<uint8_t>(e);
                        }
                    }
                }
            }
            if constexpr (!APPEND) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (!on[u] || page[u / kGroups] == -2) continue;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint4 c = x[w][u];
                        uint4* out = reinterpret_cast<uint4*>(p.dense[w] + off[u]);
                        if constexpr (FP8) {
                            const float s = __uint_as_float(c.z << 23);
                            *out = make_uint4(widen2(c.x, s), widen2(c.x >> 16, s), widen2(c.y, s), widen2(c.y >> 16, s));
                        } else {
                            *out = c;
                        }
                    }
                }
            }
        }
    }
}

DeviceState g_dev[kMaxDevices];

template <int D, bool FP8, bool APPEND>
void launch(const KvParams& p, int tokens, unsigned grid, cudaStream_t s) {
    if (tokens == 1)
        kv_kernel<D, FP8, APPEND, 1><<<grid, kThreads, 0, s>>>(p);
    else if (tokens == 2)
        kv_kernel<D, FP8, APPEND, 2><<<grid, kThreads, 0, s>>>(p);
    else
        kv_kernel<D, FP8, APPEND, 4><<<grid, kThreads, 0, s>>>(p);
}

template <bool APPEND>
int run(const fa_kv_cache* c, const fa_kv_batch* b, const void* k, const void* v, int64_t token_stride,
        int64_t head_stride, int* dev_status, void* stream) {
    int rc = check_sizes(c, b);
    if (rc == 1) return FA_OK;
    if (rc != FA_OK) return rc;
    if ((rc = check_pointers(c, b)) != FA_OK) return rc;
    if (!k || !v) return FA_ERR_NULL;
    if ((rc = check_alignment(c, b)) != FA_OK) return rc;
    if (!packed_ok(k, token_stride, head_stride, b->tokens, c->heads) ||
        !packed_ok(v, token_stride, head_stride, b->tokens, c->heads) || !host::aligned(dev_status, 4))
        return FA_ERR_ALIGN;
    int sms = 0;
    if ((rc = device_ready(g_dev, sms, [] { return int(FA_OK); })) != FA_OK) return rc;
    const bool fp8 = c->type == FA_KV_E4M3;
    const int64_t item = fp8 ? 1 : 2;
    KvParams p;
    p.b = device_batch(c, b);
    p.cache[0] = static_cast<uint8_t*>(c->k);
    p.cache[1] = static_cast<uint8_t*>(c->v);
    p.exps[0] = c->k_exp;
    p.exps[1] = c->v_exp;
    p.dense[0] = static_cast<uint8_t*>(const_cast<void*>(k));
    p.dense[1] = static_cast<uint8_t*>(const_cast<void*>(v));
    p.page_stride = c->page_stride * item;
    p.head_stride = c->head_stride * item;
    p.row_stride = c->row_stride * item;
    p.token_stride = token_stride * 2;
    p.dense_head_stride = head_stride * 2;
    p.heads = static_cast<int>(c->heads);
    p.status = dev_status;
    // groups of heads of a token: with one or two, a warp takes four or two tokens
    const int64_t rows = 32 / (c->d / 8), groups = (c->heads + rows - 1) / rows;
    const int tokens = groups == 1 ? 4 : groups == 2 ? 2 : 1;
    p.items = (b->tokens + tokens - 1) / tokens;
    // several times the blocks that run at once, each with at least one item for every
    // warp: longer stretches save look-ups, but a last round of few blocks costs more (appending
    // 15,667 rows of 8 heads: 24 us with as many as run, 22 with 48 a SM; reading 64,575: 77
    // with 8 a SM, 72 with 12, 70 with 20)
    const int64_t cap = static_cast<int64_t>(sms) * (APPEND ? 48 : 20), each = (p.items + cap - 1) / cap;
    p.per_block = each > kThreads / 32 ? each : kThreads / 32;
    const unsigned grid = static_cast<unsigned>((p.items + p.per_block - 1) / p.per_block);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c->d == 128)
        fp8 ? launch<128, true, APPEND>(p, tokens, grid, s) : launch<128, false, APPEND>(p, tokens, grid, s);
    else
        fp8 ? launch<64, true, APPEND>(p, tokens, grid, s) : launch<64, false, APPEND>(p, tokens, grid, s);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace paged
}  // namespace fa

extern "C" int fa_kv_append(const fa_kv_cache* cache, const fa_kv_batch* batch, const void* k, const void* v,
                            int64_t token_stride, int64_t head_stride, int* dev_status, void* stream) {
    return fa::paged::run<true>(cache, batch, k, v, token_stride, head_stride, dev_status, stream);
}

extern "C" int fa_kv_read(const fa_kv_cache* cache, const fa_kv_batch* batch, void* k, void* v,
                          int64_t token_stride, int64_t head_stride, int* dev_status, void* stream) {
    return fa::paged::run<false>(cache, batch, k, v, token_stride, head_stride, dev_status, stream);
}
