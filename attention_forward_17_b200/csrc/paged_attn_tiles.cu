// Paged attention for many query rows per key head (prompt chunks) on the
// tensor cores' tiles (tcgen05), for sm_100a.
//
// 4 d flops per visible (query, key) pair against 2 d bytes per key and tensor that
// hundreds of rows share: the tensor cores bound it.  The inner loop is that of
// the dense multi-tile kernel (fa_fwd_2q_kernel.cuh): two 128-row query tiles share
// every 128-key tile of K and V, one warp issues all products in a fixed
// alternating order, softmax threads own one row each, P goes back to tensor
// memory over its scores and is released in two parts, three quarters and one
// quarter of the keys.  What differs:
//   - query rows are the G heads of a key head, token by token (RT = 256 rows an
//     item), so grouped heads share K and V within the tile.  With G a power of two up to 128 a
//     tile of them is one TMA box of [128 / G tokens][G heads] per 64 columns, loaded when the last
//     segment's rows are done with; otherwise the softmax warps gather them;
//   - a CTA is persistent and works through its stretch of the work list
//     (paged_attn.cuh).  A scheduler warp writes the next segment's description to
//     shared memory while the current one runs, so the producer starts on its
//     pages before the current segment has ended;
//   - K and V come page by page: one TMA box per page (or 128 rows of it) and
//     64 columns, issued by the lanes of the producer warp in parallel;
//   - keys that no row of the item sees (past the end, before the window) may be
//     anything: their scores are replaced, and their rows of V are zeroed in shared
//     memory before the product, so that a weight of zero meets a zero.
//
// e4m3 caches: four more warps widen each tile to f16 in shared memory.  A row is
// multiplied by 2^(b - B + 6), B the largest b of the tile, which is exact while
// b >= B - 21; 2^(B - 6) then belongs to the whole tile: K's goes into the factor of the scores, V's joins
// the exponent of the weights as in the row kernel.  Q goes to f16 after a power-of-two scale per row.
// Tiles whose scales lie further apart (K: 2^21; V: 2^8, since B also lifts the running maximum of rows
// that do not see the largest row, and f16 weights have 22 bits of room below it) are widened
// without their scales, and the softmax threads take each key's own (step_by_key).  Rows at the lowest scale,
// zeros among them, may count as zeros and do not make a tile such.
//
// Measured on one B200 (device time): a 512-token chunk over 16,384 cached, 8 key heads of 4 query
// heads, d = 128, bf16: 119 to 122 us with the join, 1,110 to 1,140 TFLOP/s, 0.67 to 0.69 of the measured cuBLAS burst
// (141 us, 960 TFLOP/s, call after call through the API).  A 256 x 128 step takes about 2,850 cycles
// against 2,048 of tensor work (the softmax's chain, as in the dense kernel, 1,600 TFLOP/s if it were all);
// the rest is the start (about 7,000 cycles until the first scores), each segment's end (4,000) and the join.
// e4m3: 3,200 cycles a step, since widening shares the issue slots with the softmax.  d = 64: 2,048 rows
// over 16,384, 376 us bf16 and 368 e4m3, 685 and 700 TFLOP/s, 0.42: the 32,768 exponentials of a step, all on the
// special-function unit (16 a cycle), take 2,048 cycles against 1,024 of tensor work.
//
// Threads: warps 0-3 and 4-7 softmax of the two tiles, 8 producer, 9 issuer, 10
// tensor memory and scheduling, 11 idle, 12-15 widening (e4m3 only).
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "paged_attn.cuh"

namespace fa {
namespace paged {
namespace {

constexpr int kRT = kTileRows, kBN = 128;
constexpr int kProducer = 8, kIssuer = 9, kSched = 10, kWiden = 12;
constexpr float kTauF16 = 15.f, kTopF16 = 8.f;     // f16 weights: the maximum's lag, and where a fresh one sits (base 2)
constexpr int kSpanK = 21, kSpanV = 8;             // e4m3: scales of a tile that share a factor (base 2)

template <int D, bool FP8>
struct Cfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    static constexpr int kLaunchRegs = FP8 ? 128 : 168;
    static constexpr uint32_t kRegsSoft = FP8 ? 184 : 208;
    static constexpr uint32_t kRegsRest = FP8 ? 72 : 88;
    static_assert(256 * kRegsSoft + (kThreads - 256) * kRegsRest <= kThreads * kLaunchRegs, "register split");
    static constexpr int kBoxes = D / 64;                      // 64-column boxes of a 16-bit tile
    static constexpr int kBoxBytes = 128 * 128;
    static constexpr int kTileBytes = kBoxes * kBoxBytes;      // 128 rows of Q, K or V in 16 bits
    static constexpr int kSlots = FP8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
    static constexpr int kRawBytes = FP8 ? 128 * D : 0;        // a tile as stored
    static constexpr int kRaws = FP8 ? (D == 128 ? 3 : 4) : 0;
    static constexpr int kExpBytes = FP8 ? 2048 : 0;           // scales of K and of V: [2][8 pieces][128]
    static constexpr int kSlotOff = 2 * kTileBytes;
    static constexpr int kRawOff = kSlotOff + kSlots * kTileBytes;
    static constexpr int kExpOff = kRawOff + kRaws * kRawBytes;
    static constexpr int kBarOff = kExpOff + kRaws * kExpBytes;
    static constexpr int kSmemBytes = 1024 + kBarOff + (FP8 ? 2944 : 640);
    static_assert(kSmemBytes <= 232448 - 512, "shared memory per CTA");
    static constexpr uint32_t kColO = 256;
};

// A segment, and by tile: every row sees the keys of [none, all).
struct TileSegment : Segment {
    int all[2], none[2];
};

template <int D, bool FP8>
struct Bars {
    using C = Cfg<D, FP8>;
    uint64_t kv_full[C::kSlots], kv_empty[C::kSlots];
    uint64_t raw_full[FP8 ? C::kRaws : 1], raw_empty[FP8 ? C::kRaws : 1];
    uint64_t q_raw[2], q_free[2];        // loaded by TMA: arrived (e4m3), rows written or converted before done with
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2];
    uint64_t seg_full[2], seg_empty[2];
    TileSegment seg[2];
    uint32_t tmem_base;
    volatile uint32_t abort;
    float fac[FP8 ? 8 : 1];              // e4m3: of unit u: K's tile factor (2 (u % 4)), V's exponent (+ 1); 0: by key
    uint32_t by_key[FP8 ? 4 : 1][2][FP8 ? 32 : 1];     // scale bytes of K and V of unit u % 4, if taken by key
    int red[FP8 ? 16 : 1];               // largest exponents, and smallest << 8, by warp, two units
    float row_scale[FP8 ? 256 : 1];      // Q's power of two by row
};

// tcgen05 instruction descriptor, kind::f16, f16 (0) or bf16 (1) operands.
__host__ __device__ constexpr uint32_t idesc_of(bool f16, int N, bool b_mn) {
    return f16 ? (idesc_bf16_f32(128, N, b_mn) & ~((1u << 7) | (1u << 10))) : idesc_bf16_f32(128, N, b_mn);
}

template <int N>
__device__ __forceinline__ void store_words(uint32_t taddr, uint32_t* w) {
    static_assert(N == 48 || N == 16, "whole stores");
    auto& a = *reinterpret_cast<uint32_t(*)[16]>(w + (N == 48 ? 32 : 0));
    if constexpr (N == 48) {
        auto& b = *reinterpret_cast<uint32_t(*)[32]>(w);
        reg_fence32(b);
        reg_fence16(a);
        tmem_st32(taddr, b);
        tmem_st16(taddr + 32, a);
        tmem_wait_st();
        reg_fence32(b);
        reg_fence16(a);
    } else {
        reg_fence16(a);
        tmem_st16(taddr, a);
        tmem_wait_st();
        reg_fence16(a);
    }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// 2^x in f16, x <= 15: normal, subnormal or 0.
__device__ __forceinline__ uint32_t f16_power(int x) {
    return x >= -14 ? static_cast<uint32_t>(x + 15) << 10 : x >= -24 ? 1u << (x + 24) : 0u;
}

// e4m3 tiles whose scales lie far apart: a softmax thread's whole step, with each key's own scales, in
// short loops out of line (chunks of 4 sequences over 31,477 cached, d = 128, and 2,048 rows over 16,384, d = 64,
// where no tile comes here: 576 and 378 us without it; 606 and 426 with it inlined; 580 and 393 called from the
// step's own loop; 584 and 369 so.  1,542 us when every tile of the first comes here).  S becomes
// t_j = s_j + b_j in place.  The row sees the keys below a of the tile that are not below b, or are below z.
template <int D>
__device__ __noinline__ void step_by_key(const uint32_t* ek, const uint32_t* ev, uint32_t ts, uint32_t to, int a, int b, int z,
                                         float cl, bool rescale, uint32_t p_half, uint32_t p_full, float& m, float& l) {
    const auto seen = [&](int j) { return bits_below(a - j) & (~bits_below(b - j) | bits_below(z - j)); };
    float top = -INFINITY, sum = 0.f, alpha = 1.f;
#pragma unroll 1
    for (int j = 0; j < kBN; j += 16) {
        uint32_t t[16];
        tmem_ld32x16(ts + j, t);
        tmem_wait_ld();
        reg_fence16(t);
        const uint32_t see = seen(j);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int e = ek[(j + k) >> 2] >> (8 * (k & 3)) & 0xff, f = ev[(j + k) >> 2] >> (8 * (k & 3)) & 0xff;
            const float kf = __uint_as_float(static_cast<uint32_t>(max(e - 6, 0)) << 23);
            float v = fmaf(__uint_as_float(t[k]), cl * kf, static_cast<float>(f - 133));
            if (!(see & (1u << k))) v = -INFINITY;
            t[k] = __float_as_uint(v);
            top = fmaxf(top, v);
        }
        reg_fence16(t);
        tmem_st16(ts + j, t);
    }
    tmem_wait_st();
    if (top > m + kTauF16) {
        alpha = ex2_approx(m - (top - kTopF16));
        m = top - kTopF16;
    }
    if (rescale && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int j = 0; j < D; j += 16) {
            uint32_t o[16];
            tmem_ld32x16(to + j, o);
            tmem_wait_ld();
            reg_fence16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            reg_fence16(o);
            tmem_st16(to + j, o);
        }
    }
    const float off = m == -INFINITY ? 0.f : m;
#pragma unroll 1
    for (int j = 0; j < kBN; j += 16) {
        uint32_t t[16], w[8];
        tmem_ld32x16(ts + j, t);
        tmem_wait_ld();
        reg_fence16(t);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            const float w0 = ex2_approx(__uint_as_float(t[k]) - off), w1 = ex2_approx(__uint_as_float(t[k + 1]) - off);
            const uint32_t f = ev[(j + k) >> 2] >> (8 * (k & 3));
            // a hidden key's scale may be anything, but adds a finite 0
            sum = fmaf(w0, __uint_as_float((260 - max(f & 0xff, 6u)) << 23), sum);
            sum = fmaf(w1, __uint_as_float((260 - max(f >> 8 & 0xff, 6u)) << 23), sum);
            w[k / 2] = pack_f16x2(w0, w1);
        }
        reg_fence8(w);
        tmem_st8(ts + j / 2, w);                         // over scores that have been read
        tmem_wait_st();
        if (j == 80 || j == 112) {
            tc_fence_before();
            mbar_arrive(j == 80 ? p_half : p_full);
        }
    }
    l = fmaf(l, alpha, sum);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams p) {
    using C = Cfg<D, FP8>;
    using B = Bars<D, FP8>;
    static_assert(sizeof(B) <= C::kSmemBytes - 1024 - C::kBarOff, "barrier block");
    constexpr int kW0 = 48, kW1 = 16;                  // words (key pairs) of P's two releases
    extern __shared__ uint8_t smem_raw[];
    __shared__ Scratch scratch;
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);
    auto* bars = reinterpret_cast<B*>(smem + C::kBarOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t* abort = &bars->abort;
    const auto bar = [](const uint64_t& b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(bar(bars->kv_full[s]), FP8 ? 4 : 1);
            mbar_init(bar(bars->kv_empty[s]), 1);
        }
        for (int s = 0; s < C::kRaws; ++s) {
            mbar_init(bar(bars->raw_full[s]), 1);
            mbar_init(bar(bars->raw_empty[s]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bars->q_raw[i]), 1);
            mbar_init(bar(bars->q_free[i]), 4);
            mbar_init(bar(bars->q_full[i]), !FP8 && p.q_tma ? 1 : 128);
            mbar_init(bar(bars->s_full[i]), 1);
            mbar_init(bar(bars->p_half[i]), 128);
            mbar_init(bar(bars->p_full[i]), 128);
            mbar_init(bar(bars->o_full[i]), 1);
            mbar_init(bar(bars->seg_full[i]), 1);
            mbar_init(bar(bars->seg_empty[i]), FP8 ? 14 : 10);   // warps that read it
        }
        bars->abort = p.abandoned;
        fence_barrier_init();
    }
    if (warp == kSched) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    let_next_start();
    Start start{0, 0, 0, 0, 0, 0};
    if (!few_seqs(p)) start = locate_block<kRT, kBN>(p, blockIdx.x, &scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const int pr_log2 = min(p.b.page_log2, 7);          // rows of a page piece: 16 .. 128
    const int pr = 1 << pr_log2;

    // Segment k sits in seg[k % 2]; every reading warp waits for it and hands it back.
    const auto seg_wait = [&](uint32_t k) -> const TileSegment& {
        wait_bar(bar(bars->seg_full[k & 1]), (k >> 1) & 1, abort, p.status);
        return bars->seg[k & 1];
    };
    const auto seg_done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars->seg_empty[k & 1]));
    };
    if (warp < 8) {
        regs_increase<C::kRegsSoft>();
        // ============================================================ softmax, one row per thread
        const int ti = warp >> 2, quarter = warp & 3;
        const int r = 32 * quarter + lane;
        const uint32_t lane_w = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t t_s = tmem + lane_w + 128u * ti;
        const uint32_t t_o = tmem + lane_w + C::kColO + static_cast<uint32_t>(D) * ti;
        const uint32_t qtile = base + ti * C::kTileBytes;
        constexpr float kTau = FP8 ? kTauF16 : 32.f, kTop = FP8 ? kTopF16 : 0.f;
        uint32_t steps = 0, segs = 0;
        uint32_t done_o = 0;
        uint32_t unit_no = 0;                            // units of earlier segments (both tiles alike)
        // Q of a segment, D / 8 lanes a row
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;
        const auto load_q = [&](const TileSegment& g, uint4 (&qv)[32 / kPer]) {
            // this lane's rows are kPer apart: token and head of the group advance with them
            int x = g.r0 + 128 * ti + 32 * quarter + lane / kLanes;
            int t = x / p.group, hd = x - t * p.group;
#pragma unroll
            for (int i = 0; i < 32 / kPer; ++i) {
                qv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (x < g.r1)
                    qv[i] = ld_global_nc_v4(p.q + static_cast<int64_t>(g.row0 + t) * p.q_ts +
                                            static_cast<int64_t>(g.head * p.group + hd) * p.q_hs + 8 * (lane % kLanes));
                x += kPer;
                hd += kPer;
                while (hd >= p.group) {
                    hd -= p.group;
                    ++t;
                }
            }
        };
        for (;; ++segs) {
            const TileSegment& g = seg_wait(segs);
            const int n = g.n;
            if (n == 0) break;
            const int rows = g.r1 - g.r0 - 128 * ti;     // rows of this tile (may be <= 0)
            if (rows <= 0) {
                unit_no += n;
                seg_done(segs);
                continue;
            }
            // ---- Q in its tile (128-byte swizzle), this warp's 32 rows, D / 8 lanes a row
            const auto to_f16 = [&](int rr, uint4 v) {       // e4m3: f16 after a power of two per row
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = min(max(static_cast<int>(top >> 7), 1), 253);
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                if (lane % kLanes == 0) bars->row_scale[128 * ti + rr] = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = pack_f16x2(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xffff0000u) * inv);
                return make_uint4(w[0], w[1], w[2], w[3]);
            };
            const auto q_at = [&](int rr) {
                const int ch = lane % kLanes;
                return qtile + (ch >> 3) * C::kBoxBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
            };
            if (p.q_tma) {
                // the scheduler has it loaded; e4m3: to f16 in place
                if constexpr (FP8) {
                    wait_bar(bar(bars->q_raw[ti]), done_o & 1, abort, p.status);
#pragma unroll 2
                    for (int i = 0; i < 32; i += kPer) {
                        const int rr = 32 * quarter + i + lane / kLanes;
                        const uint4 v = to_f16(rr, ld_shared_v4(q_at(rr)));
                        st_shared_v4(q_at(rr), v.x, v.y, v.z, v.w);
                    }
                }
            } else {
                uint4 qv[32 / kPer];                     // every load in flight at once
                load_q(g, qv);
#pragma unroll
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int rr = 32 * quarter + kPer * i + lane / kLanes;
                    uint4 v = qv[i];
                    if constexpr (FP8) v = to_f16(rr, v);
                    st_shared_v4(q_at(rr), v.x, v.y, v.z, v.w);
                }
            }
            if (FP8 || !p.q_tma) {
                fence_proxy_async_smem();
                tc_fence_before();                       // the last segment's reads of O and S
                __syncwarp();
                mbar_arrive(bar(bars->q_full[ti]));
            }
            float cl = p.scale_log2;
            if constexpr (FP8) cl *= bars->row_scale[128 * ti + r];

            float m = -INFINITY, l = 0.f, lh = 0.f;
            for (int u = 0; u < n; ++u, ++steps) {
                // (the rare tile taken by key is left to the outer loop, which keeps its call out of this one)
                for (; u < n; ++u, ++steps) {
                    const int k0 = key_tile(g, u) * kBN;
                    wait_bar(bar(bars->s_full[ti]), steps & 1, abort, p.status);
                    tc_fence_after();
                    float vb = 0.f, c = cl;
                    if constexpr (FP8) {
                        const uint32_t f = (unit_no + u) & 3;
                        const float fk = bars->fac[2 * f];
                        if (__builtin_expect(fk == 0.f, 0)) break;
                        // never 0, as it would be for a row of zeros over small keys: hidden scores are -inf, and
                        // 0 times that is NaN.  |S| stays below 2^23, so at the least c every exponent is 0 to 2^-100.
                        c = fmaxf(cl * fk, 1.17549435e-38f);
                        vb = bars->fac[2 * f + 1];
                    }
                    const bool masked = k0 + kBN > g.all[ti] || (k0 < g.none[ti] && k0 + kBN > p.sinks);
                    uint32_t s[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
                    if (masked) {
                        // visible keys of this row: j < a + k0 and (j >= b + k0 or j < sinks)
                        const int x = g.r0 + 128 * ti + r, pos = g.p0 + x / p.group;
                        const int a = (x < g.r1 ? min(pos + 1, g.hi) : 0) - k0;
                        const int b = (p.window == kNoWindow ? 0 : pos - p.window + 1) - k0, z = p.sinks - k0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // bit i: key 32 q + i is visible
                            const uint32_t see = bits_below(a - 32 * q) & (~bits_below(b - 32 * q) | bits_below(z - 32 * q));
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(see & (1u << k))) s[32 * q + k] = __float_as_uint(-INFINITY);
                        }
                    }
                    float xm[8];
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        xm[ch] = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 16; k += 2)
                            xm[ch] = max3f(xm[ch], __uint_as_float(s[16 * ch + k]), __uint_as_float(s[16 * ch + k + 1]));
                    }
                    float mn = fmaxf(max3f(xm[0], xm[1], xm[2]), max3f(xm[3], xm[4], fmaxf(xm[5], max3f(xm[6], xm[7], xm[7])))) * c;
                    if constexpr (FP8) mn += vb;
                    const bool grow = mn > m + kTau;
                    float alpha = 1.f;
                    if (grow) {
                        alpha = ex2_approx(m - (mn - kTop));
                        m = mn - kTop;
                        l *= alpha;
                        lh *= alpha;
                    }
                    // this row's O holds the products of the segment's earlier tiles, all
                    // complete: S of this step was issued after them
                    if (__any_sync(0xffffffffu, grow && u > 0)) {
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t o[32];
                            tmem_ld32(t_o + 32 * q, o);
                            tmem_wait_ld();
                            reg_fence32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            reg_fence32(o);
                            tmem_st32(t_o + 32 * q, o);
                        }
                    }
                    const float off = (FP8 ? vb : 0.f) - (m == -INFINITY ? 0.f : m);
                    const uint64_t c2 = f2(c, c), off2 = f2(off, off);
                    uint64_t la0 = 0, la1 = 0;
                    float hl0 = 0.f, hh0 = 0.f, hl1 = 0.f, hh1 = 0.f;
                    uint32_t pw[kW0];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int k = 0; k < (h ? kW1 : kW0); ++k) {
                            const int sk = 2 * ((h ? kW0 : 0) + k);
                            const uint64_t xv = fma2(f2(__uint_as_float(s[sk]), __uint_as_float(s[sk + 1])), c2, off2);
                            float e0, e1;
                            f2_split(xv, e0, e1);
                            const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                            const uint32_t w = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                            if (k & 1) {
                                la1 = add2(la1, f2(p0, p1));
                                if constexpr (!FP8) add_bf16x2_halves(hl1, hh1, w);
                            } else {
                                la0 = add2(la0, f2(p0, p1));
                                if constexpr (!FP8) add_bf16x2_halves(hl0, hh0, w);
                            }
                            pw[k] = w;
                        }
                        if (h == 0)
                            store_words<kW0>(t_s, pw);
                        else
                            store_words<kW1>(t_s + kW0, pw);
                        tc_fence_before();
                        mbar_arrive(bar(h == 0 ? bars->p_half[ti] : bars->p_full[ti]));
                    }
                    float v0, v1;
                    f2_split(add2(la0, la1), v0, v1);
                    if constexpr (FP8)
                        l = fmaf(v0 + v1, __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(vb)) << 23), l);
                    else
                        l += v0 + v1;
                    lh += (hl0 + hh0) + (hl1 + hh1);
                }
                if (!FP8 || u == n) break;
                if constexpr (FP8) {
                    const uint32_t f = (unit_no + u) & 3;
                    const int k0 = key_tile(g, u) * kBN, x = g.r0 + 128 * ti + r, pos = g.p0 + x / p.group;
                    step_by_key<D>(bars->by_key[f][0], bars->by_key[f][1], t_s, t_o, (x < g.r1 ? min(pos + 1, g.hi) : 0) - k0,
                                   (p.window == kNoWindow ? 0 : pos - p.window + 1) - k0, p.sinks - k0, cl, u > 0,
                                   bar(bars->p_half[ti]), bar(bars->p_full[ti]), m, l);
                }
            }
            if constexpr (FP8) lh = l;

            // ---- the rows: whole items are finished here, parts go to their slot
            wait_bar(bar(bars->o_full[ti]), done_o & 1, abort, p.status);
            ++done_o;
            tc_fence_after();
            const int x = g.r0 + 128 * ti + r;
            const bool mine = x < g.r1;
            const int t = x / p.group;
            const int64_t token = g.row0 + t;
            const int head = g.head * p.group + (x - t * p.group);
            if (g.slot < 0) {
                const float inv = lh == 0.f ? 0.f : 1.f / lh;
                // through this warp's rows of the Q tile (its products are complete), so
                // that the stores to the packed tensor are whole rows
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld32(t_o + 32 * q, o);
                    tmem_wait_ld();
                    reg_fence32(o);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        st_shared_v4(qtile + (q >> 1) * C::kBoxBytes + r * 128 + (((4 * (q & 1) + v) ^ (r & 7)) << 4),
                                     pack_bf16x2(__uint_as_float(o[8 * v + 0]) * inv, __uint_as_float(o[8 * v + 1]) * inv),
                                     pack_bf16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv),
                                     pack_bf16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv),
                                     pack_bf16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv));
                }
                __syncwarp();
                {
                    const int ch = lane % kLanes;
                    int y = g.r0 + 128 * ti + 32 * quarter + lane / kLanes;
                    int yt = y / p.group, hd = y - yt * p.group;
#pragma unroll 4
                    for (int i = 0; i < 32; i += kPer) {
                        const int rr = 32 * quarter + i + lane / kLanes;
                        const uint4 w = ld_shared_v4(qtile + (ch >> 3) * C::kBoxBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
                        if (y < g.r1)
                            *reinterpret_cast<uint4*>(p.o + static_cast<int64_t>(g.row0 + yt) * p.o_ts +
                                                      static_cast<int64_t>(g.head * p.group + hd) * p.o_hs + 8 * ch) = w;
                        y += kPer;
                        hd += kPer;
                        while (hd >= p.group) {
                            hd -= p.group;
                            ++yt;
                        }
                    }
                }
                __syncwarp();
                if (mine) {
                    p.lse[token * p.heads_q + head] = unless_aborted(lse_of(m, l), abort);
                }
            } else {
                float* slot = slot_at<kRT, D>(p, blockIdx.x, g.slot);
                const int rr = 128 * ti + r;
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld32(t_o + 32 * q, o);
                    tmem_wait_ld();
                    reg_fence32(o);
                    if (mine) {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<uint4*>(slot + ((8 * q + v) * kRT + rr) * 4) =
                                make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    }
                }
                if (mine) {
                    slot[kRT * D + rr] = m;
                    slot[kRT * (D + 1) + rr] = unless_aborted(l, abort);
                    slot[kRT * (D + 2) + rr] = lh;
                }
            }
            unit_no += n;
            if (p.q_tma) {
                fence_proxy_async_smem();                // the rows written there, before TMA writes
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bars->q_free[ti]));
            }
            seg_done(segs);
        }
    } else if (warp == kProducer) {
        regs_decrease<C::kRegsRest>();
        // ============================================================ TMA producer
        const int pcs_log2 = 7 - pr_log2, pieces = 1 << pcs_log2;        // pieces of a tile: 1 .. 8
        const int per_batch = 32 >> pcs_log2;
        uint32_t ld = 0;                                                 // tiles loaded so far
        for (uint32_t k = 0;; ++k) {
            const TileSegment& g = seg_wait(k);
            const int n = g.n;
            if (n == 0) break;
            const int32_t* table = p.b.table + g.seq * p.b.table_stride;
            const int head = g.head;
            for (int u0 = 0; u0 < n; u0 += per_batch) {
                const int lu = u0 + (lane >> pcs_log2);
                int id = -1, row = 0;
                if (lu < n) {
                    const int at = key_tile(g, lu) * kBN + (lane & (pieces - 1)) * pr;
                    row = at & ((1 << p.b.page_log2) - 1);
                    if (at < g.hi && (at + pr > g.lo || at < g.sk)) {
                        id = __ldg(table + (at >> p.b.page_log2));
                        if (id < 0 || id >= p.b.pages) {
                            report_page(p.status);
                            id = -1;                                     // reads as zeros
                        }
                    }
                }
                const int nb = min(per_batch, n - u0);
                for (int i = 0; i < nb; ++i) {
                    // boxes of a 16-bit tile: lane = piece * boxes + column box; of a
                    // stored e4m3 tile: one per piece, then (with K) the scales of K and V
                    const int piece = FP8 ? lane & (pieces - 1) : lane / C::kBoxes & (pieces - 1);
                    const int src = (i << pcs_log2) + piece;
                    const int page = __shfl_sync(0xffffffffu, id, src);
                    const int y = __shfl_sync(0xffffffffu, row, src);
#pragma unroll
                    for (int t = 0; t < 2; ++t, ++ld) {
                        const void* map = t ? &maps.v : &maps.k;
                        if constexpr (!FP8) {
                            const int s = ld % C::kSlots;
                            const uint32_t use = ld / C::kSlots;
                            if (use > 0) wait_bar(bar(bars->kv_empty[s]), (use - 1) & 1, abort, p.status);
                            const uint32_t full = bar(bars->kv_full[s]);
                            if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
                            __syncwarp();
                            if (lane < pieces * C::kBoxes) {
                                const int bx = lane % C::kBoxes;
                                const uint32_t dst = base + C::kSlotOff + s * C::kTileBytes + bx * C::kBoxBytes + piece * pr * 128;
                                if constexpr (D == 128)
                                    tma_load_5d(dst, map, 0, y, bx, head, page, full);
                                else
                                    tma_load_4d(dst, map, 0, y, head, page, full);
                            }
                        } else {
                            const int s = ld % C::kRaws;
                            const uint32_t use = ld / C::kRaws;
                            if (use > 0) wait_bar(bar(bars->raw_empty[s]), (use - 1) & 1, abort, p.status);
                            const uint32_t full = bar(bars->raw_full[s]);
                            if (lane == 0) mbar_arrive_expect_tx(full, C::kRawBytes + (t == 0 ? 2 * kBN : 0));
                            __syncwarp();
                            const int what = lane >> pcs_log2;
                            if (what == 0)
                                tma_load_4d(base + C::kRawOff + s * C::kRawBytes + piece * pr * D, map, 0, y, head, page, full);
                            else if (t == 0 && what <= 2)
                                tma_load_3d(base + C::kExpOff + s * C::kExpBytes + (what - 1) * 1024 + piece * 128,
                                            what == 1 ? &maps.ke : &maps.ve, y, head, page, full, policy_evict_first());
                        }
                        __syncwarp();
                    }
                }
            }
            seg_done(k);
        }
        // nothing may still be landing in this CTA's shared memory when it exits: neither
        // a copy (aborted kernels) nor a commit's arrival
        if constexpr (FP8) {
            if (*abort)
                for (uint32_t i = ld > C::kRaws ? ld - C::kRaws : 0; i < ld; ++i)
                    wait_bar(bar(bars->raw_full[i % C::kRaws]), (i / C::kRaws) & 1, abort, p.status);
        } else if (*abort) {
            for (uint32_t i = ld > C::kSlots ? ld - C::kSlots : 0; i < ld; ++i)
                wait_bar(bar(bars->kv_full[i % C::kSlots]), (i / C::kSlots) & 1, abort, p.status);
        }
        for (uint32_t i = ld > C::kSlots ? ld - C::kSlots : 0; i < ld; ++i)
            wait_bar(bar(bars->kv_empty[i % C::kSlots]), (i / C::kSlots) & 1, abort, p.status);
    } else if (warp == kIssuer) {
        regs_decrease<C::kRegsRest>();
        // ============================================================ products, in a fixed order
        constexpr uint32_t idesc_s = idesc_of(FP8, kBN, false), idesc_o = idesc_of(FP8, D, true);
        const uint64_t desc_k = smem_desc_sw128(0, 16, 1024);
        const uint64_t desc_v = smem_desc_sw128(0, C::kBoxBytes, 1024);
        uint32_t waited = 0;                             // tiles waited for
        const auto slot_addr = [&](uint32_t i) { return base + C::kSlotOff + (i % C::kSlots) * C::kTileBytes; };
        const auto wait_kv = [&](uint32_t i) {
            while (waited <= i) {
                wait_bar(bar(bars->kv_full[waited % C::kSlots]), (waited / C::kSlots) & 1, abort, p.status);
                ++waited;
            }
            tc_fence_after();
        };
        const auto issue_s = [&](int ti, uint32_t i) {
            const uint64_t a = desc_k + ((base + ti * C::kTileBytes) >> 4), b = desc_k + (slot_addr(i) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
                mma_ss_elect(tmem + 128u * ti, a + o, b + o, idesc_s, kk > 0 ? 1u : 0u);
            }
            mma_commit_elect(bar(bars->s_full[ti]));
        };
        const auto issue_pv = [&](int ti, uint32_t i, bool first, int h) {
            const uint64_t b = desc_v + (slot_addr(i) >> 4);
            const uint32_t a = tmem + 128u * ti, d = tmem + C::kColO + static_cast<uint32_t>(D) * ti;
#pragma unroll
            for (int k4 = 0; k4 < (h ? kW1 : kW0) / 8; ++k4) {
                const int kk = (h ? kW0 / 8 : 0) + k4;
                mma_ts_elect(d, a + kk * 8, b + kk * (2048 >> 4), idesc_o, (!first || kk > 0) ? 1u : 0u);
            }
        };
        uint32_t ld = 0;                                 // tiles of earlier segments
        uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
        for (uint32_t k = 0;; ++k) {
            const TileSegment& g = seg_wait(k);
            const int n = g.n;
            if (n == 0) break;
            const int tiles = g.r1 - g.r0 > 128 ? 2 : 1;
            for (int ti = 0; ti < tiles; ++ti) {
                wait_kv(ld);
                wait_bar(bar(bars->q_full[ti]), qn[ti]++ & 1, abort, p.status);
                tc_fence_after();
                issue_s(ti, ld);
            }
            mma_commit_elect(bar(bars->kv_empty[ld % C::kSlots]));
            for (int u = 0; u < n; ++u) {
                const uint32_t vi = ld + 2 * u + 1;
                for (int ti = 0; ti < tiles; ++ti) {
                    wait_bar(bar(bars->p_half[ti]), pn[ti] & 1, abort, p.status);
                    tc_fence_after();
                    wait_kv(vi);
                    if constexpr (!FP8) {
                        const int k0 = key_tile(g, u) * kBN;
                        if (ti == 0 && (k0 + kBN > g.hi || (k0 < g.lo && k0 + kBN > g.sk))) {
                            // rows of V that no query row sees
                            const uint32_t v = slot_addr(vi);
                            for (int x = lane; x < kBN * 8; x += 32)
                                if (!alive(g, k0 + (x >> 3))) {
#pragma unroll
                                    for (int bx = 0; bx < C::kBoxes; ++bx)
                                        st_shared_v4(v + bx * C::kBoxBytes + 16 * x, 0u, 0u, 0u, 0u);
                                }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    issue_pv(ti, vi, u == 0, 0);
                    wait_bar(bar(bars->p_full[ti]), pn[ti] & 1, abort, p.status);
                    ++pn[ti];
                    tc_fence_after();
                    issue_pv(ti, vi, u == 0, 1);
                    if (u + 1 < n) {
                        wait_kv(vi + 1);
                        issue_s(ti, vi + 1);
                    } else {
                        mma_commit_elect(bar(bars->o_full[ti]));
                    }
                }
                mma_commit_elect(bar(bars->kv_empty[vi % C::kSlots]));
                if (u + 1 < n) mma_commit_elect(bar(bars->kv_empty[(vi + 1) % C::kSlots]));
            }
            ld += 2 * n;
            seg_done(k);
        }
    } else if (warp == kSched) {
        regs_decrease<C::kRegsRest>();
        // ============================================================ segments
        if (few_seqs(p)) start = locate_warp<kRT, kBN>(p, blockIdx.x, lane);
        Walk<kRT, kBN> walk;
        walk.begin(p, start);
        const Item& it = walk.it;
        uint32_t loads[2] = {0, 0};                      // of Q's tiles
        for (uint32_t k = 0;; ++k) {
            if (k >= 2) wait_bar(bar(bars->seg_empty[k & 1]), ((k >> 1) - 1) & 1, abort, p.status);
            TileSegment g;
            g.n = 0;
            int unit, n;
            if (walk.segment(p, unit, n)) {
                fill_segment(g, it, unit, n);
#pragma unroll
                for (int ti = 0; ti < 2; ++ti) {
                    const int a = it.r0 + 128 * ti, e = min(it.r1, a + 128) - 1;
                    g.all[ti] = min(it.p0 + a / p.group + 1, it.hi);
                    g.none[ti] = p.window == kNoWindow ? 0 : it.p0 + e / p.group - p.window + 1;
                }
            }
            if (lane == 0) {
                bars->seg[k & 1] = g;
                mbar_arrive(bar(bars->seg_full[k & 1]));
            }
            __syncwarp();
            if (g.n == 0) break;
            if (p.q_tma) {
                // Q's tiles as boxes of [tokens][heads of the group][64], once the last
                // segment is done with them
#pragma unroll
                for (int ti = 0; ti < 2; ++ti) {
                    if (g.r1 - g.r0 <= 128 * ti) continue;
                    if (loads[ti] > 0) wait_bar(bar(bars->q_free[ti]), (loads[ti] - 1) & 1, abort, p.status);
                    ++loads[ti];
                    const uint32_t full = bar(FP8 ? bars->q_raw[ti] : bars->q_full[ti]);
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
                        for (int bx = 0; bx < C::kBoxes; ++bx)
                            tma_load_3d(base + ti * C::kTileBytes + bx * C::kBoxBytes, &maps.q, 64 * bx, g.head * p.group,
                                        g.row0 + (g.r0 + 128 * ti) / p.group, full, policy_evict_first());
                    }
                    __syncwarp();
                }
            }
            walk.next(p);
        }
        // (aborted kernels) none of Q's copies may land after the CTA has gone
        if (*abort)
            for (int ti = 0; ti < 2; ++ti)
                if (loads[ti] > 0)
                    wait_bar(bar(FP8 ? bars->q_raw[ti] : bars->q_full[ti]), (loads[ti] - 1) & 1, abort, p.status);
    } else if (FP8 && warp >= kWiden) {
        regs_decrease<C::kRegsRest>();
        // ============================================================ e4m3 tiles to f16, one row per thread
        if constexpr (FP8) {
            const int r = threadIdx.x - 32 * kWiden, w4 = warp - kWiden;
            uint32_t i = 0;                              // tiles so far
            for (uint32_t k = 0;; ++k) {
                const TileSegment& g = seg_wait(k);
                const int n = g.n;
                if (n == 0) break;
                uint32_t mul_v = 0;
                bool live = true;
                // one copy of the loop for K and V, and short unrolling: with the softmax's
                // code this has to stay within the instruction cache (fully unrolled, a third of
                // the stalls were instruction fetches)
#pragma unroll 1
                for (int x = 0; x < 2 * n; ++x, ++i) {
                    const int rs = i % C::kRaws, s = i % C::kSlots;
                    wait_bar(bar(bars->raw_full[rs]), (i / C::kRaws) & 1, abort, p.status);
                    uint32_t mul = mul_v;
                    if ((x & 1) == 0) {
                        live = alive(g, key_tile(g, x >> 1) * kBN + r);
                        // the largest and smallest scales of the tile, of K and of V
                        const uint8_t* ex = smem + C::kExpOff + rs * C::kExpBytes + ((r >> pr_log2) << 7) + (r & (pr - 1));
                        const int ek = live ? min(static_cast<int>(ex[0]), 253) : 0;
                        const int ev = live ? min(static_cast<int>(ex[1024]), 253) : 0;
                        const int mk = __reduce_max_sync(0xffffffffu, ek), mv = __reduce_max_sync(0xffffffffu, ev);
                        // (rows at the lowest scale, zeros among them, may count as zeros)
                        const int nk = __reduce_min_sync(0xffffffffu, ek > 64 ? ek : 255);
                        const int nv = __reduce_min_sync(0xffffffffu, ev > 64 ? ev : 255);
                        const int par = (i >> 1) & 1;
                        if (lane == 0) {
                            bars->red[8 * par + w4] = mk | nk << 8;
                            bars->red[8 * par + 4 + w4] = mv | nv << 8;
                        }
                        named_barrier_sync(3, 128);
                        int tk = 64, tv = 64, lk = 255, lv = 255;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int wk = bars->red[8 * par + q], wv = bars->red[8 * par + 4 + q];
                            tk = max(tk, wk & 0xff);
                            tv = max(tv, wv & 0xff);
                            lk = min(lk, wk >> 8);
                            lv = min(lv, wv >> 8);
                        }
                        const uint32_t f = (i >> 1) & 3;
                        // taken by key: codes times 2^6
                        const bool by_key = tk > lk + kSpanK || tv > lv + kSpanV;
                        mul = f16_power(by_key ? 6 : ek - tk + 6) * 0x10001u;
                        mul_v = f16_power(by_key ? 6 : ev - tv + 6) * 0x10001u;
                        if (r == 0) {
                            bars->fac[2 * f] = by_key ? 0.f : __uint_as_float(static_cast<uint32_t>(tk - 6) << 23);
                            bars->fac[2 * f + 1] = static_cast<float>(tv - 6 - 127);
                        }
                        if (by_key) {
                            reinterpret_cast<uint8_t*>(bars->by_key[f][0])[r] = static_cast<uint8_t>(ek);
                            reinterpret_cast<uint8_t*>(bars->by_key[f][1])[r] = static_cast<uint8_t>(ev);
                        }
                    }
                    if (i >= C::kSlots) wait_bar(bar(bars->kv_empty[s]), (i / C::kSlots - 1) & 1, abort, p.status);
                    const uint32_t raw = base + C::kRawOff + rs * C::kRawBytes + r * D;
                    const uint32_t out = base + C::kSlotOff + s * C::kTileBytes + r * 128;
                    const uint32_t sw = r & 7, rsw = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll 2
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t v[4], h[8];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                     : "r"(raw + ((c ^ rsw) << 4))
                                     : "memory");
                        // a row that no query sees may hold anything: it becomes zeros
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            widen4(live ? v[q] : 0u, h[2 * q], h[2 * q + 1]);
                            h[2 * q] = mul_f16x2(h[2 * q], mul);
                            h[2 * q + 1] = mul_f16x2(h[2 * q + 1], mul);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = 2 * c + e;
                            st_shared_v4(out + (ch >> 3) * C::kBoxBytes + (((ch & 7) ^ sw) << 4), h[4 * e], h[4 * e + 1],
                                         h[4 * e + 2], h[4 * e + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(bars->raw_empty[rs]));
                        mbar_arrive(bar(bars->kv_full[s]));
                    }
                }
                seg_done(k);
            }
        }
    } else {
        regs_decrease<C::kRegsRest>();
    }

    // This kernel's end stands for the end of all of the call's earlier ones.
    if (p.after_rows) wait_for_previous();
    tc_fence_before();
    __syncthreads();
    if (warp == kSched) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool FP8>
int launch(const fa_kv_cache* c, const AttnParams& p, const AttnParams* beside, int rows, cudaStream_t s) {
    using C = Cfg<D, FP8>;
    alignas(64) Maps maps{};
    if (c->prepared) {
        const Prepared* m = static_cast<const Prepared*>(c->prepared);
        memcpy(&maps, &m->k, 4 * sizeof(CUtensorMap));
    } else {
        alignas(64) Prepared m;
        if (encode_tiles(m, c) != FA_OK) return FA_ERR_CUDA;
        memcpy(&maps, &m.k, 4 * sizeof(CUtensorMap));
    }
    if (p.q_tma && encode_q(&maps.q, p, c->d) != FA_OK) return FA_ERR_CUDA;
    if (p.after_rows) {
        const int rc = launch_early(tiles_kernel<D, FP8>, dim3(p.ctas), C::kThreads, C::kSmemBytes, s, maps, p);
        if (rc != FA_OK) return rc;
    } else {
        tiles_kernel<D, FP8><<<p.ctas, C::kThreads, C::kSmemBytes, s>>>(maps, p);
        if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    }
    if (!beside) return launch_join<kRT, D>(p, s);
    switch (rows) {
        case 8: return launch_join_both<8, D>(*beside, p, s);
        case 16: return launch_join_both<16, D>(*beside, p, s);
        case 32: return launch_join_both<32, D>(*beside, p, s);
        default: return launch_join_both<64, D>(*beside, p, s);
    }
}

template <int D, bool FP8>
bool opt_in() {
    return cudaFuncSetAttribute(tiles_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<D, FP8>::kSmemBytes) == cudaSuccess;
}

}  // namespace

int launch_tiles(const fa_kv_cache* c, const AttnParams& p, const AttnParams* beside, int rows, cudaStream_t s) {
    const bool fp8 = c->type == FA_KV_E4M3;
    if (c->d == 128) return fp8 ? launch<128, true>(c, p, beside, rows, s) : launch<128, false>(c, p, beside, rows, s);
    return fp8 ? launch<64, true>(c, p, beside, rows, s) : launch<64, false>(c, p, beside, rows, s);
}

int encode_tiles(Prepared& m, const fa_kv_cache* c) {
    const int rows = static_cast<int>(c->page_size < kBN ? c->page_size : kBN);
    if (encode_cache(&m.k, c, c->k, rows, true) || encode_cache(&m.v, c, c->v, rows, true)) return FA_ERR_CUDA;
    memset(&m.ke, 0, sizeof(m.ke));
    memset(&m.ve, 0, sizeof(m.ve));
    if (c->type == FA_KV_E4M3 && (encode_exps(&m.ke, c, c->k_exp, rows) || encode_exps(&m.ve, c, c->v_exp, rows)))
        return FA_ERR_CUDA;
    return FA_OK;
}

int tiles_setup() {
    return opt_in<128, true>() && opt_in<128, false>() && opt_in<64, true>() && opt_in<64, false>() ? FA_OK
                                                                                                   : FA_ERR_CUDA;
}

}  // namespace paged
}  // namespace fa
