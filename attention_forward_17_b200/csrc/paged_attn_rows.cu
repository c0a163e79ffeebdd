// Paged attention for few query rows per key head: single tokens, a few
// tokens at a time, or groups of heads ("decoding").
//
// Every cached key and value is read once and used by the 8 to 48 query rows
// of an item, so HBM bounds the kernel: 2 d bytes (bf16) or d + 1 (e4m3) per
// cached row and tensor against 4 d flops per row pair.  The matrix unit is reached
// through warp-level products (mma m16n8k16) with the keys (and V's columns) along
// their 16-wide side and the query rows along the 8-wide one:
//     S^T = K Q^T,   O^T = V^T P^T,
// so that the usual 1 to 8 rows of a key head fill a product, where a 128-row
// tcgen05 tile would be 15/16 or more empty.  An e4m3 value goes from shared memory to the
// product through registers, widened on the way, without a trip back to shared memory.
//
// One CTA per SM (384 threads) works through its stretch of the work list
// (paged_attn.cuh) in units of kUnit keys: 16 KiB of K and V (8 for e4m3 at d = 64),
// since a unit costs the loading warps the same whatever its size (bf16, d = 64, 32 sequences over
// 8,192: 121 us with units of 32 keys, 86 with 64; 64 rows an item 60 and 63):
//   warps 8-11  producers: 8 and 10 of K, 9 and 11 of V, one pair for the even units and one for the odd
//               ones.  The first also cuts the work list and writes each segment's
//               description to shared memory for the others.  Each looks the page ids of up
//               to 32 units up at a time, and one of its lanes loads its tensor (and scales)
//               of one key head with TMA, one box per page, into a ring of stages of one
//               unit.  The instructions spent on a unit here bound short units and small
//               pages: 64 tokens over 269,572 cached e4m3, 125 us with one warp for all and the lanes
//               issuing side by side, 116 with two warps, 102 with one lane working through a
//               list, 99 with four warps (d = 64, 32 over 8,192: 84 and 70; bf16, d = 64,
//               pages of 16, 64 over 3,001: 93 and 74).
//   warps 0-7   consumers: MT row tiles of 8 NR rows x the unit's 32-key parts x groups.  Units go
//               round robin over the groups, each unit to the warps of one group;
//               every warp keeps its own running maximum, sums and output, so the
//               warps share nothing until a segment ends, when the groups'
//               results are joined through shared memory.
// A ring of 128 KiB keeps enough bytes in flight to cover HBM's latency (about 45 KB per SM).
//
// e4m3 caches.  K codes are widened to f16 (exact) and Q to f16 after each row
// is scaled by a power of two to a largest magnitude in [1, 2) (its 8 significant bits fit; an
// element below 2^-24 of the row's largest is lost, 2^-17 of that element's rounding at
// the top).  V's scale 2^b_j is a power of two, so it joins the exponent of the
// weight: with t_j = s_j + b_j (base 2) and m the running maximum of t,
//     O = sum 2^(t_j - m) code_j / l,   l = sum 2^(t_j - m) 2^-b_j,
// and the weights that meet the codes are f16 numbers 2^(t_j - m) between 2^15 and 2^-24, kept
// near 2^8 at the top, so weights down to 2^-22 of the largest keep all 11 bits.  (8-bit warp-level
// products with Q in two e4m3 parts need no widening of K, but took more instructions in the end,
// not fewer: 134 us instead of 127.)
//
// Measured on one B200 (device time, inputs larger than L2): 2 sequences x 131,071 cached tokens, 8
// key heads of 4 query heads, d = 128, bf16: 162 us with the join, 1.07 GB, 6.6 TB/s, 1.0 of the measured
// copy.  64 sequences, 269,572 cached e4m3: 99 us, 0.557 GB, 5.7 TB/s, 0.86: there the widening
// (ALU 48 % busy) and 512 items' starts and ends cost beside the loads (the loads
// without the arithmetic: 92 us).
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "paged_attn.cuh"

namespace fa {
namespace paged {
namespace {

constexpr int kConsumers = 8;
constexpr int kProducers = 4;
constexpr int kThreads = 32 * (kConsumers + kProducers);

template <int D, bool FP8>
struct Cfg {
    static constexpr int kUnitLog2 = FP8 || D == 64 ? 6 : 5;
    static constexpr int kUnit = 1 << kUnitLog2;         // keys of a unit, a stage of the ring
    // Warps that share a unit, 32 keys each: with one warp to a unit of 64 keys every stage could be
    // in work and none loading.
    static constexpr int kParts = kUnit / 32;
    static constexpr int kRowBytes = FP8 ? D : 2 * D;
    static constexpr int kTensorBytes = kUnit * kRowBytes;
    static constexpr int kStageBytes = 2 * kTensorBytes;
    // A multiple of the 8 consumer warps, so that a stage always belongs to the same
    // group: a warp then waits for use k of a stage after it has itself seen use k - 1,
    // without which the wait's parity could stand for use k - 2.
    static constexpr int kStages = FP8 && D == 64 ? 16 : 8;
    static_assert(kStages % kConsumers == 0, "stages belong to groups");
    static constexpr int kExpBytes = FP8 ? 1024 : 0;     // scales per stage: [k, v][4 pieces][128]
    static constexpr int kExpOff = kStages * kStageBytes;
    static constexpr int kMergeOff = kExpOff + kStages * kExpBytes;
    static constexpr int kPitch = D + 4;                 // floats
    static constexpr int kMergeBytes = kConsumers * 16 * kPitch * 4;     // room for NR = 2
    static constexpr int kStatOff = kMergeOff + kMergeBytes;
    static constexpr int kStatBytes = kConsumers * 16 * 3 * 4;
    static constexpr int kBarOff = kStatOff + kStatBytes;
    static constexpr int kSegOff = kBarOff + 16 * kStages + 32;     // ring barriers, segment barriers, segments
    static constexpr int kSmemBytes = 1024 + kSegOff + 2 * static_cast<int>(sizeof(Segment)) + 16;
    static_assert(kSmemBytes <= 232448 - 1024, "shared memory per CTA");
    static_assert(kStageBytes % 1024 == 0, "stages on 1024-byte boundaries (swizzle)");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// D += A B, 16 x 8 x 16; FP8 caches run in f16, bf16 caches in bf16.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 to two f16 pairs.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Over the eight lanes that hold the same query rows.
__device__ __forceinline__ float keys_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float keys_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
// An 8 x 8 tile of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// A row's running maximum may lag by this much (base 2) before its output is
// rescaled: weights stay below 2^16 (bf16) or 2^15 (f16, whose fresh maximum is
// placed at 2^8).
template <bool FP8>
struct Lazy {
    static constexpr float kTau = FP8 ? 15.f : 16.f;
    static constexpr float kTop = FP8 ? 8.f : 0.f;
};

// NR: tiles of 8 query rows per warp.
template <int D, bool FP8, int NR, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams p) {
    using C = Cfg<D, FP8>;
    constexpr int kWarpRows = 8 * NR, RT = kWarpRows * MT;
    constexpr int kAhead = NR == 1 ? 4 : 2;              // k steps of K's fragments loaded ahead (registers)
    constexpr int kUnit = C::kUnit, kGroups = kConsumers / MT / C::kParts;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Scratch scratch;
    __shared__ int2 lists[32 * kProducers];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t full = base + C::kBarOff, empty = full + 8 * C::kStages;
    const uint32_t seg_full = empty + 8 * C::kStages, seg_empty = seg_full + 16;
    Segment* segs = reinterpret_cast<Segment*>(smem + C::kSegOff);
    volatile uint32_t* abort = reinterpret_cast<uint32_t*>(segs + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + 8 * s, 2);                  // a producer of K and one of V
            mbar_init(empty + 8 * s, MT * C::kParts);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(seg_full + 8 * i, 1);
            mbar_init(seg_empty + 8 * i, kConsumers + kProducers - 1);
        }
        *abort = p.abandoned;
        fence_barrier_init();
    }
    let_next_start();
    Start start{0, 0, 0, 0, 0, 0};
    if (!few_seqs(p)) start = locate_block<RT, kUnit>(p, blockIdx.x, &scratch);
    __syncthreads();

    const int pr_log2 = min(p.b.page_log2, C::kUnitLog2);     // rows of a page piece: 16 .. kUnit
    const int pr = 1 << pr_log2;

    if (warp >= kConsumers) {
        // ============================================================ producers: K, V
        const int tensor = (warp - kConsumers) & 1, first = (warp - kConsumers) >> 1;
        const bool leader = warp == kConsumers;
        const int pcs_log2 = C::kUnitLog2 - pr_log2, pieces = 1 << pcs_log2;   // 1, 2 or 4
        const int per_batch = 32 >> pcs_log2;
        const int page_mask = (1 << p.b.page_log2) - 1;
        const uint32_t piece_bytes = pr * C::kRowBytes;
        const void* map = tensor ? &maps.v : &maps.k;
        const void* emap = tensor ? &maps.ve : &maps.ke;
        const uint32_t tiles = base + tensor * C::kTensorBytes;
        int2* list = lists + 32 * (warp - kConsumers);                // page id and first row of each piece
        Walk<RT, kUnit> walk;                            // (the first producer only)
        if (leader) {
            if (few_seqs(p)) start = locate_warp<RT, kUnit>(p, blockIdx.x, lane);
            walk.begin(p, start);
        }
        const uint64_t keep = policy_evict_first();
        uint32_t g = 0, s = 0, use = 0;                  // units so far; the next one's stage, and that stage's uses
        for (uint32_t k = 0;; ++k) {
            if (leader) {
                if (k >= 2) wait_bar(seg_empty + 8 * (k & 1), ((k >> 1) - 1) & 1, abort, p.status);
                int unit, n;
                const bool more = walk.segment(p, unit, n);
                if (lane == 0) {
                    if (more)
                        fill_segment(segs[k & 1], walk.it, unit, n);
                    else
                        segs[k & 1].n = 0;
                    mbar_arrive(seg_full + 8 * (k & 1));
                }
                __syncwarp();
            } else {
                wait_bar(seg_full + 8 * (k & 1), (k >> 1) & 1, abort, p.status);
            }
            const Segment& sg = segs[k & 1];
            const int n = sg.n, head = sg.head, hi = sg.hi, lo = sg.lo, sinks = sg.sk;
            if (n == 0) break;
            const int32_t* table = p.b.table + sg.seq * p.b.table_stride;
            for (int u0 = 0; u0 < n; u0 += per_batch) {
                // page id and first row of this lane's (unit, piece)
                const int lu = u0 + (lane >> pcs_log2);
                int id = -1, row = 0;
                if (lu < n) {
                    const int pos = key_tile(sg, lu) * kUnit + (lane & (pieces - 1)) * pr;
                    row = pos & page_mask;
                    if (pos < hi && (pos + pr > lo || pos < sinks)) {
                        id = __ldg(table + (pos >> p.b.page_log2));
                        if (id < 0 || id >= p.b.pages) {
                            report_page(p.status);
                            id = -1;                     // the load fills with zeros
                        }
                    }
                }
                list[lane] = make_int2(id, row);
                __syncwarp();
                // one lane issues, from the list: what a unit costs here is what bounds short units
                const int nb = min(per_batch, n - u0);
                if (lane == 0) {
                    const int2* e = list;
                    for (int i = 0; i < nb; ++i) {
                        if (((g + i) & 1) == first) {          // the stage count is even: a stage has one pair of producers
                            const uint32_t bar = full + 8 * s;
                            if (use > 0) wait_one(empty + 8 * s, (use - 1) & 1, abort, p.status);
                            mbar_arrive_expect_tx(bar, C::kTensorBytes + (FP8 ? kUnit : 0));
                            uint32_t dst = tiles + s * C::kStageBytes;
                            uint32_t edst = base + C::kExpOff + s * C::kExpBytes + tensor * 512;
#pragma unroll 1
                            for (int pc = 0; pc < pieces; ++pc, ++e, dst += piece_bytes, edst += 128) {
                                const int2 at = *e;
                                if constexpr (!FP8 && D == 128)
                                    tma_load_5d(dst, map, 0, at.y, 0, head, at.x, bar);
                                else
                                    tma_load_4d(dst, map, 0, at.y, head, at.x, bar);
                                if constexpr (FP8) tma_load_3d(edst, emap, at.y, head, at.x, bar, keep);
                            }
                        } else {
                            e += pieces;
                        }
                        if (++s == C::kStages) {
                            s = 0;
                            ++use;
                        }
                    }
                }
                g += nb;
                s = g % C::kStages;
                use = g / C::kStages;
                __syncwarp();
            }
            if (leader)
                walk.next(p);
            else if (lane == 0)
                mbar_arrive(seg_empty + 8 * (k & 1));
        }
        // no copy may still be landing when the CTA exits
        if (*abort)
            for (uint32_t k = g > C::kStages ? g - C::kStages : 0; k < g; ++k)
                wait_bar(full + 8 * (k % C::kStages), (k / C::kStages) & 1, abort, p.status);
        return;
    }

    // ================================================================ consumers
    const int gr = lane >> 2, c4 = lane & 3;             // row (and key) of a fragment, column pair
    const int mt = warp % MT, sub = 32 * (warp / MT % C::kParts), group = warp / MT / C::kParts;
    float* merge = reinterpret_cast<float*>(smem + C::kMergeOff);
    float* stats = reinterpret_cast<float*>(smem + C::kStatOff);
    // offset of key r of a unit in its stage, before the swizzled chunk
    const auto key_off = [&](int r) -> uint32_t {
        if constexpr (!FP8 && D == 128)
            return (r >> pr_log2) * (pr * 256) + (r & (pr - 1)) * 128;
        else
            return r * C::kRowBytes;
    };
    uint32_t gbase = 0;
    for (uint32_t sk = 0;; ++sk) {
        wait_bar(seg_full + 8 * (sk & 1), (sk >> 1) & 1, abort, p.status);
        const Segment& sg = segs[sk & 1];
        const int n = sg.n;
        if (n == 0) break;
        const int rbase = sg.r0 + kWarpRows * mt;
        const bool idle = rbase >= sg.r1;
        // Q as B fragments: row 8 q + gr of the warp's, and the factors of the scores of
        // the rows whose scores this lane gets: 8 q + 2 c4 + {0, 1}
        uint32_t qf[NR][D / 16][2];
        float cr[NR][2];
        // every row of the warp sees the keys of [none, all)
        int all = 0, none = 0;
        if (!idle) {
            all = min(sg.p0 + rbase / p.group + 1, sg.hi);
            none = p.window == kNoWindow ? 0 : sg.p0 + (min(rbase + kWarpRows, sg.r1) - 1) / p.group - p.window + 1;
#pragma unroll
            for (int q = 0; q < NR; ++q) {
                const int r = rbase + 8 * q + gr;
                const bool ok = r < sg.r1;
                const uint16_t* src = p.q;
                if (ok) {
                    int64_t token;
                    int head;
                    row_place(p, sg.row0, sg.head, r, token, head);
                    src = p.q + token * p.q_ts + head * p.q_hs;
                }
                if constexpr (!FP8) {
                    // elements 16 ks + 2 c4 .. + 1 and + 8
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            qf[q][ks][k] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 * k + 2 * c4)) : 0u;
                    cr[q][0] = cr[q][1] = p.scale_log2;
                } else {
                    // this lane's D / 4 consecutive elements: k step ks takes the
                    // next four (K's fragments are read in the same order)
                    uint32_t v[D / 8];
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 t = ok ? __ldg(reinterpret_cast<const uint4*>(src + (D / 4) * c4 + 8 * i))
                                           : make_uint4(0u, 0u, 0u, 0u);
                        v[4 * i] = t.x;
                        v[4 * i + 1] = t.y;
                        v[4 * i + 2] = t.z;
                        v[4 * i + 3] = t.w;
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // scale the row by 2^(127 - e), e the exponent field of its largest element
                    const int e = min(max(static_cast<int>(top >> 7), 1), 253);
                    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            qf[q][ks][k] = pack_f16x2(__uint_as_float(v[2 * ks + k] << 16) * inv,
                                                      __uint_as_float(v[2 * ks + k] & 0xffff0000u) * inv);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        cr[q][x] = p.scale_log2 *
                                   __uint_as_float(static_cast<uint32_t>(__shfl_sync(0xffffffffu, e, 4 * (2 * c4 + x))) << 23);
                }
            }
        }
        float o[NR][D / 16][4];                          // O^T: 16 columns x 8 rows each
        float m[NR][2], l[NR][2], lh[NR][2];
#pragma unroll
        for (int q = 0; q < NR; ++q) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[q][i][0] = o[q][i][1] = o[q][i][2] = o[q][i][3] = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                m[q][x] = -INFINITY;
                l[q][x] = lh[q][x] = 0.f;
            }
        }

        for (int u = (group + kGroups - static_cast<int>(gbase % kGroups)) % kGroups; u < n; u += kGroups) {
            const uint32_t g = gbase + u;
            const int s = g % C::kStages;
            const int k0 = key_tile(sg, u) * kUnit;
            wait_bar(full + 8 * s, (g / C::kStages) & 1, abort, p.status);
            // this warp's 32 keys: two tiles of 16
            if (!idle) {
                const int j0 = k0 + sub;
                const uint32_t ks_ = base + s * C::kStageBytes, vs_ = ks_ + C::kTensorBytes;
                float t[NR][2][4];                       // S^T: keys gr, gr + 8 x rows 2 c4, 2 c4 + 1
#pragma unroll
                for (int q = 0; q < NR; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) t[q][i][0] = t[q][i][1] = t[q][i][2] = t[q][i][3] = 0.f;
                // ---- scores; K's fragments are loaded ahead of the products
                if constexpr (!FP8) {
                    const int kr = lane & 15;
                    const uint32_t b0 = ks_ + key_off(sub + kr), b1 = ks_ + key_off(sub + kr + 16);
                    const uint32_t ch = lane >> 4, sw = lane & 7;
#pragma unroll
                    for (int kb = 0; kb < D / 16; kb += kAhead) {
                        uint32_t f0[kAhead][4], f1[kAhead][4];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const uint32_t off = (kb >> 2) * (pr * 128) + (((2 * ((kb + k) & 3) + ch) ^ sw) << 4);
                            ldsm4(f0[k], b0 + off);
                            ldsm4(f1[k], b1 + off);
                        }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
#pragma unroll
                            for (int q = 0; q < NR; ++q) {
                                mma16816<false>(t[q][0], f0[k], qf[q][kb + k][0], qf[q][kb + k][1]);
                                mma16816<false>(t[q][1], f1[k], qf[q][kb + k][0], qf[q][kb + k][1]);
                            }
                    }
                } else {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        uint4 x[4];                      // keys gr, gr + 8 of both tiles
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = sub + 8 * i + gr;
                            const uint32_t ch = D == 128 ? (2 * c4 + hf) ^ (r & 7) : c4 ^ ((r >> 1) & 3);
                            x[i] = lds128(ks_ + r * D + (ch << 4));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t f[4];
                                widen4(k == 0 ? x[2 * i].x : k == 1 ? x[2 * i].y : k == 2 ? x[2 * i].z : x[2 * i].w, f[0], f[2]);
                                widen4(k == 0 ? x[2 * i + 1].x : k == 1 ? x[2 * i + 1].y : k == 2 ? x[2 * i + 1].z : x[2 * i + 1].w,
                                       f[1], f[3]);
#pragma unroll
                                for (int q = 0; q < NR; ++q)
                                    mma16816<true>(t[q][i], f, qf[q][4 * hf + k][0], qf[q][4 * hf + k][1]);
                            }
                    }
                }
                // ---- scale, mask
                float vinv[2][2];                        // e4m3: 2^-b of V's scale, of this lane's four keys
                if constexpr (FP8) {
                    const uint32_t eb = base + C::kExpOff + s * C::kExpBytes;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int r = sub + 16 * i + 8 * y + gr;
                            const uint32_t at = eb + ((r >> pr_log2) << 7) + (r & (pr - 1));
                            const uint32_t ek = min(lds_u8(at), 253u), ev = min(lds_u8(at + 512), 253u);
                            const float kf = __uint_as_float(ek << 23);
                            const float vb = static_cast<float>(static_cast<int>(ev) - 127);
                            vinv[i][y] = __uint_as_float((254u - ev) << 23);
#pragma unroll
                            for (int q = 0; q < NR; ++q)
#pragma unroll
                                for (int x = 0; x < 2; ++x) t[q][i][2 * y + x] = fmaf(t[q][i][2 * y + x], cr[q][x] * kf, vb);
                        }
                } else {
#pragma unroll
                    for (int q = 0; q < NR; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) t[q][i][e] *= p.scale_log2;
                }
                const bool masked = j0 + 32 > all || (j0 < none && j0 + 32 > p.sinks);
                // masks of V's key pairs: keys that no row of the item sees hold
                // anything, so they must not meet their weight of zero
                uint32_t dead[4];
                if (masked) {
#pragma unroll
                    for (int q = 0; q < NR; ++q)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            // visible keys of the row: j < h and (j >= w or j < sinks)
                            const int r = rbase + 8 * q + 2 * c4 + x, pos = sg.p0 + r / p.group;
                            const int h = r < sg.r1 ? min(pos + 1, sg.hi) : 0;
                            const int w = p.window == kNoWindow ? 0 : pos - p.window + 1;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int j = j0 + 16 * i + 8 * y + gr;
                                    if (!(j < h && (j >= w || j < p.sinks))) t[q][i][2 * y + x] = -INFINITY;
                                }
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + 8 * i + 2 * c4;
                        dead[i] = (alive(sg, j) ? 0xffffu : 0u) | (alive(sg, j + 1) ? 0xffff0000u : 0u);
                    }
                }
                // ---- running maximum
                bool grow = false;
                float alpha[NR][2];
#pragma unroll
                for (int q = 0; q < NR; ++q)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float mx = keys_max(fmaxf(max3f(t[q][0][x], t[q][0][x + 2], t[q][1][x]), t[q][1][x + 2]));
                        alpha[q][x] = 1.f;
                        if (mx > m[q][x] + Lazy<FP8>::kTau) {
                            grow = true;
                            alpha[q][x] = ex2_approx(m[q][x] - (mx - Lazy<FP8>::kTop));
                            m[q][x] = mx - Lazy<FP8>::kTop;
                        }
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int q = 0; q < NR; ++q) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            l[q][x] *= alpha[q][x];
                            lh[q][x] *= alpha[q][x];
                        }
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[q][i][e] *= alpha[q][e & 1];
                    }
                }
                // ---- weights, their sums, and P^T as B fragments (the 8 x 8 tiles of
                // keys x rows transposed across the warp)
                uint32_t pf[NR][2][2];
#pragma unroll
                for (int q = 0; q < NR; ++q) {
                    const float m0 = m[q][0] == -INFINITY ? 0.f : m[q][0], m1 = m[q][1] == -INFINITY ? 0.f : m[q][1];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float w0 = ex2_approx(t[q][i][2 * y] - m0), w1 = ex2_approx(t[q][i][2 * y + 1] - m1);
                            uint32_t pk;
                            if constexpr (FP8) {
                                // the sum takes the unrounded weights: a small row of V may
                                // carry a weight too small for f16 that still counts in l
                                pk = pack_f16x2(w0, w1);
                                l[q][0] = fmaf(w0, vinv[i][y], l[q][0]);
                                l[q][1] = fmaf(w1, vinv[i][y], l[q][1]);
                            } else {
                                pk = pack_bf16x2(w0, w1);
                                l[q][0] += w0;
                                l[q][1] += w1;
                                lh[q][0] += __uint_as_float(pk << 16);
                                lh[q][1] += __uint_as_float(pk & 0xffff0000u);
                            }
                            pf[q][i][y] = transpose8x8(pk);
                        }
                }
                // ---- O^T += V^T P^T
                if constexpr (!FP8) {
                    // 8 x 8 tiles of V (keys x columns), transposed on the way: keys 0-7 and
                    // 8-15 of columns 0-7 and 8-15 in the order of an A fragment
                    const int kr = ((lane >> 4) << 3) + (lane & 7);
                    const uint32_t ch = (lane >> 3) & 1, sw = lane & 7;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const uint32_t b = vs_ + key_off(sub + kr + 16 * kk);
#pragma unroll
                        for (int nb = 0; nb < D / 16; nb += 4) {
                            uint32_t f[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                ldsm4t(f[i], b + (nb >> 2) * (pr * 128) + (((2 * i + ch) ^ sw) << 4));
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) f[i][e] &= dead[2 * kk + (e >> 1)];
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int q = 0; q < NR; ++q) mma16816<false>(o[q][nb + i], f[i], pf[q][kk][0], pf[q][kk][1]);
                        }
                    }
                } else {
                    // this lane takes columns (D/8) gr .. + D/8 - 1, two per product: bytes of
                    // the four keys of its k indices, paired by key
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t x[4][D / 32];           // keys 2c, 2c+1, 2c+8, 2c+9
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = sub + 16 * kk + 2 * c4 + (k & 1) + 8 * (k >> 1);
                            if constexpr (D == 128) {
                                const uint4 v = lds128(vs_ + r * D + ((gr ^ (r & 7)) << 4));
                                x[k][0] = v.x;
                                x[k][1] = v.y;
                                x[k][2] = v.z;
                                x[k][3] = v.w;
                            } else {
                                const uint2 v = lds64(vs_ + r * D + (((gr >> 1) ^ ((r >> 1) & 3)) << 4) + 8 * (gr & 1));
                                x[k][0] = v.x;
                                x[k][1] = v.y;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t f[2][4];            // [column pair][fragment register]
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                widen4(__byte_perm(x[2 * k][i], x[2 * k + 1][i], 0x5140), f[0][2 * k], f[0][2 * k + 1]);
                                widen4(__byte_perm(x[2 * k][i], x[2 * k + 1][i], 0x7362), f[1][2 * k], f[1][2 * k + 1]);
                            }
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    f[0][e] &= dead[2 * kk + (e >> 1)];
                                    f[1][e] &= dead[2 * kk + (e >> 1)];
                                }
                            }
#pragma unroll
                            for (int b = 0; b < 2; ++b)
#pragma unroll
                                for (int q = 0; q < NR; ++q)
                                    mma16816<true>(o[q][2 * i + b], f[b], pf[q][kk][0], pf[q][kk][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * s);
        }

        // ---- join the groups through shared memory and write the rows
        if (!idle) {
            float* mw = merge + warp * kWarpRows * C::kPitch;
#pragma unroll
            for (int q = 0; q < NR; ++q)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float ls = keys_sum(l[q][x]), lhs = FP8 ? ls : keys_sum(lh[q][x]);
                    const int r = 8 * q + 2 * c4 + x;
                    if (rbase + r < sg.r1) {
                        if (gr == 0) {
                            stats[(warp * kWarpRows + r) * 3] = m[q][x];
                            stats[(warp * kWarpRows + r) * 3 + 1] = ls;
                            stats[(warp * kWarpRows + r) * 3 + 2] = lhs;
                        }
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            float* w = mw + r * C::kPitch;
                            if constexpr (FP8) {
                                *reinterpret_cast<float2*>(w + (D / 8) * gr + 2 * i) = make_float2(o[q][i][x], o[q][i][x + 2]);
                            } else {
                                w[16 * i + gr] = o[q][i][x];
                                w[16 * i + gr + 8] = o[q][i][x + 2];
                            }
                        }
                    }
                }
        }
        named_barrier_sync(1, 32 * kConsumers);
        float* slot = slot_at<RT, D>(p, blockIdx.x, sg.slot > 0);
        const int nrows = sg.r1 - sg.r0;
        for (int i = threadIdx.x; i < nrows * (D / 4); i += 32 * kConsumers) {
            const int r = i / (D / 4), col = 4 * (i % (D / 4));
            const int at0 = r;                           // in group 0: warp r / kWarpRows, row r % kWarpRows of it
            float M = -INFINITY;
#pragma unroll
            for (int gI = 0; gI < kConsumers / MT; ++gI) M = fmaxf(M, stats[(at0 + gI * RT) * 3]);
            const float U = M == -INFINITY ? 0.f : M;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f, LH = 0.f;
#pragma unroll
            for (int gI = 0; gI < kConsumers / MT; ++gI) {
                const int at = at0 + gI * RT;
                const float k = ex2_approx(stats[at * 3] - U);
                const float4 v = *reinterpret_cast<const float4*>(merge + at * C::kPitch + col);
                L = fmaf(stats[at * 3 + 1], k, L);
                LH = fmaf(stats[at * 3 + 2], k, LH);
                a.x = fmaf(v.x, k, a.x);
                a.y = fmaf(v.y, k, a.y);
                a.z = fmaf(v.z, k, a.z);
                a.w = fmaf(v.w, k, a.w);
            }
            if (sg.slot < 0) {
                int64_t token;
                int head;
                row_place(p, sg.row0, sg.head, sg.r0 + r, token, head);
                const float inv = LH == 0.f ? 0.f : 1.f / LH;
                uint2 out;
                out.x = pack_bf16x2(a.x * inv, a.y * inv);
                out.y = pack_bf16x2(a.z * inv, a.w * inv);
                *reinterpret_cast<uint2*>(p.o + token * p.o_ts + head * p.o_hs + col) = out;
                if (col == 0) p.lse[token * p.heads_q + head] = unless_aborted(lse_of(M, L), abort);
            } else {
                *reinterpret_cast<float4*>(slot + (col / 4 * RT + r) * 4) = a;
                if (col == 0) {
                    slot[RT * D + r] = M;
                    slot[RT * (D + 1) + r] = unless_aborted(L, abort);
                    slot[RT * (D + 2) + r] = LH;
                }
            }
        }
        gbase += n;
        named_barrier_sync(1, 32 * kConsumers);
        if (lane == 0) mbar_arrive(seg_empty + 8 * (sk & 1));
    }
}

template <int D, bool FP8, int NR, int MT>
int launch(const fa_kv_cache* c, const AttnParams& p, bool join, cudaStream_t s) {
    alignas(64) Maps maps{};
    if (c->prepared) {
        const Prepared* m = static_cast<const Prepared*>(c->prepared);
        memcpy(&maps.k, &m->rows_k, sizeof(CUtensorMap));
        memcpy(&maps.v, &m->rows_v, sizeof(CUtensorMap));
        memcpy(&maps.ke, &m->rows_ke, sizeof(CUtensorMap));
        memcpy(&maps.ve, &m->rows_ve, sizeof(CUtensorMap));
    } else {
        alignas(64) Prepared m;
        if (encode_rows(m, c) != FA_OK) return FA_ERR_CUDA;
        maps.k = m.rows_k;
        maps.v = m.rows_v;
        maps.ke = m.rows_ke;
        maps.ve = m.rows_ve;
    }
    rows_kernel<D, FP8, NR, MT><<<p.ctas, kThreads, Cfg<D, FP8>::kSmemBytes, s>>>(maps, p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    return join ? launch_join<8 * NR * MT, D>(p, s) : FA_OK;
}

template <int D, bool FP8, int NR, int MT>
bool opt_in() {
    return cudaFuncSetAttribute(rows_kernel<D, FP8, NR, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<D, FP8>::kSmemBytes) == cudaSuccess;
}
template <int D, bool FP8>
bool opt_in_all() {
    return opt_in<D, FP8, 1, 1>() && opt_in<D, FP8, 2, 1>() && opt_in<D, FP8, 2, 2>() && opt_in<D, FP8, 2, 4>();
}
template <int D, bool FP8>
int launch_rt(const fa_kv_cache* c, const AttnParams& p, int rows, bool join, cudaStream_t s) {
    switch (rows) {
        case 8: return launch<D, FP8, 1, 1>(c, p, join, s);
        case 16: return launch<D, FP8, 2, 1>(c, p, join, s);
        case 32: return launch<D, FP8, 2, 2>(c, p, join, s);
        default: return launch<D, FP8, 2, 4>(c, p, join, s);
    }
}

}  // namespace

int launch_rows(const fa_kv_cache* c, const AttnParams& p, int rows, bool join, cudaStream_t s) {
    const bool fp8 = c->type == FA_KV_E4M3;
    if (c->d == 128) return fp8 ? launch_rt<128, true>(c, p, rows, join, s) : launch_rt<128, false>(c, p, rows, join, s);
    return fp8 ? launch_rt<64, true>(c, p, rows, join, s) : launch_rt<64, false>(c, p, rows, join, s);
}

int encode_rows(Prepared& m, const fa_kv_cache* c) {
    static_assert(Cfg<128, true>::kUnit == Cfg<64, true>::kUnit && Cfg<64, true>::kUnit == Cfg<64, false>::kUnit, "boxes");
    const int unit = c->type == FA_KV_E4M3 || c->d == 64 ? Cfg<64, false>::kUnit : Cfg<128, false>::kUnit;
    const int rows = static_cast<int>(c->page_size < unit ? c->page_size : unit);
    if (encode_cache(&m.rows_k, c, c->k, rows, false) || encode_cache(&m.rows_v, c, c->v, rows, false)) return FA_ERR_CUDA;
    memset(&m.rows_ke, 0, sizeof(m.rows_ke));
    memset(&m.rows_ve, 0, sizeof(m.rows_ve));
    if (c->type == FA_KV_E4M3 && (encode_exps(&m.rows_ke, c, c->k_exp, rows) || encode_exps(&m.rows_ve, c, c->v_exp, rows)))
        return FA_ERR_CUDA;
    return FA_OK;
}

int rows_setup() {
    return opt_in_all<128, true>() && opt_in_all<128, false>() && opt_in_all<64, true>() && opt_in_all<64, false>()
               ? FA_OK
               : FA_ERR_CUDA;
}

}  // namespace paged
}  // namespace fa
