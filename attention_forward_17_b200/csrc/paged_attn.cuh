// What the two paged attention kernels and their joining pass share: the
// parameters, the list of work, and the partial results.
//
// Work list.  An item is (sequence, row tile, key head).  The rows of an item
// are the query rows that share the key head, token by token and within a token
// the G = heads_q / heads of them, cut into tiles of RT rows.  A unit is one tile of BN
// keys of an item: the tiles that hold visible keys (under a window, those of
// the first `sinks` tokens and then those of the window), at least one per item
// so that rows without keys are written too.  All units, in the order
// (sequence, row tile, head, key tile), are cut into contiguous
// stretches of equal weight, one per CTA.  So every SM gets the same number of key tiles
// whatever the lengths are, nothing about the lengths is needed on the host,
// and a long sequence is split exactly where the machine needs it.  A CTA works
// through its stretch segment by segment (a segment is the part of one item it owns);
// an item with several CTAs leaves one partial result per CTA, which the
// joining kernel adds up in the order of the keys, so results do not depend on
// timing.  A CTA has at most two partial segments, its first and its last: the
// workspace holds two slots per CTA.
#pragma once

#include "paged_common.cuh"
#include "waits.cuh"

namespace fa {
namespace paged {

constexpr int kNoWindow = 0x7fffffff;

struct AttnParams {
    Batch b;
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int64_t q_ts, q_hs, o_ts, o_hs;     // elements
    int heads_q, heads, group;          // group = heads_q / heads
    int window, sinks;                  // window = kNoWindow for none
    float scale_log2;                   // scale * log2(e)
    int min_rows, max_rows;             // this kernel's sequences: min_rows < n * group <= max_rows
    int ctas, min_units, over;          // parts of the work list, the least weight of one, and
                                        // the weight of an item besides its units
    int after_rows;                     // tile kernel: may start while the row kernel of the call still runs
    int q_tma;                          // tile kernel: the group is a power of two up to 128
    int whole;                          // items are not cut: a part takes those that start in it
    uint32_t abandoned;                 // self-test: 1, every CTA starts as if one of its waits had run out of time
    float* ws;
    int* status;
};

// Work list position: units [unit, units) of the item (seq, tile, head).
struct Item {
    Seq q;
    int seq, tile, head;
    int rows;              // n * group: query rows of the sequence per key head
    int r0, r1;            // the item's rows
    int p0;                // position of the sequence's first row
    int pmin, pmax;        // positions of rows r0 and r1 - 1
    int hi, lo, sk;        // some row sees key j iff j < hi and (j >= lo or j < sk)
    int w0, ns, units;     // key tiles 0 .. ns-1 and w0 ..
};

template <int RT, int BN>
struct Sched {
    __device__ static bool mine(const AttnParams& p, const Seq& q) {
        const int64_t rows = static_cast<int64_t>(q.n) * p.group;
        return rows > p.min_rows && rows <= p.max_rows;
    }
    __device__ static int tiles(const AttnParams& p, const Seq& q) { return (q.n * p.group + RT - 1) / RT; }

    // Fills the item's ranges from seq, tile, q.
    __device__ static void ranges(const AttnParams& p, Item& it) {
        it.rows = it.q.n * p.group;
        it.r0 = it.tile * RT;
        it.r1 = min(it.rows, it.r0 + RT);
        it.p0 = it.q.kv - it.q.n;
        it.pmin = it.p0 + it.r0 / p.group;
        it.pmax = it.p0 + (it.r1 - 1) / p.group;
        it.hi = min(max(it.pmax + 1, 0), table_capacity(p.b));
        it.lo = 0;
        if (p.window != kNoWindow) it.lo = min(max(it.pmin - p.window + 1, 0), it.hi);
        it.sk = min(p.sinks, it.lo);
        it.w0 = it.lo / BN;
        it.ns = min((it.sk + BN - 1) / BN, it.w0);
        it.units = max(1, it.ns + (it.hi + BN - 1) / BN - it.w0);
    }
    __device__ static int units(const AttnParams& p, const Seq& q, int tile) {
        Item it;
        it.q = q;
        it.tile = tile;
        ranges(p, it);
        return it.units;
    }
    // The next item after `it` in the list (there is one).
    __device__ static void next(const AttnParams& p, Item& it) {
        if (++it.head < p.heads) return;
        it.head = 0;
        if (++it.tile >= tiles(p, it.q)) {
            it.tile = 0;
            do {
                ++it.seq;
                if (it.seq >= p.b.seqs) {          // past the list: never used
                    it.seq = p.b.seqs - 1;
                    break;
                }
                it.q = load_seq(p.b, it.seq);
            } while (!mine(p, it.q));
        }
        ranges(p, it);
    }
};

// A segment as the warps of a CTA see it: units [unit, unit + n) of one item.
// One warp writes it to shared memory, the others read it there.
struct Segment {
    int n;                   // units; 0 ends the kernel
    int seq, head, unit;
    int row0, p0, r0, r1;
    int hi, lo, sk, w0, ns;
    int slot;                // -1: the whole item; else which of the CTA's two partial results
};

__device__ __forceinline__ void fill_segment(Segment& g, const Item& it, int unit, int n) {
    g.n = n;
    g.seq = it.seq;
    g.head = it.head;
    g.unit = unit;
    g.row0 = it.q.row0;
    g.p0 = it.p0;
    g.r0 = it.r0;
    g.r1 = it.r1;
    g.hi = it.hi;
    g.lo = it.lo;
    g.sk = it.sk;
    g.w0 = it.w0;
    g.ns = it.ns;
    g.slot = unit == 0 && n == it.units ? -1 : unit == 0;
}
// Key tile of the segment's unit u.
__device__ __forceinline__ int key_tile(const Segment& g, int u) {
    const int x = g.unit + u;
    return x < g.ns ? x : g.w0 + (x - g.ns);
}
// Some row of the item sees key j.
__device__ __forceinline__ bool alive(const Segment& g, int j) { return j < g.hi && (j >= g.lo || j < g.sk); }

// ---------------------------------------------------------------- cutting the work list
// Each item weighs its units plus p.over: what starting and ending a segment costs, in
// units, ahead of the units.  Part c owns the weights [c per, (c + 1) per).  Its record, kept
// at the start of the workspace for the joining kernel: the first unit of its own in
// the item it starts in (0: the item is not cut there), and that item.
struct alignas(16) Part {
    int unit, units, head, row0, r0, r1;
    int64_t per;
};
static_assert(sizeof(Part) == 32, "workspace layout");

struct Scratch {
    int64_t weight[16];      // by warp
    int64_t room;
    int seq, tile, head, skip;
};

// Where a part starts: `skip` into the weight of an item; and the weight from that item's
// start to the part's end (0: an empty part).
struct Start {
    int seq, tile, head, skip;
    int64_t room, per;
};

__device__ __forceinline__ int64_t inclusive_sum(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
    }
    return v;
}

// 32 sequences, one a lane, and their row tiles numbered through.
struct Chunk {
    Seq q;
    int tiles, upto;         // row tiles of this sequence (0: past the end, or another kernel's), and up to its end
    int count;               // of all
};
template <class S>
__device__ Chunk load_chunk(const AttnParams& p, int s, int end, int lane) {
    Chunk c{Seq{0, 0, 0}, 0, 0, 0};
    if (s < end) {
        c.q = load_seq(p.b, s);
        if (S::mine(p, c.q)) c.tiles = S::tiles(p, c.q);
    }
    c.upto = c.tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, c.upto, o);
        if (lane >= o) c.upto += a;
    }
    c.count = __shfl_sync(0xffffffffu, c.upto, 31);
    return c;
}
// A row tile of a chunk: the lane of its sequence, its number there, its weight per key head.
struct TileAt {
    int lane_seq, tile, each;
};
// Of the 32 tiles from f0 on, one a lane: the tile, its weight and the weight from f0 to its end.
// Returns the weight of all.
template <class S>
__device__ __forceinline__ int64_t chunk_sums(const AttnParams& p, const Chunk& c, int f0, int lane, TileAt& at, int64_t& own,
                                              int64_t& inc) {
    const int f = f0 + lane;
    int src = 0;                     // the first lane with upto > f
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xffffffffu, c.upto, src + step - 1) <= f) src += step;
    src = min(src, 31);
    const Seq w{0, __shfl_sync(0xffffffffu, c.q.n, src), __shfl_sync(0xffffffffu, c.q.kv, src)};
    const int t = f - __shfl_sync(0xffffffffu, c.upto - c.tiles, src);
    at = TileAt{src, t, f < c.count ? S::units(p, w, t) + p.over : 0};
    own = static_cast<int64_t>(at.each) * p.heads;
    inc = inclusive_sum(own, lane);
    return __shfl_sync(0xffffffffu, inc, 31);
}
// The weight before the tile that holds weight v of the chunk, and that tile; v < 0: the
// weight of the chunk.
template <class S>
__device__ int64_t walk_chunk(const AttnParams& p, const Chunk& c, int64_t v, int lane, TileAt& at) {
    int64_t before = 0;
#pragma unroll 1
    for (int f0 = 0; f0 < c.count; f0 += 32) {
        int64_t own, inc;
        const int64_t sum = chunk_sums<S>(p, c, f0, lane, at, own, inc);
        const unsigned hit = __ballot_sync(0xffffffffu, v >= 0 && v < before + inc);
        if (hit) {
            const int tl = __ffs(hit) - 1;
            at = TileAt{__shfl_sync(0xffffffffu, at.lane_seq, tl), __shfl_sync(0xffffffffu, at.tile, tl),
                        __shfl_sync(0xffffffffu, at.each, tl)};
            return before + __shfl_sync(0xffffffffu, inc - own, tl);
        }
        before += sum;
    }
    return before;
}
// The start of the part that begins `v` into the chunk's weight.
template <class S>
__device__ Start find_in(const AttnParams& p, const Chunk& c, int s0, int64_t v, int lane) {
    TileAt at{0, 0, 1};
    // the rest is below heads * weight of an item: 32 bits
    const unsigned rem = static_cast<unsigned>(v - walk_chunk<S>(p, c, v, lane, at));
    const unsigned each = static_cast<unsigned>(at.each);
    return Start{s0 + at.lane_seq, at.tile, static_cast<int>(rem / each), static_cast<int>(rem % each), 0, 0};
}

__device__ __forceinline__ int64_t weight_per_part(const AttnParams& p, int64_t total) {
    int64_t per = total < 0x7fffffffLL - p.ctas ? static_cast<unsigned>(total + p.ctas - 1) / static_cast<unsigned>(p.ctas)
                                               : (total + p.ctas - 1) / p.ctas;
    return per < p.min_units ? p.min_units : per;
}

// With at most 32 sequences one warp finds its part's start by itself; with more, the
// block's warps (at most 16) look through their shares of them together.
__device__ __forceinline__ bool few_seqs(const AttnParams& p) { return p.b.seqs <= 32; }

template <int RT, int BN>
__device__ Start locate_warp(const AttnParams& p, int cta, int lane) {
    using S = Sched<RT, BN>;
    const Chunk c = load_chunk<S>(p, lane, p.b.seqs, lane);
    Start r{0, 0, 0, 0, 0, 0};
    TileAt at{0, 0, 1};
    // the whole weight, then the part's start: from the same sums when they are of at most 32
    // tiles, else in a second walk
    int64_t own, inc, w;
    const int64_t total = c.count <= 32 ? chunk_sums<S>(p, c, 0, lane, at, own, inc) : walk_chunk<S>(p, c, -1, lane, at);
    const int64_t per = weight_per_part(p, total), v = cta * per;
    if (v < total) {
        if (c.count <= 32) {
            const int tl = __ffs(__ballot_sync(0xffffffffu, v < inc)) - 1;
            at = TileAt{__shfl_sync(0xffffffffu, at.lane_seq, tl), __shfl_sync(0xffffffffu, at.tile, tl),
                        __shfl_sync(0xffffffffu, at.each, tl)};
            w = __shfl_sync(0xffffffffu, inc - own, tl);
        } else {
            w = walk_chunk<S>(p, c, v, lane, at);
        }
        const unsigned rem = static_cast<unsigned>(v - w), each = static_cast<unsigned>(at.each);
        r = Start{at.lane_seq, at.tile, static_cast<int>(rem / each), static_cast<int>(rem % each), 0, 0};
        r.room = r.skip + (total - v < per ? total - v : per);
    }
    r.per = per;
    return r;
}

// The same by the whole block: every thread calls it, and gets the answer.
template <int RT, int BN>
__device__ Start locate_block(const AttnParams& p, int cta, Scratch* sc) {
    using S = Sched<RT, BN>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int share = (p.b.seqs + 32 * warps - 1) / (32 * warps) * 32;
    const int lo = min(warp * share, p.b.seqs), hi = min(lo + share, p.b.seqs);
    int64_t sub = 0;
    TileAt none{0, 0, 1};
    for (int s0 = lo; s0 < hi; s0 += 32) sub += walk_chunk<S>(p, load_chunk<S>(p, s0 + lane, hi, lane), -1, lane, none);
    if (lane == 0) sc->weight[warp] = sub;
    if (threadIdx.x == 0) {
        sc->seq = sc->tile = sc->head = sc->skip = 0;
        sc->room = 0;
    }
    __syncthreads();
    int64_t total = 0, base = 0;
    for (int w = 0; w < warps; ++w) {
        if (w == warp) base = total;
        total += sc->weight[w];
    }
    const int64_t per = weight_per_part(p, total), v = cta * per;
    if (v >= base && v < base + sub) {
        for (int s0 = lo; s0 < hi; s0 += 32) {
            const Chunk c = load_chunk<S>(p, s0 + lane, hi, lane);
            const int64_t sum = walk_chunk<S>(p, c, -1, lane, none);
            if (v < base + sum) {
                const Start r = find_in<S>(p, c, s0, v - base, lane);
                if (lane == 0) {
                    sc->seq = r.seq;
                    sc->tile = r.tile;
                    sc->head = r.head;
                    sc->skip = r.skip;
                    sc->room = r.skip + (total - v < per ? total - v : per);
                }
                break;
            }
            base += sum;
        }
    }
    __syncthreads();
    return Start{sc->seq, sc->tile, sc->head, sc->skip, sc->room, per};
}

// Walks a part's segments (one warp of the block), after leaving the part's record.
template <int RT, int BN>
struct Walk {
    using S = Sched<RT, BN>;
    Item it;
    int skip;
    int64_t room;
    __device__ void begin(const AttnParams& p, const Start& r) {
        skip = r.skip;
        room = r.room;
        it.seq = r.seq;
        it.tile = r.tile;
        it.head = r.head;
        it.q = load_seq(p.b, r.seq);
        Part part{0, 0, 0, 0, 0, 0, r.per};
        if (room > 0) {
            S::ranges(p, it);
            part = Part{max(skip - p.over, 0), it.units, it.head, it.q.row0, it.r0, it.r1, r.per};
        }
        if ((threadIdx.x & 31) == 0) reinterpret_cast<Part*>(p.ws)[blockIdx.x] = part;
    }
    // The next segment with units: true and `it`, its first unit and their number.  A row whose
    // own position the page table does not reach is reported.
    __device__ bool segment(const AttnParams& p, int& unit, int& n) {
        const bool more = advance(p, unit, n);
        if (more && it.pmax >= table_capacity(p.b)) report_page(p.status);
        return more;
    }
    __device__ bool advance(const AttnParams& p, int& unit, int& n) {
        if (p.whole && skip > 0) next(p);
        while (room > 0) {
            if (p.whole) {
                unit = 0;
                n = it.units;
                return true;
            }
            unit = max(skip - p.over, 0);
            const int64_t most = room - p.over;
            n = static_cast<int>(most < it.units ? most : it.units) - unit;
            if (n > 0) return true;
            next(p);
        }
        n = 0;
        return false;
    }
    // On to the item after `it`.
    __device__ void next(const AttnParams& p) {
        room -= it.units + p.over;
        skip = 0;
        if (room > 0) S::next(p, it);
    }
};

// ---------------------------------------------------------------- partial results
// A slot: O [D / 4][RT][4] (not normalised, relative to m; neighbouring rows side by side,
// so that a thread that owns a row writes whole lines with its warp), then m, l, lh [RT] each:
// the running maximum (base 2), the sum of the weights, and the sum of the
// weights as rounded for the product with V (which normalises O, so a constant
// V of a bf16 cache comes back as that constant; for e4m3, lh = l).
template <int RT, int D>
__host__ __device__ constexpr int64_t slot_floats() {
    return static_cast<int64_t>(RT) * (D + 3);
}
template <int RT, int D>
__device__ __forceinline__ float* slot_at(const AttnParams& p, int64_t cta, int second) {
    return p.ws + p.ctas * (sizeof(Part) / 4) + (2 * cta + second) * slot_floats<RT, D>();
}
inline int64_t workspace_of(int64_t rt, int64_t d, int64_t ctas) {
    return ctas * static_cast<int64_t>(sizeof(Part)) + 2 * ctas * rt * (d + 3) * 4;
}

// One row's place in the packed tensors: row r of the sequence that starts at packed row
// row0, key head `khead`.
__device__ __forceinline__ void row_place(const AttnParams& p, int row0, int khead, int r, int64_t& token, int& head) {
    const int t = r / p.group;
    token = row0 + t;
    head = khead * p.group + (r - t * p.group);
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + lg2_approx(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// Early launches.  Every kernel of a call lets the next one start at once; what the next one
// needs of the previous ones' results it reads after waiting for their end.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the partial results of the items that span several parts.  Block (x, y): the item that
// part x + 1 starts inside of, if it starts in part x; rows R y .. R y + R - 1 of it.  A thread has
// eight columns of a row at a time.  Launched while the main kernel still runs; it waits for it here.
constexpr int kJoinThreads = 256;
template <int RT, int D>
__device__ __forceinline__ void join_rows(const AttnParams& p, int y) {
    constexpr int R = RT < 32 ? RT : 32;
    const int rt = R * y + threadIdx.x % R;
    const int cta = static_cast<int>(blockIdx.x) + 1, before = cta - 1;
    const Part me = reinterpret_cast<const Part*>(p.ws)[cta];
    if (me.unit == 0) return;                                          // no cut inside an item
    // weight at which the item's units start
    const int64_t first = cta * me.per - me.unit;
    if (before * me.per > first) return;                               // it starts earlier: another block's
    const int r = me.r0 + rt;
    if (r >= me.r1) return;
    const int last = static_cast<int>((first + me.units - 1) / me.per);
    int64_t token;
    int head;
    row_place(p, me.row0, me.head, r, token, head);
    for (int c8 = threadIdx.x / R; c8 < D / 8; c8 += kJoinThreads / R) {
        float m = -INFINITY, l = 0.f, lh = 0.f, acc[8] = {};
        for (int c0 = before; c0 <= last; c0 += 4) {                   // four parts in flight
            float pm[4], pl[4], ph[4];
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pm[i] = -INFINITY;
                pl[i] = ph[i] = 0.f;
                a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + i <= last) {
                    const float* s = slot_at<RT, D>(p, c0 + i, c0 + i == before);
                    pm[i] = s[RT * D + rt];
                    pl[i] = s[RT * (D + 1) + rt];
                    ph[i] = s[RT * (D + 2) + rt];
                    a[i] = *reinterpret_cast<const float4*>(s + ((2 * c8) * RT + rt) * 4);
                    b[i] = *reinterpret_cast<const float4*>(s + ((2 * c8 + 1) * RT + rt) * 4);
                }
            }
            const float mn = fmaxf(m, fmaxf(max3f(pm[0], pm[1], pm[2]), pm[3]));
            const float u = mn == -INFINITY ? 0.f : mn, k = ex2_approx(m - u);
            m = mn;
            l *= k;
            lh *= k;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= k;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ex2_approx(pm[i] - u);
                l = fmaf(pl[i], w, l);
                lh = fmaf(ph[i], w, lh);
                acc[0] = fmaf(a[i].x, w, acc[0]);
                acc[1] = fmaf(a[i].y, w, acc[1]);
                acc[2] = fmaf(a[i].z, w, acc[2]);
                acc[3] = fmaf(a[i].w, w, acc[3]);
                acc[4] = fmaf(b[i].x, w, acc[4]);
                acc[5] = fmaf(b[i].y, w, acc[5]);
                acc[6] = fmaf(b[i].z, w, acc[6]);
                acc[7] = fmaf(b[i].w, w, acc[7]);
            }
        }
        const float inv = lh == 0.f ? 0.f : 1.f / lh;
        uint4 o;
        o.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        o.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
        o.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
        o.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(p.o + token * p.o_ts + head * p.o_hs + 8 * c8) = o;
        if (c8 == 0) p.lse[token * p.heads_q + head] = lse_of(m, l);
    }
}

template <int RT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnParams p) {
    let_next_start();
    wait_for_previous();
    join_rows<RT, D>(p, blockIdx.y);
}
// For a call of both kernels, after both: a join between them would take the registers that the
// tile kernel needs to start beside the row kernel.
template <int RT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_both_kernel(const AttnParams rows, const AttnParams tiles) {
    constexpr int kRowBlocks = RT < 32 ? 1 : RT / 32;
    let_next_start();
    wait_for_previous();
    if (blockIdx.y < kRowBlocks)
        join_rows<RT, D>(rows, blockIdx.y);
    else
        join_rows<256, D>(tiles, blockIdx.y - kRowBlocks);
}

// A launch that may start while the previous kernel of the stream still runs.
template <class... Args, class... Given>
inline int launch_early(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t s, const Given&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
template <int RT, int D>
inline int launch_join(const AttnParams& p, cudaStream_t s) {
    if (p.ctas < 2 || p.whole) return FA_OK;
    constexpr int R = RT < 32 ? RT : 32;
    return launch_early(join_kernel<RT, D>, dim3(p.ctas - 1, RT / R), kJoinThreads, 0, s, p);
}

template <int RT, int D>
inline int launch_join_both(const AttnParams& rows, const AttnParams& tiles, cudaStream_t s) {
    if (tiles.ctas < 2) return FA_OK;
    return launch_early(join_both_kernel<RT, D>, dim3(tiles.ctas - 1, (RT < 32 ? 1 : RT / 32) + 256 / 32), kJoinThreads, 0, s,
                        rows, tiles);
}

// ---------------------------------------------------------------- bounded waits
// For a single thread.
__device__ __forceinline__ void wait_one(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int* status) {
    if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, abort, status, kWaitLimitNs, kWaitLimitAbortNs);
}
// For a whole warp.  Lanes may see the phase complete at different polls; they
// meet again before the warp-collective instructions (ldmatrix, mma, tcgen05)
// that follow a wait.
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int* status) {
    if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, abort, status, kWaitLimitNs, kWaitLimitAbortNs);
    __syncwarp();
}

// What a row gets in place of its logarithm or sum when a wait of its CTA ran out of time.
__device__ __forceinline__ float unless_aborted(float x, const volatile uint32_t* abort) {
    return *abort ? __int_as_float(0x7fc00000) : x;
}

// ---------------------------------------------------------------- TMA over the pages
// Cache tensor maps.  bf16 at d = 128: [pages][heads][2 halves of 64][page rows][64];
// otherwise [pages][heads][page rows][d].  A box is `rows` rows of one page and head.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

struct Maps {
    CUtensorMap k, v, ke, ve, q;
};

// Map of one cache tensor with boxes of `rows` rows: of all d columns (two
// halves for bf16 at d = 128), or with `one_half` of 64 bf16 columns.
int encode_cache(CUtensorMap* map, const fa_kv_cache* c, const void* ptr, int rows, bool one_half);
// Map of one scale tensor, boxes of `rows` scales.
int encode_exps(CUtensorMap* map, const fa_kv_cache* c, const void* ptr, int rows);
// The maps of both kernels, as fa_kv_prepare keeps them.
struct Prepared {
    CUtensorMap rows_k, rows_v, rows_ke, rows_ve;    // boxes of a unit of the row kernel
    CUtensorMap k, v, ke, ve;                        // of the tile kernel
};
static_assert(sizeof(Prepared) == FA_KV_PREPARED_BYTES, "size in the header");
int encode_rows(Prepared& m, const fa_kv_cache* c);
int encode_tiles(Prepared& m, const fa_kv_cache* c);
// Map of the packed queries, boxes of 64 columns of the heads of a group and 128 / group tokens.
int encode_q(CUtensorMap* map, const AttnParams& p, int64_t d);

// Kernel entry points (host).  rows: 8, 16, 32 or 64 query rows per item.
int launch_rows(const fa_kv_cache* c, const AttnParams& p, int rows, bool join, cudaStream_t s);
int rows_setup();
// beside: the row kernel's parameters if the call runs it too and its parts are still to be joined.
int launch_tiles(const fa_kv_cache* c, const AttnParams& p, const AttnParams* beside, int rows, cudaStream_t s);
int tiles_setup();
constexpr int kTileRows = 256;        // query rows per item of the tile kernel

}  // namespace paged
}  // namespace fa
