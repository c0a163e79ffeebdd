// Host side of the paged attention: argument checks, tensor maps, choice of
// kernels, workspace.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

int encode_cache(CUtensorMap* map, const fa_kv_cache* c, const void* ptr, int rows, bool one_half) {
    auto enc = host::tensor_map_encoder();
    if (!enc) return FA_ERR_CUDA;
    const bool fp8 = c->type == FA_KV_E4M3;
    const cuuint64_t item = fp8 ? 1 : 2;
    // the stride of a dimension of one row is never used, but has to be valid
    const auto bytes = [&](int64_t stride, int64_t extent) {
        return extent > 1 ? static_cast<cuuint64_t>(stride) * item : static_cast<cuuint64_t>(c->d) * item;
    };
    const cuuint64_t row = bytes(c->row_stride, c->page_size), head = bytes(c->head_stride, c->heads),
                     page = bytes(c->page_stride, c->pages);
    const cuuint64_t P = static_cast<cuuint64_t>(c->page_size), H = static_cast<cuuint64_t>(c->heads),
                     N = static_cast<cuuint64_t>(c->pages);
    const cuuint32_t R = static_cast<cuuint32_t>(rows);
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    CUresult r;
    if (!fp8 && c->d == 128) {
        const cuuint64_t dims[5] = {64, P, 2, H, N};
        const cuuint64_t strides[4] = {row, 128, head, page};
        const cuuint32_t box[5] = {64, R, one_half ? 1u : 2u, 1, 1};
        r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        const cuuint32_t D = static_cast<cuuint32_t>(c->d);
        const cuuint64_t dims[4] = {D, P, H, N};
        const cuuint64_t strides[3] = {row, head, page};
        const cuuint32_t box[4] = {D, R, 1, 1};
        r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                D * item == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

int encode_exps(CUtensorMap* map, const fa_kv_cache* c, const void* ptr, int rows) {
    auto enc = host::tensor_map_encoder();
    if (!enc) return FA_ERR_CUDA;
    const cuuint64_t P = static_cast<cuuint64_t>(c->page_size), H = static_cast<cuuint64_t>(c->heads);
    const cuuint64_t dims[3] = {P, H, static_cast<cuuint64_t>(c->pages)};
    const cuuint64_t strides[2] = {P, P * H};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(rows), 1, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

int encode_q(CUtensorMap* map, const AttnParams& p, int64_t d) {
    auto enc = host::tensor_map_encoder();
    if (!enc) return FA_ERR_CUDA;
    // the stride of a dimension of one row is never used, but has to be valid
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.heads_q),
                                static_cast<cuuint64_t>(p.b.tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.heads_q > 1 ? p.q_hs : d) * 2,
                                   static_cast<cuuint64_t>(p.b.tokens > 1 ? p.q_ts : d) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

namespace {

DeviceState g_dev[kMaxDevices];

int device_ready(int& sms) {
    return device_ready(g_dev, sms, [] { return rows_setup() == FA_OK ? tiles_setup() : FA_ERR_CUDA; });
}

// Contexts of at most this many keys are not cut by the row kernel: one unit of 32 for each of its 8
// warps, and no second launch.  (At 1,024 keys the call itself is 4 us shorter, but 8 items on 8 SMs
// take 15.4 us where 128 keys to an SM and a join take 10.4.)
constexpr int64_t kWholeKeys = 256;

// The row kernel alone takes sequences of up to this many query rows per key head.  Row kernel
// and tile kernel in us, 8 key heads, d = 64 bf16 and e4m3, d = 128 bf16 and e4m3: 16 sequences over 4,096, 32 rows:
// 38, 62; 42, 63; 57, 72; 65, 81.  4 over 2,000, 48 rows: 17, 22; 18, 23; 24, 28; 27, 28.  16 over 4,096, 64 rows:
// 65, 61; 73, 63; 90, 73; 115, 81.
constexpr int64_t kRowLimit = 48;

struct Plan {
    int rows;         // the row kernel's rows per item, 0: it does not run
    bool tiles;       // the tile kernel runs, for the sequences with more rows
};

int row_tile(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// From the sizes known on the host (the lengths are on the device).  The row
// kernel takes the smallest tile that holds the longest sequence's rows.  When
// some sequence may have more than kRowLimit rows, single tokens go to the row
// kernel and all others to the tile kernel, or all when there is only one sequence.
// (So a sequence of a few tokens takes the tile kernel when another one of the batch has a chunk, and the row
// kernel otherwise.  A 700-token chunk among 16 sequences over 4,096, d = 128, bf16 and e4m3: 108 and 98 us with
// one token each, 117 and 130 with four.  A row kernel for them beside the chunk was not tried.)
Plan make_plan(const fa_kv_batch* b, int64_t group) {
    const int64_t n = b->max_new < b->tokens ? b->max_new : b->tokens;
    const int64_t rows = n * group;
    if (rows <= kRowLimit) return Plan{row_tile(rows), false};
    return Plan{b->seqs == 1 || group > kRowLimit ? 0 : row_tile(group), true};
}

int check_heads(const fa_kv_cache* c, const fa_kv_batch* b, int64_t heads_q) {
    if (heads_q < 1 || heads_q % c->heads != 0 || heads_q > (int64_t(1) << 23)) return FA_ERR_SHAPE;
    if (b->tokens * (heads_q / c->heads) > 0x7fffffffLL - 1023) return FA_ERR_SHAPE;
    return FA_OK;
}

int64_t workspace_bytes_for(const fa_kv_cache* c, const fa_kv_batch* b, int64_t heads_q, int sms) {
    const Plan plan = make_plan(b, heads_q / c->heads);
    const int64_t a = plan.rows ? workspace_of(plan.rows, c->d, sms) : 0;
    const int64_t t = plan.tiles ? workspace_of(kTileRows, c->d, sms) : 0;
    return (a + 15) / 16 * 16 + t;           // the kernels may run at the same time
}

int attend(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* o, int64_t o_token_stride,
           int64_t o_head_stride, float* lse, int64_t heads_q, const fa_kv_cache* cache, const fa_kv_batch* batch,
           int64_t window, int64_t sinks, float scale, void* workspace, int64_t workspace_bytes, int* dev_status,
           uint32_t abandoned, void* stream) {
    using host::aligned;
    const int empty = check_sizes(cache, batch);
    if (empty < 0) return empty;
    int rc = check_heads(cache, batch, heads_q);
    if (rc != FA_OK) return rc;
    if (window < 0 || window > (int64_t(1) << 30) || sinks < 0 || sinks > (int64_t(1) << 30)) return FA_ERR_SHAPE;
    if (empty) return FA_OK;
    if ((rc = check_pointers(cache, batch)) != FA_OK) return rc;
    if (!q || !o || !lse || !workspace) return FA_ERR_NULL;
    if ((rc = check_alignment(cache, batch)) != FA_OK) return rc;
    if (!packed_ok(q, q_token_stride, q_head_stride, batch->tokens, heads_q) ||
        !packed_ok(o, o_token_stride, o_head_stride, batch->tokens, heads_q) || !aligned(lse, 4) ||
        !aligned(workspace, 16) || !aligned(dev_status, 4))
        return FA_ERR_ALIGN;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
    int sms = 0;
    if ((rc = device_ready(sms)) != FA_OK) return rc;
    if (workspace_bytes < workspace_bytes_for(cache, batch, heads_q, sms)) return FA_ERR_SHAPE;
    AttnParams p;
    p.b = device_batch(cache, batch);
    p.q = static_cast<const uint16_t*>(q);
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.o_ts = o_token_stride;
    p.o_hs = o_head_stride;
    p.heads_q = static_cast<int>(heads_q);
    p.heads = static_cast<int>(cache->heads);
    p.group = static_cast<int>(heads_q / cache->heads);
    p.window = window == 0 ? kNoWindow : static_cast<int>(window);
    p.sinks = window == 0 ? 0 : static_cast<int>(sinks);
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.ctas = sms;
    p.whole = 0;
    p.after_rows = 0;
    p.abandoned = abandoned;
    p.q_tma = p.group <= 128 && (p.group & (p.group - 1)) == 0;
    p.ws = static_cast<float*>(workspace);
    p.status = dev_status;
    const Plan plan = make_plan(batch, p.group);
    AttnParams beside;
    bool join_later = false;
    if (plan.rows) {
        p.min_rows = 0;
        p.max_rows = plan.tiles ? plan.rows : 0x7fffffff;
        p.min_units = 4;         // (one token over 1,000, d = 64: 10.6 us at 8, 8.9 at 4, 8.7 at 2)
        // in units: what starting and ending a segment costs beside its loads (64 tokens over 269,572
        // cached e4m3, 512 items: 113 us at 5 units, 102 at 8, 103 at 12, 105 at 16)
        p.over = 8;
        // short contexts (by the page table's width): whole items, and no second kernel
        p.whole = batch->table_width * cache->page_size <= kWholeKeys;
        join_later = plan.tiles && !p.whole;
        beside = p;
        if ((rc = launch_rows(cache, p, plan.rows, !join_later, static_cast<cudaStream_t>(stream))) != FA_OK) return rc;
    }
    if (plan.tiles) {
        // The row kernel started after everything earlier on the stream, so this one may start as
        // soon as SMs are free; its parts have a workspace of their own.
        p.after_rows = plan.rows != 0;
        if (plan.rows) p.ws += (workspace_of(plan.rows, cache->d, sms) + 15) / 16 * 4;
        p.min_rows = plan.rows;
        p.max_rows = 0x7fffffff;
        p.min_units = 2;
        // (chunks of 4 sequences over 31,477 cached e4m3: 621 us at 2 units, 604 at 3, 594 at 4;
        // 2,048 rows under a window: 109, 110, 113)
        p.over = 3;
        p.whole = 0;
        if ((rc = launch_tiles(cache, p, join_later ? &beside : nullptr, plan.rows, static_cast<cudaStream_t>(stream))) != FA_OK)
            return rc;
    }
    return FA_OK;
}

}  // namespace
}  // namespace paged
}  // namespace fa

extern "C" int fa_kv_prepare(const fa_kv_cache* cache, void* out) {
    using namespace fa::paged;
    if (!cache) return FA_ERR_NULL;
    int rc = check_cache_sizes(cache);
    if (rc != FA_OK || (rc = check_cache_kind(cache)) != FA_OK) return rc;
    if (!out || (rc = check_cache_pointers(cache)) != FA_OK) return FA_ERR_NULL;
    if ((rc = check_cache_alignment(cache)) != FA_OK) return rc;
    alignas(64) Prepared m;
    if (encode_rows(m, cache) != FA_OK || encode_tiles(m, cache) != FA_OK) return FA_ERR_CUDA;
    memcpy(out, &m, sizeof(m));
    return FA_OK;
}

extern "C" int64_t fa_paged_attn_workspace(const fa_kv_cache* cache, const fa_kv_batch* batch, int64_t heads_q) {
    using namespace fa::paged;
    int rc = check_sizes(cache, batch);
    if (rc < 0) return rc;
    int rc2 = check_heads(cache, batch, heads_q);
    if (rc2 != FA_OK) return rc2;
    if (rc == 1) return 0;
    int sms = 0;
    if ((rc = device_ready(sms)) != FA_OK) return rc;
    return workspace_bytes_for(cache, batch, heads_q, sms);
}

extern "C" int fa_paged_attn(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* o,
                             int64_t o_token_stride, int64_t o_head_stride, float* lse, int64_t heads_q,
                             const fa_kv_cache* cache, const fa_kv_batch* batch, int64_t window, int64_t sinks,
                             float scale, void* workspace, int64_t workspace_bytes, int* dev_status,
                             void* stream) {
    using namespace fa::paged;
    return attend(q, q_token_stride, q_head_stride, o, o_token_stride, o_head_stride, lse, heads_q, cache, batch, window, sinks,
                  scale, workspace, workspace_bytes, dev_status, 0, stream);
}

extern "C" int fa_selftest_paged_attn_abandoned(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* o,
                                                int64_t o_token_stride, int64_t o_head_stride, float* lse, int64_t heads_q,
                                                const fa_kv_cache* cache, const fa_kv_batch* batch, int64_t window,
                                                int64_t sinks, float scale, void* workspace, int64_t workspace_bytes,
                                                int* dev_status, void* stream) {
    return fa::paged::attend(q, q_token_stride, q_head_stride, o, o_token_stride, o_head_stride, lse, heads_q, cache, batch,
                             window, sinks, scale, workspace, workspace_bytes, dev_status, 1, stream);
}
