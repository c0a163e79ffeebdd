// Shared parts of the paged key/value cache operators: the batch as the
// kernels see it (every value read on the device is clamped before use, so no
// input can lead outside the given arrays), and the host-side checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/fa.h"
#include "host_common.h"
#include "ptx.cuh"

namespace fa {
namespace paged {

struct Batch {
    const int32_t* __restrict__ cu;
    const int32_t* __restrict__ kv_len;
    const int32_t* __restrict__ table;
    int64_t table_stride;
    int seqs, tokens, table_width, page_log2, pages;
};

// One sequence: its first packed row, number of rows, cached tokens.
struct Seq {
    int row0, n, kv;
};

__device__ __forceinline__ Seq load_seq(const Batch& b, int s) {
    const int a = min(max(__ldg(b.cu + s), 0), b.tokens);
    const int e = min(max(__ldg(b.cu + s + 1), a), b.tokens);
    return Seq{a, e - a, max(__ldg(b.kv_len + s), 0)};
}

// Positions the page table covers.
__device__ __forceinline__ int table_capacity(const Batch& b) { return b.table_width << b.page_log2; }

__device__ __forceinline__ void report_page(int* status) {
    if (status) atomicExch(status, FA_ERR_PAGE);
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

struct DeviceState {
    std::once_flag once;
    int status = FA_OK;
    int sms = 0;
};
// The current device's number of SMs, and what became of its check (compute capability 10.0: the code is
// sm_100a) and of `setup`, both made once.
template <class Setup>
inline int device_ready(DeviceState (&states)[kMaxDevices], int& sms, Setup setup) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    DeviceState& st = states[dev];
    std::call_once(st.once, [&] {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            st.status = FA_ERR_CUDA;
        else if (major != 10 || minor != 0)
            st.status = FA_ERR_ARCH;
        else
            st.status = setup();
    });
    sms = st.sms;
    return st.status;
}

inline int check_cache_sizes(const fa_kv_cache* c) {
    if (c->pages < 1 || c->pages > 0x7fffffffLL || c->heads < 1 || c->heads > 65535) return FA_ERR_SHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
        c->page_size != 256)
        return FA_ERR_SHAPE;
    return FA_OK;
}
inline int check_cache_kind(const fa_kv_cache* c) {
    if (c->d != 64 && c->d != 128) return FA_ERR_HEADDIM;
    return c->type == FA_KV_BF16 || c->type == FA_KV_E4M3 ? FA_OK : FA_ERR_ARG;
}

// Checks of the cache and the batch up to "empty": 0 to go on, 1 when there is
// nothing to do, else a status.
inline int check_sizes(const fa_kv_cache* c, const fa_kv_batch* b) {
    if (!c || !b) return FA_ERR_NULL;
    int rc = check_cache_sizes(c);
    if (rc != FA_OK) return rc;
    if (b->seqs < 0 || b->seqs > (1 << 20) || b->tokens < 0 || b->tokens > (int64_t(1) << 30) ||
        b->table_width < 0 || b->max_new < 0 || b->table_width > (int64_t(1) << 30) / c->page_size ||
        b->table_width * c->page_size > (int64_t(1) << 36) / c->heads)
        return FA_ERR_SHAPE;
    if ((rc = check_cache_kind(c)) != FA_OK) return rc;
    return (b->tokens == 0 || b->seqs == 0) ? 1 : 0;
}

inline bool stride_ok(int64_t stride, int64_t item, int64_t extent) {
    return extent <= 1 || (stride > 0 && stride < (int64_t(1) << 39) / item && (stride * item) % 16 == 0);
}

inline int check_cache_pointers(const fa_kv_cache* c) {
    return c->k && c->v && (c->type != FA_KV_E4M3 || (c->k_exp && c->v_exp)) ? FA_OK : FA_ERR_NULL;
}
inline int check_pointers(const fa_kv_cache* c, const fa_kv_batch* b) {
    if (!b->cu || !b->kv_len || (b->table_width > 0 && !b->table)) return FA_ERR_NULL;
    return check_cache_pointers(c);
}

inline int check_cache_alignment(const fa_kv_cache* c) {
    using host::aligned;
    const int64_t item = c->type == FA_KV_BF16 ? 2 : 1;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_ALIGN;
    if (c->type == FA_KV_E4M3 && (!aligned(c->k_exp, 16) || !aligned(c->v_exp, 16))) return FA_ERR_ALIGN;
    if (!stride_ok(c->page_stride, item, c->pages) || !stride_ok(c->head_stride, item, c->heads) ||
        !stride_ok(c->row_stride, item, c->page_size))
        return FA_ERR_ALIGN;
    return FA_OK;
}
inline int check_alignment(const fa_kv_cache* c, const fa_kv_batch* b) {
    using host::aligned;
    if (!aligned(b->cu, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4)) return FA_ERR_ALIGN;
    if (b->table_stride < b->table_width && b->seqs > 1) return FA_ERR_ALIGN;
    return check_cache_alignment(c);
}

// Packed tensors: token and head strides in elements of a 16-bit type.
inline bool packed_ok(const void* p, int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads) {
    return host::aligned(p, 16) && stride_ok(token_stride, 2, tokens) && stride_ok(head_stride, 2, heads);
}

inline Batch device_batch(const fa_kv_cache* c, const fa_kv_batch* b) {
    Batch d;
    d.cu = b->cu;
    d.kv_len = b->kv_len;
    d.table = b->table;
    d.table_stride = b->table_stride;
    d.seqs = static_cast<int>(b->seqs);
    d.tokens = static_cast<int>(b->tokens);
    d.table_width = static_cast<int>(b->table_width);
    d.pages = static_cast<int>(c->pages);
    d.page_log2 = 0;
    while ((int64_t(1) << d.page_log2) < c->page_size) ++d.page_log2;
    return d;
}

}  // namespace paged
}  // namespace fa
