// paged.cuh -- device-side view of a paged 8-bit cache and the launchers of its kernels.
// Internal to libtkv (the C ABI and the data layout are in include/tkv.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tkv.h"
#include "tkv_internal.cuh"

namespace tkv {
namespace paged {

constexpr int kMaxGroup = 16;          // query heads per kv head
constexpr int kMaxLen = 1 << 30;       // tokens of a sequence
constexpr float kLeastScale = 5.421010862427522e-20f;      // 2^-64, the least that the append writes: of zeros
constexpr float kLog2e = 1.4426950408889634f;

struct View {
    int B, Hkv, G, D, page, page_log2, pages, max_pages, code, dtype;
    uint8_t *k_pool, *v_pool;
    float *k_scale, *v_scale;
    uint32_t *err;        // [0] first status, [1] count, [2] detail
};

// A [rows][heads][D] array; strides in elements.
struct Rows {
    const void *p;
    long long token, head;
};

// Detail words of latched errors.
enum : uint32_t {
    kBadRows = 0x501,     // cu decreases or leaves [0, T], or more rows than max_new
    kBadLen = 0x502,      // kv_len below 0, above kMaxLen, or (append) below the sequence's rows
    kBadPage = 0x503,     // page id outside [0, pages)
    kNoPage = 0x504,      // page id -1, or the table's row is too short
    kWaitTimeout = 0x505, // a bounded wait inside a kernel gave up
};

// The rows and length of sequence b: first row, number of rows, tokens in the cache (fewer
// than its rows only in attention calls: its first rows see nothing).  false (and *bad its
// detail) where they cannot be used.
struct Seq {
    int row0, n, len;
};
__device__ __forceinline__ bool load_seq(const int32_t *cu, const int32_t *kv_len, int b, int T, Seq *s,
                                         uint32_t *bad) {
    int r0 = b, r1 = b + 1;
    if (cu) { r0 = cu[b]; r1 = cu[b + 1]; }
    s->row0 = r0;
    s->n = r1 - r0;
    s->len = kv_len[b];
    if (r0 < 0 || r1 < r0 || r1 > T) { *bad = kBadRows; return false; }
    if (s->len < 0 || s->len > kMaxLen) { *bad = kBadLen; return false; }
    return true;
}

// Page id of block i of sequence b; -1 where there is none to use, with *bad its detail.
__device__ __forceinline__ int load_page(const View &c, const int32_t *block_table, int b, int i, uint32_t *bad) {
    if (i >= c.max_pages) { *bad = kNoPage; return -1; }
    const int id = block_table[(size_t)b * c.max_pages + i];
    if (id >= 0 && id < c.pages) return id;
    *bad = id == -1 ? kNoPage : kBadPage;
    return -1;
}

__device__ __forceinline__ void latch(const View &c, uint32_t bad) {
    raise_error(c.err, bad == kNoPage ? kErrCapacity : kErrInvalid, bad);
}

cudaError_t launch_norm_rope(const tkv_rope &rope, Rows q, Rows k, const int32_t *pos, Rows qo, Rows ko, int T, int Hq,
                             int Hkv, int D, int dtype, cudaStream_t st);
cudaError_t launch_append(const View &c, const tkv_rope &rope, Rows k, Rows v, Rows q, Rows qo, int T,
                          const int32_t *block_table, const int32_t *kv_len, const int32_t *cu, int max_new,
                          cudaStream_t st, int64_t *launches);
cudaError_t launch_attention(const View &c, Rows q, Rows out, int T, const int32_t *block_table,
                             const int32_t *kv_len, const int32_t *cu, int max_q, int window, float scale,
                             cudaStream_t st, int64_t *launches);

}  // namespace paged
}  // namespace tkv
