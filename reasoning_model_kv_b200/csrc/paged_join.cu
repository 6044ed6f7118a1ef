// paged_join.cu -- joins the partial results of attention items that were cut over blocks.
//
// out = sum_p w_p O_p / sum_p w_p z_p, w_p = 2^(M_p - max M), the parts in block order.  A row
// is joined by WS warps, each every WS-th part, its parts' maxima and sums a lane each, so a
// row's reads are all in flight at once: what bounds it is their latency (eight items of 74
// parts in about 5 us behind the attention kernel, whose end its launch overlaps).  Many parts of few
// rows (single tokens) take WS = 8, few parts of many rows (prompt chunks) one warp a row.
//
// Behind prompt chunks it also forms the rows that the fp16 weights of the matrix instructions
// cannot (see paged_attention_tiles.cu), which costs calls without any 0.5 us (33 rows on 1000
// keys: 15.3 -> 16.1 us, with the looking for them).
#include <climits>

#include "norm_rope.cuh"
#include "paged_attention.cuh"
#include "paged_codes.cuh"

namespace tkv {
namespace paged {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float4 code_values(int code, uint32_t w) {
    uint32_t lo, hi;
    if (code == TKV_CODE_E4M3) code_pairs<TKV_CODE_E4M3>(w, lo, hi);
    else code_pairs<TKV_CODE_INT8>(w, lo, hi);
    const float2 a = __half22float2(attn::u32_as_h2(lo)), b = __half22float2(attn::u32_as_h2(hi));
    return make_float4(a.x, a.y, b.x, b.y);
}

// One row from the definition, in fp32, by a warp: a key a lane for the logits, D / 32 dims a lane
// for the values; q: the row's query.  Keys that the row does not see are not read.
template <typename T, int D>
__device__ __forceinline__ void plain_row(const AttnArgs &a, int b, int kv_head, int pos, const float *q, T *dst) {
    constexpr int E = D / 32;
    const View &c = a.c;
    const int lane = threadIdx.x & 31, hi = min(pos + 1, a.room), lo = a.window ? max(0, pos - a.window + 1) : 0;
    float M = attn::kNoMax, z = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j0 = lo & ~31; j0 < hi; j0 += 32) {
        const int j = j0 + lane;
        int id = -1;
        uint32_t bad;
        if (j >= lo && j < hi) id = load_page(c, a.block_table, b, j >> c.page_log2, &bad);
        const size_t at = (size_t)max(id, 0) * c.Hkv + kv_head, row = ((at << c.page_log2) + (j & (c.page - 1))) * D;
        float x = -INFINITY, vs = 0.f;
        if (id >= 0) {
            x = 0.f;
#pragma unroll 2
            for (int i = 0; i < D; i += 16) {
                const uint4 u = *reinterpret_cast<const uint4 *>(c.k_pool + row + i);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 v = code_values(c.code, w[k]), y = *reinterpret_cast<const float4 *>(q + i + 4 * k);
                    x = fmaf(v.x, y.x, fmaf(v.y, y.y, fmaf(v.z, y.z, fmaf(v.w, y.w, x))));
                }
            }
            x *= c.k_scale[at] * a.scale_log2;
            vs = c.v_scale[at];
        }
        float top = fmaxf(M, x);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(attn::kFull, top, s));
        const float back = attn::ex2(M - top), p = id >= 0 ? attn::ex2(x - top) : 0.f;
        z = z * back + p;
        M = top;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= back;
        for (uint32_t left = __ballot_sync(attn::kFull, id >= 0); left; left &= left - 1) {
            const int n = __ffs(left) - 1;
            const uint8_t *src = c.v_pool + (((((size_t)__shfl_sync(attn::kFull, id, n) * c.Hkv + kv_head) << c.page_log2) +
                                              ((j0 + n) & (c.page - 1))) * D + E * lane);
            const float pn = __shfl_sync(attn::kFull, p, n), f = __shfl_sync(attn::kFull, vs, n);
            const float4 v = code_values(c.code, E == 4 ? *reinterpret_cast<const uint32_t *>(src)
                                                        : *reinterpret_cast<const uint16_t *>(src));
            o[0] = fmaf(pn, v.x * f, o[0]);
            o[1] = fmaf(pn, v.y * f, o[1]);
            if constexpr (E == 4) {
                o[2] = fmaf(pn, v.z * f, o[2]);
                o[3] = fmaf(pn, v.w * f, o[3]);
            }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(attn::kFull, z, s);
    const float f = z > 0.f || z != z ? 1.f / z : 0.f;
    dst += E * lane;
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(o[0] * f, o[1] * f), pack2<T>(o[2] * f, o[3] * f));
    else *reinterpret_cast<uint32_t *>(dst) = pack2<T>(o[0] * f, o[1] * f);
}

// The rows of the items that begin in this block's stretch of the work, from number `from` on (the
// cut one alone: INT_MAX), a row a warp.  The rows' outputs have not been written, so the queries
// are there even if they lie in the same place.  Slow: two chunks of 2048 rows x 32 heads on 14k and
// 16k keys, all of them marked, take 167 ms (0.9 otherwise).
template <typename T, int D>
__device__ __noinline__ void plain_items(const AttnArgs &a, int from, float (&q)[kWarps][D]) {
    __shared__ Plan plan;
    const View &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * kWarps + warp;
    const int tok = row / c.G, hd = row - tok * c.G;
    long long begin, share;
    make_plan<32 * kWarps, false>(a, plan, kTileUnitLog2, &begin, &share);
    if (begin >= plan.total) return;
    const long long end = min(begin + share, plan.total);
    Cursor k;
    cursor_start(a, plan, begin, kTileUnitLog2, &k);
    int n = 0;
    do {
        int u0, nu;
        cursor_units(k, begin, end, &u0, &nu);
        if (nu == 0) continue;
        if (u0 == 0 && tok < min(a.tile_tokens, k.s.n - k.i0) && (n >= from || item_parts(k, share).count > 1)) {
            const long long at = k.s.row0 + k.i0 + tok;
            const int head = k.h * c.G + hd;
            __syncwarp();
            if (4 * lane < D) {
                const T *src = static_cast<const T *>(a.q.p) + at * a.q.token + (long long)head * a.q.head + 4 * lane;
                const uint2 u = *reinterpret_cast<const uint2 *>(src);
                const float2 x = unpack2<T>(u.x), y = unpack2<T>(u.y);
                *reinterpret_cast<float4 *>(&q[warp][4 * lane]) = make_float4(x.x, x.y, y.x, y.y);
            }
            __syncwarp();
            plain_row<T, D>(a, k.b, k.h, k.r.first + tok, q[warp],
                            static_cast<T *>(const_cast<void *>(a.out.p)) + at * a.out.token + (long long)head * a.out.head);
        }
        ++n;
    } while (cursor_next(a, kTileUnitLog2, end, &k));
}

template <typename T, int D, int WS>
__global__ void __launch_bounds__(32 * kWarps, 5) join_kernel(const __grid_constant__ AttnArgs a, int item_rows, int tile_rows) {
    constexpr int kRowsHere = kWarps / WS, E = D / 32;        // rows of a block, elements of a lane
    __shared__ float sm_m[kWarps], sm_z[kWarps];
    __shared__ __align__(16) float sm_o[kWarps][D];
    attn::grid_dependency_wait();
    const int blk = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CutItem cut = a.cut[blk];
    if (cut.parts < 2 && cut.plain == 0) return;
    bool marked = false;              // the cut item, by one of the other blocks that hold parts: their first
    if constexpr (WS == 1) {          // prompt chunks only
        if (cut.plain != 0) {
            plain_items<T, D>(a, cut.plain - 1, sm_o);
            return;
        }
        for (int p = 1 + lane; p < cut.parts; p += 32) marked |= a.cut[blk + p].plain == 1;
    }
    const int G = a.c.G;
    const int i = blockIdx.y * kRowsHere + warp / WS;            // row of the item's output
    if ((int)blockIdx.y * kRowsHere >= cut.tokens * G) return;
    const bool live = i < cut.tokens * G;
    const int tok = i / G, hd = i - tok * G, per = tile_rows / G;
    const int r = tok / per * tile_rows + (tok % per) * G + hd;
    const size_t stride = (size_t)item_rows * (D + 2);
    auto part = [&](int p) { return part_at(a, stride, blk, blk + p); };
    float M = attn::kNoMax, z = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int p0 = warp % WS; live && p0 < cut.parts; p0 += 32 * WS) {
        const int p = p0 + lane * WS, n = min(32, (cut.parts - p0 + WS - 1) / WS);
        const float m = p < cut.parts ? part(p)[r] : attn::kNoMax;
        const float zz = p < cut.parts ? part(p)[item_rows + r] : 0.f;
        float top = fmaxf(M, m);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float w = attn::ex2(m - top), back = attn::ex2(M - top);
        z = z * back + zz * w;             // a lane's share
        M = top;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= back;
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float *q = part(p0 + j * WS) + 2 * item_rows + (size_t)r * D + E * lane;
            const float wj = __shfl_sync(0xffffffffu, w, j);
            if constexpr (E == 4) {
                const float4 u = *reinterpret_cast<const float4 *>(q);
                o[0] = fmaf(u.x, wj, o[0]); o[1] = fmaf(u.y, wj, o[1]);
                o[2] = fmaf(u.z, wj, o[2]); o[3] = fmaf(u.w, wj, o[3]);
            } else {
                const float2 u = *reinterpret_cast<const float2 *>(q);
                o[0] = fmaf(u.x, wj, o[0]); o[1] = fmaf(u.y, wj, o[1]);
            }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    if constexpr (WS > 1) {
        if (lane == 0) { sm_m[warp] = M; sm_z[warp] = z; }
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][E * lane + e] = o[e];
        __syncthreads();
        if (warp % WS != 0) return;
        float top = M;
        for (int w = 1; w < WS; ++w) top = fmaxf(top, sm_m[warp + w]);
        const float back = attn::ex2(M - top);
        z *= back;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= back;
        for (int w = 1; w < WS; ++w) {
            const float f = attn::ex2(sm_m[warp + w] - top);
            z = fmaf(sm_z[warp + w], f, z);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(sm_o[warp + w][E * lane + e], f, o[e]);
        }
    }
    if constexpr (WS == 1) {
        if (__any_sync(attn::kFull, marked)) {         // all the block's warps
            plain_items<T, D>(a, INT_MAX, sm_o);
            return;
        }
    }
    if (!live) return;
    const float f = z > 0.f || z != z ? 1.f / z : 0.f;
    T *dst = static_cast<T *>(const_cast<void *>(a.out.p)) + (long long)(cut.row0 + tok) * a.out.token +
             (long long)(cut.head0 + hd) * a.out.head + E * lane;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(o[0] * f, o[1] * f), pack2<T>(o[2] * f, o[3] * f));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack2<T>(o[0] * f, o[1] * f);
}

template <typename T, int D, int WS>
cudaError_t run(const AttnArgs &a, int blocks, int item_rows, int tile_rows, cudaStream_t st) {
    // launched while the kernel before it ends; it waits for that kernel's results
    cudaLaunchConfig_t cfg = {};
    constexpr int rows = kWarps / WS;
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)((item_rows + rows - 1) / rows), 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, D, WS>, a, item_rows, tile_rows);
}
template <typename T, int D>
cudaError_t run_rows(const AttnArgs &a, int blocks, int item_rows, int tile_rows, cudaStream_t st) {
    return item_rows <= 32 ? run<T, D, 8>(a, blocks, item_rows, tile_rows, st)
                           : run<T, D, 1>(a, blocks, item_rows, tile_rows, st);
}

}  // namespace

cudaError_t launch_join(const AttnArgs &a, int blocks, int item_rows, int tile_rows, cudaStream_t st) {
    if (a.c.dtype == TKV_DTYPE_BF16)
        return a.c.D == 64 ? run_rows<__nv_bfloat16, 64>(a, blocks, item_rows, tile_rows, st)
                           : run_rows<__nv_bfloat16, 128>(a, blocks, item_rows, tile_rows, st);
    return a.c.D == 64 ? run_rows<__half, 64>(a, blocks, item_rows, tile_rows, st)
                       : run_rows<__half, 128>(a, blocks, item_rows, tile_rows, st);
}

}  // namespace paged
}  // namespace tkv
