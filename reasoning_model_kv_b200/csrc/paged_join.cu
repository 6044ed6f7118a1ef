// paged_join.cu -- joins the partial results of attention items that were cut over blocks.
//
// out = sum_p w_p O_p / sum_p w_p z_p, w_p = 2^(M_p - max M), the parts in block order.  A row
// is joined by WS warps, each every WS-th part, its parts' maxima and sums a lane each, so a
// row's reads are all in flight at once: what bounds it is their latency (eight items of 74
// parts in about 5 us behind the attention kernel, whose end its launch overlaps).  Many parts of few
// rows (single tokens) take WS = 8, few parts of many rows (prompt chunks) one warp a row.
#include "norm_rope.cuh"
#include "paged_attention.cuh"

namespace tkv {
namespace paged {
namespace {

constexpr int kWarps = 8;

template <typename T, int D, int WS>
__global__ void __launch_bounds__(32 * kWarps) join_kernel(const AttnArgs a, int item_rows, int tile_rows) {
    constexpr int kRowsHere = kWarps / WS, E = D / 32;        // rows of a block, elements of a lane
    __shared__ float sm_m[kWarps], sm_z[kWarps], sm_o[kWarps][D];
    attn::grid_dependency_wait();
    const int blk = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CutItem cut = a.cut[blk];
    if (cut.parts < 2) return;
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
