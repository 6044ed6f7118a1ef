// paged_join.cu -- joins the partial results of attention items that were cut over blocks.
//
// A warp (half a warp at 64 dims) takes a row: the parts' common maximum, then the sum of
// 2^(M_p - M) times their sums and outputs, in block order.  Bound by reading the parts once.
#include "norm_rope.cuh"
#include "paged_attention.cuh"

namespace tkv {
namespace paged {
namespace {

constexpr int kThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const AttnArgs a, int item_rows, int tile_rows) {
    constexpr int L = D / 4;
    const int blk = blockIdx.x;
    const CutItem cut = a.cut[blk];
    if (cut.parts < 2) return;
    const int G = a.c.G;
    const int i = blockIdx.y * (kThreads / L) + threadIdx.x / L, lane = threadIdx.x % L;     // row of the item's output
    if (i >= cut.tokens * G) return;
    const int tok = i / G, hd = i - tok * G, per = tile_rows / G;
    const int r = tok / per * tile_rows + (tok % per) * G + hd;
    const size_t stride = (size_t)item_rows * (D + 2);
    const float *const first = a.part + (2 * (size_t)blk + cut.second) * stride;
    const float *const rest = a.part + 2 * (size_t)blk * stride;       // part p > 0: + 2 p strides
    auto part = [&](int p) { return p == 0 ? first : rest + 2 * (size_t)p * stride; };
    float M = attn::kNoMax;
    for (int p = 0; p < cut.parts; ++p) M = fmaxf(M, part(p)[r]);
    float z = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < cut.parts; ++p) {
        const float *const q = part(p);
        const float w = attn::ex2(q[r] - M);
        const float4 u = *reinterpret_cast<const float4 *>(q + 2 * item_rows + (size_t)r * D + 4 * lane);
        z = fmaf(q[item_rows + r], w, z);
        o.x = fmaf(u.x, w, o.x); o.y = fmaf(u.y, w, o.y); o.z = fmaf(u.z, w, o.z); o.w = fmaf(u.w, w, o.w);
    }
    const float f = z > 0.f || z != z ? 1.f / z : 0.f;
    T *dst = static_cast<T *>(const_cast<void *>(a.out.p)) + (long long)(cut.row0 + tok) * a.out.token +
             (long long)(cut.head0 + hd) * a.out.head + 4 * lane;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(o.x * f, o.y * f), pack2<T>(o.z * f, o.w * f));
}

}  // namespace

cudaError_t launch_join(const AttnArgs &a, int blocks, int item_rows, int tile_rows, cudaStream_t st) {
    const int per = kThreads / (a.c.D / 4);
    const dim3 grid(blocks, (item_rows + per - 1) / per);
    if (a.c.dtype == TKV_DTYPE_BF16) {
        if (a.c.D == 64) join_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(a, item_rows, tile_rows);
        else join_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(a, item_rows, tile_rows);
    } else {
        if (a.c.D == 64) join_kernel<__half, 64><<<grid, kThreads, 0, st>>>(a, item_rows, tile_rows);
        else join_kernel<__half, 128><<<grid, kThreads, 0, st>>>(a, item_rows, tile_rows);
    }
    return cudaGetLastError();
}

}  // namespace paged
}  // namespace tkv
