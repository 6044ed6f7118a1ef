// norm_rope.cu -- norm and rotation of queries and keys in one pass (tkv_qk_norm_rope).
//
// A warp takes a token's heads (several warps for a few tokens), so its angles are formed once;
// packed fp32 arithmetic keeps the instructions below what the memory needs.  Bound by HBM:
// 32768 tokens of 32 + 8 heads of 128, 671 MB, in 108 us (6.2 TB/s); 5003 tokens of 64 + 8
// heads of 64, 92 MB, in 21 us, where two rounds of warps for 34 warps an SM show; one token in
// 2.4 us.
#include "norm_rope.cuh"
#include "encode_rows.cuh"

namespace tkv {
namespace paged {
namespace {

constexpr int kThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(tkv_rope rope, Rows q, Rows k, const int32_t *pos, Rows qo,
                                                             Rows ko, int T_, int Hq, int Hkv, int groups, int per) {
    const int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = w / groups;
    if (t >= T_) return;
    const int h0 = (w - t * groups) * per;
    encode_rows<T, D>(rope, q, k, qo, ko, t, pos[t], h0, min(h0 + per, Hq + Hkv), Hq);
}

template <typename T, int D>
cudaError_t launch(const tkv_rope &rope, Rows q, Rows k, const int32_t *pos, Rows qo, Rows ko, int T_, int Hq, int Hkv,
                   cudaStream_t st) {
    const int per = heads_per_warp<D>(T_, Hq + Hkv);
    const int groups = (Hq + Hkv + per - 1) / per;
    const long long warps = (long long)T_ * groups;
    const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (warps > INT32_MAX - kThreads) return cudaErrorInvalidValue;
    norm_rope_kernel<T, D><<<(unsigned)blocks, kThreads, 0, st>>>(rope, q, k, pos, qo, ko, T_, Hq, Hkv, groups, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const tkv_rope &rope, Rows q, Rows k, const int32_t *pos, Rows qo, Rows ko, int T, int Hq,
                             int Hkv, int D, int dtype, cudaStream_t st) {
    if (dtype == TKV_DTYPE_BF16)
        return D == 64 ? launch<__nv_bfloat16, 64>(rope, q, k, pos, qo, ko, T, Hq, Hkv, st)
                       : launch<__nv_bfloat16, 128>(rope, q, k, pos, qo, ko, T, Hq, Hkv, st);
    return D == 64 ? launch<__half, 64>(rope, q, k, pos, qo, ko, T, Hq, Hkv, st)
                   : launch<__half, 128>(rope, q, k, pos, qo, ko, T, Hq, Hkv, st);
}

}  // namespace paged
}  // namespace tkv
