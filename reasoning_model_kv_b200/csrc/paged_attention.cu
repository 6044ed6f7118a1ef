// paged_attention.cu -- attention over the paged 8-bit cache.
//
// One block per (query row, kv head); its four warps take the row's G heads in turn and walk
// the keys with the running maximum and sum of a softmax, a lane holding D / 32 dims.
#include <climits>

#include <cuda_fp8.h>

#include "paged.cuh"

namespace tkv {
namespace paged {
namespace {

struct AttnArgs {
    View c;
    Rows q, out;
    const int32_t *block_table, *kv_len, *cu;
    int T, window;
    float scale_log2;       // softmax_scale * log2(e)
};

template <int CODE>
__device__ __forceinline__ float code_value(uint8_t w) {
    if constexpr (CODE == TKV_CODE_E4M3)
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(w, __NV_E4M3)));
    else
        return (float)(int8_t)w;
}

template <typename T, int D, int CODE>
__global__ void __launch_bounds__(128) attend_kernel(const AttnArgs a) {
    const View &c = a.c;
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31;
    constexpr int E = D / 32;
    int b = t;
    if (a.cu) {
        b = 0;
        for (int i = 0; i < c.B; i += 32) b += __popc(__ballot_sync(0xffffffffu, i + lane < c.B && a.cu[i + lane + 1] <= t));
    }
    if (b >= c.B) return;
    Seq s;
    uint32_t bad;
    // the rows of a sequence whose length cannot be used are zeros
    const bool ok = load_seq(a.cu, a.kv_len, b, a.T, &s, &bad);
    if (!ok && threadIdx.x == 0 && h == 0) latch(c, bad);
    if (ok && (t < s.row0 || t >= s.row0 + s.n)) return;
    if (!ok && bad == kBadRows) return;
    const int pos = s.len - s.n + (t - s.row0);
    const int lo = a.window ? max(0, pos - a.window + 1) : 0;
    for (int g = threadIdx.x >> 5; g < c.G; g += 4) {
        const T *q = static_cast<const T *>(a.q.p) + t * a.q.token + (h * c.G + g) * a.q.head + lane * E;
        T *o = static_cast<T *>(const_cast<void *>(a.out.p)) + t * a.out.token + (h * c.G + g) * a.out.head + lane * E;
        float qv[E], acc[E], m = -INFINITY, z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) { qv[e] = (float)q[e]; acc[e] = 0.f; }
        for (int j = ok ? lo : pos + 1; j <= pos; ++j) {
            const int id = load_page(c, a.block_table, b, j >> c.page_log2, &bad);
            if (id < 0) {
                if (lane == 0 && g == 0 && h == 0) latch(c, bad);
                j |= c.page - 1;
                continue;
            }
            const size_t ps = (size_t)id * c.Hkv + h;
            const size_t off = ((ps << c.page_log2) + (j & (c.page - 1))) * D + lane * E;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(qv[e], code_value<CODE>(c.k_pool[off + e]), x);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
            x *= c.k_scale[ps] * a.scale_log2;
            const float mn = fmaxf(m, x), r = exp2f(m - mn), p = exp2f(x - mn), pv = p * c.v_scale[ps];
            z = z * r + p;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], r, pv * code_value<CODE>(c.v_pool[off + e]));
            m = mn;
        }
        const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = (T)(acc[e] * inv);
    }
}

template <typename T>
cudaError_t run(const AttnArgs &a, cudaStream_t st) {
    const dim3 grid(a.T, a.c.Hkv);
    if (a.c.code == TKV_CODE_E4M3) {
        if (a.c.D == 64) attend_kernel<T, 64, TKV_CODE_E4M3><<<grid, 128, 0, st>>>(a);
        else attend_kernel<T, 128, TKV_CODE_E4M3><<<grid, 128, 0, st>>>(a);
    } else {
        if (a.c.D == 64) attend_kernel<T, 64, TKV_CODE_INT8><<<grid, 128, 0, st>>>(a);
        else attend_kernel<T, 128, TKV_CODE_INT8><<<grid, 128, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(const tkv_paged_config &) { return 0; }

cudaError_t launch_attention(const View &c, Rows q, Rows out, int T, const int32_t *block_table,
                             const int32_t *kv_len, const int32_t *cu, int max_q, int window, float scale,
                             cudaStream_t st, int64_t *launches) {
    (void)max_q;
    AttnArgs a{c, q, out, block_table, kv_len, cu, T, window, scale * 1.4426950408889634f};
    const cudaError_t e = c.dtype == TKV_DTYPE_BF16 ? run<__nv_bfloat16>(a, st) : run<__half>(a, st);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace paged
}  // namespace tkv
