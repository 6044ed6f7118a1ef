// norm_rope.cuh -- norm and rotation of one head's row, the part that the encoding kernel
// and the paged append share.
//
// A row of D elements is held by D / 8 lanes, two chunks of four elements each.  The chunks
// are chosen so that both members of every rotated pair are in one lane: with `rot` a
// multiple of 8 the first rot/8 lanes hold chunks j and j + rot/8 (elements i and i + rot/2
// of split pairs), the others two neighbouring chunks of the part that is not rotated;
// interleaved pairs lie in neighbouring chunks anyway.  So a rotation needs no exchange
// between lanes, and a lane's four angles serve every head of its token.
#pragma once

#include "paged.cuh"

namespace tkv {
namespace paged {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(uint2 a, uint2 b, float (&x)[8]) {
    const float2 p = unpack2<T>(a.x), q = unpack2<T>(a.y), r = unpack2<T>(b.x), s = unpack2<T>(b.y);
    x[0] = p.x; x[1] = p.y; x[2] = q.x; x[3] = q.y;
    x[4] = r.x; x[5] = r.y; x[6] = s.x; x[7] = s.y;
}

// The elements that lane j of a row's D / 8 holds: offsets of its two chunks of four.
struct Chunks {
    int a, b;
    bool turns;      // they are rotated pairs
};
__device__ __forceinline__ Chunks row_chunks(const tkv_rope &r, int j) {
    const int n = r.rot >> 3;
    Chunks c;
    c.turns = j < n;
    if (r.interleaved || j >= n) { c.a = 8 * j; c.b = 8 * j + 4; }
    else { c.a = 4 * j; c.b = 4 * (j + n); }
    return c;
}

// Turns per position of the lane's four pairs.
__device__ __forceinline__ void load_turns(const tkv_rope &r, int j, bool turns, double (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = turns ? (double)r.inv_freq[4 * j + i] * 0.15915494309189533577 : 0.0;
}

// cos and sin of position * inv_freq: whole turns are dropped in fp64, so a position of a
// million costs no accuracy, and the rest is an fp32 angle within half a turn.
__device__ __forceinline__ void turn_angles(const double (&f)[4], int pos, float (&cs)[4], float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double t = (double)pos * f[i];
        sincospif(2.f * (float)(t - rint(t)), &sn[i], &cs[i]);
    }
}

// x: the lane's eight elements.  w: the norm's weights at the same places.
template <int D>
__device__ __forceinline__ void row_norm(float (&x)[8], const float (&w)[8], float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

__device__ __forceinline__ void row_turn(float (&x)[8], const float (&cs)[4], const float (&sn)[4], bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cs[i] - b * sn[i];
            x[2 * i + 1] = a * sn[i] + b * cs[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[i], b = x[i + 4];
            x[i] = a * cs[i] - b * sn[i];
            x[i + 4] = a * sn[i] + b * cs[i];
        }
    }
}

template <typename T>
__device__ __forceinline__ void load_weights(const void *w, const Chunks &c, float (&x)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 1.f;
        return;
    }
    const T *p = static_cast<const T *>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = (float)p[c.a + i]; x[i + 4] = (float)p[c.b + i]; }
}

}  // namespace paged
}  // namespace tkv
