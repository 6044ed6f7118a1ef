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

#include "f32x2.cuh"
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

// A lane's eight elements as four packed pairs, in the order of its two chunks.
struct Row8 {
    uint64_t v[4];
};
template <typename T>
__device__ __forceinline__ Row8 unpack8(uint2 a, uint2 b) {
    const float2 p = unpack2<T>(a.x), q = unpack2<T>(a.y), r = unpack2<T>(b.x), s = unpack2<T>(b.y);
    return {pack_f2(p.x, p.y), pack_f2(q.x, q.y), pack_f2(r.x, r.y), pack_f2(s.x, s.y)};
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    unpack_f2(v, a, b);
    return pack2<T>(a, b);
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

// cos and sin of position * inv_freq for a lane's pairs: (c0 c1)(c2 c3), the same of sin.
struct Angles {
    uint64_t c[2], s[2];
};
// Whole turns are dropped in fp64, so a position of a million costs no accuracy; the rest is
// within half a turn, where the hardware's sine and cosine are off by 2^-20 at most -- against
// the 2^-9 and 2^-12 of the output types' rounding, and a sixth of the exact functions' cost.
__device__ __forceinline__ Angles turn_angles(const double (&f)[4], int pos) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double t = (double)pos * f[i];
        const float x = (float)(t - rint(t)) * 6.2831853071795864769f;
        c[i] = __cosf(x);
        s[i] = __sinf(x);
    }
    return {{pack_f2(c[0], c[1]), pack_f2(c[2], c[3])}, {pack_f2(s[0], s[1]), pack_f2(s[2], s[3])}};
}

// w: the norm's weights at the lane's places.
template <int D>
__device__ __forceinline__ void row_norm(Row8 &x, const Row8 &w, float eps) {
    uint64_t s2 = mul_f2(x.v[0], x.v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma_f2(x.v[i], x.v[i], s2);
    float a, b;
    unpack_f2(s2, a, b);
    float ss = a + b;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + eps);
    const uint64_t r2 = pack_f2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = mul_f2(mul_f2(x.v[i], r2), w.v[i]);
}

__device__ __forceinline__ uint64_t neg_f2(uint64_t a) { return a ^ 0x8000000080000000ull; }

__device__ __forceinline__ void row_turn(Row8 &x, const Angles &t, bool interleaved) {
    if (interleaved) {
        float c[4], s[4];
        unpack_f2(t.c[0], c[0], c[1]);
        unpack_f2(t.c[1], c[2], c[3]);
        unpack_f2(t.s[0], s[0], s[1]);
        unpack_f2(t.s[1], s[2], s[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack_f2(x.v[i], a, b);
            x.v[i] = fma_f2(x.v[i], pack_f2(c[i], c[i]), mul_f2(pack_f2(b, a), pack_f2(-s[i], s[i])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t a = x.v[i], b = x.v[i + 2];
            x.v[i] = fma_f2(a, t.c[i], mul_f2(b, neg_f2(t.s[i])));
            x.v[i + 2] = fma_f2(b, t.c[i], mul_f2(a, t.s[i]));
        }
    }
}

template <typename T>
__device__ __forceinline__ Row8 load_weights(const void *w, const Chunks &c) {
    const T *p = static_cast<const T *>(w);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = (float)p[c.a + i]; x[i + 4] = (float)p[c.b + i]; }
    return {pack_f2(x[0], x[1]), pack_f2(x[2], x[3]), pack_f2(x[4], x[5]), pack_f2(x[6], x[7])};
}

}  // namespace paged
}  // namespace tkv
