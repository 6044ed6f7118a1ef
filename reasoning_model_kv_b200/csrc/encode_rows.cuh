// encode_rows.cuh -- one warp's share of a token's heads, read, encoded and written.
#pragma once

#include "norm_rope.cuh"

namespace tkv {
namespace paged {

// Heads that one warp takes of a token: all of them when the tokens alone fill the card,
// fewer for a few tokens, so that a single token's heads are spread over many warps.
template <int D>
inline int heads_per_warp(int T, int heads) {
    constexpr int rows = 256 / D;                    // rows that a warp holds at once
    constexpr long long want = 148 * 32;             // warps that keep the card's memory busy
    long long per = ((long long)T * heads + want - 1) / want;
    per = (per + rows - 1) / rows * rows;
    return (int)(per < heads ? per : heads);
}

// A group of up to kUnroll warp-fuls of rows; WHOLE: all of them are there.
template <typename T, int D, bool NORM, bool FULL, bool WHOLE>
__device__ __forceinline__ void encode_group(const tkv_rope &rope, const T *in, long long in_stride, T *out,
                                             long long out_stride, const Row8 &w, const Angles &ang, const Chunks &c,
                                             int left) {
    constexpr int kRows = 256 / D, kUnroll = 4;
    const int gap = c.b - c.a;
    uint2 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (!WHOLE) a[u] = b[u] = make_uint2(0, 0);
        if (WHOLE || u * kRows < left) {
            a[u] = *reinterpret_cast<const uint2 *>(in + u * kRows * in_stride);
            b[u] = *reinterpret_cast<const uint2 *>(in + u * kRows * in_stride + gap);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        Row8 x = unpack8<T>(a[u], b[u]);
        if (NORM) row_norm<D>(x, w, rope.eps);
        if (FULL || c.turns) row_turn(x, ang, rope.interleaved);
        if (WHOLE || u * kRows < left) {
            T *p = out + u * kRows * out_stride;
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(x.v[0]), pack2<T>(x.v[1]));
            *reinterpret_cast<uint2 *>(p + gap) = make_uint2(pack2<T>(x.v[2]), pack2<T>(x.v[3]));
        }
    }
}

// Heads [h0, h1) of one array, whose token's rows begin at in and out.  FULL: every element is
// rotated, so no lane differs from another.
template <typename T, int D, bool NORM, bool FULL>
__device__ __forceinline__ void encode_heads(const tkv_rope &rope, const T *in, long long in_stride, T *out,
                                             long long out_stride, const Row8 &w, const Angles &ang, const Chunks &c, int h0,
                                             int h1) {
    constexpr int L = D / 8, kRows = 32 / L, kGroup = 4 * kRows;
    const int sub = (threadIdx.x & 31) / L;
    in += (h0 + sub) * in_stride + c.a;
    out += (h0 + sub) * out_stride + c.a;
    int h = h0;
    if (in_stride == D && out_stride == D) {       // heads side by side: offsets are constants
        for (; h + kGroup <= h1; h += kGroup) {
            encode_group<T, D, NORM, FULL, true>(rope, in, D, out, D, w, ang, c, 0);
            in += kGroup * D;
            out += kGroup * D;
        }
    }
    for (; h < h1; h += kGroup) {
        encode_group<T, D, NORM, FULL, false>(rope, in, in_stride, out, out_stride, w, ang, c, h1 - h - sub);
        in += kGroup * in_stride;
        out += kGroup * out_stride;
    }
}

template <typename T, int D, bool NORM, bool FULL>
__device__ __forceinline__ void encode_rows_as(const tkv_rope &rope, const Rows &q, const Rows &k, const Rows &qo,
                                               const Rows &ko, int t, int pos, int h0, int h1, int Hq) {
    const int j = threadIdx.x & (D / 8 - 1);
    const Chunks c = row_chunks(rope, j);
    double f[4];
    load_turns(rope, j, FULL || c.turns, f);
    const Angles ang = turn_angles(f, pos);
    if (h0 < Hq) {
        const Row8 w = NORM ? load_weights<T>(rope.q_weight, c) : Row8{};
        encode_heads<T, D, NORM, FULL>(rope, static_cast<const T *>(q.p) + t * q.token, q.head,
                                       static_cast<T *>(const_cast<void *>(qo.p)) + t * qo.token, qo.head, w, ang, c, h0,
                                       min(h1, Hq));
    }
    if (h1 > Hq) {
        const Row8 w = NORM ? load_weights<T>(rope.k_weight, c) : Row8{};
        encode_heads<T, D, NORM, FULL>(rope, static_cast<const T *>(k.p) + t * k.token, k.head,
                                       static_cast<T *>(const_cast<void *>(ko.p)) + t * ko.token, ko.head, w, ang, c,
                                       max(h0, Hq) - Hq, h1 - Hq);
    }
}

// Heads [h0, h1) of token t; heads from Hq on are keys.  All 32 lanes take part.
template <typename T, int D>
__device__ __forceinline__ void encode_rows(const tkv_rope &rope, const Rows &q, const Rows &k, const Rows &qo,
                                            const Rows &ko, int t, int pos, int h0, int h1, int Hq) {
    const bool full = rope.rot == D;
    if (rope.q_weight != nullptr) {
        if (full) encode_rows_as<T, D, true, true>(rope, q, k, qo, ko, t, pos, h0, h1, Hq);
        else encode_rows_as<T, D, true, false>(rope, q, k, qo, ko, t, pos, h0, h1, Hq);
    } else {
        if (full) encode_rows_as<T, D, false, true>(rope, q, k, qo, ko, t, pos, h0, h1, Hq);
        else encode_rows_as<T, D, false, false>(rope, q, k, qo, ko, t, pos, h0, h1, Hq);
    }
}

}  // namespace paged
}  // namespace tkv
