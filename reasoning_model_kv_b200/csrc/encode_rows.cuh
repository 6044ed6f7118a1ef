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

// Heads [h0, h1) of token t; heads from Hq on are keys.  All 32 lanes take part.
template <typename T, int D>
__device__ __forceinline__ void encode_rows(const tkv_rope &rope, const Rows &q, const Rows &k, const Rows &qo,
                                            const Rows &ko, int t, int pos, int h0, int h1, int Hq) {
    constexpr int L = D / 8, kRows = 32 / L, kUnroll = 4;
    const int lane = threadIdx.x & 31, j = lane & (L - 1), sub = lane / L;
    const Chunks c = row_chunks(rope, j);
    const T *const q0 = static_cast<const T *>(q.p) + t * q.token;
    const T *const k0 = static_cast<const T *>(k.p) + t * k.token;
    T *const qo0 = static_cast<T *>(const_cast<void *>(qo.p)) + t * qo.token;
    T *const ko0 = static_cast<T *>(const_cast<void *>(ko.p)) + t * ko.token;
    float cs[4], sn[4], qw[8], kw[8];
    bool ready = false;
    for (int h = h0; h < h1; h += kRows * kUnroll) {
        uint2 a[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hh = h + u * kRows + sub;
            a[u] = b[u] = make_uint2(0, 0);
            if (hh < h1) {
                const T *p = hh < Hq ? q0 + hh * q.head : k0 + (hh - Hq) * k.head;
                a[u] = *reinterpret_cast<const uint2 *>(p + c.a);
                b[u] = *reinterpret_cast<const uint2 *>(p + c.b);
            }
        }
        if (!ready) {    // behind the first loads, which it hides in part
            double f[4];
            load_turns(rope, j, c.turns, f);
            load_weights<T>(rope.q_weight, c, qw);
            load_weights<T>(rope.k_weight, c, kw);
            turn_angles(f, pos, cs, sn);
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hh = h + u * kRows + sub;
            float x[8];
            unpack8<T>(a[u], b[u], x);
            if (rope.q_weight != nullptr) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = hh < Hq ? qw[i] : kw[i];
                row_norm<D>(x, w, rope.eps);
            }
            if (c.turns) row_turn(x, cs, sn, rope.interleaved);
            if (hh < h1) {
                T *p = hh < Hq ? qo0 + hh * qo.head : ko0 + (hh - Hq) * ko.head;
                *reinterpret_cast<uint2 *>(p + c.a) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
                *reinterpret_cast<uint2 *>(p + c.b) = make_uint2(pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
            }
        }
    }
}

}  // namespace paged
}  // namespace tkv
