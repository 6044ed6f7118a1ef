// paged_attention_rows.cu -- attention of few query rows over the paged 8-bit cache.
//
// A block's four warps share an item's units of 64 keys, 16 keys a warp.  A warp streams its
// keys' codes through its own ring of shared-memory stages with asynchronous copies (no
// barrier between warps inside an item) and keeps its own running maximum, sum and output:
//   S^T [16 keys x rows] = K Q^T    O^T [D x rows] += V^T P^T
// with keys and values as the A operands of m16n8k16 instructions.  Codes of 8 bits are exact
// in fp16: E4M3 through the hardware's conversion, integers as 0x6480 | code less 1152.  The
// dims' order along QK's sum and the order of O's rows are free, so a lane takes 16-byte
// chunks: of rows g and g + 8 of K, and of four tokens of V whose bytes it interleaves.
// A page's key scale multiplies the fp32 products of Q K, its value scale those of P V, which are
// formed for 16 keys at a time: weights are relative to weights alone, whatever the scales are.
// P is fp16 times 2^7: rounded to 11 bits, more than either output type keeps, and to multiples
// of 2^-31 of the row's largest weight.  The second rounding matters where a value is far larger
// than those that carry the weight, so keys whose scale is over 2^10 times the smallest one's are
// multiplied in fp32 (kWide): 64 x 32k tokens 673 us, 1154 with half the pages 2^12 above the others.
// The maximum moves only when a logit passes it by 2^8, so most tiles rescale nothing.
// Measured: 64 sequences of 32k E4M3 tokens, 4.30 GB, in 673 us = 6.39 TB/s (copy rate 6.55); one
// sequence of 131k int8 tokens, 269 MB, in 57 us = 4.7 TB/s (the split's ends and the join); 3 to
// 6 rows of 16 sequences with four heads a kv head (24 rows), 194 MB, in 74 us = 2.6 TB/s: eight
// warps of 255 registers an SM leave the latency of their instructions uncovered.
#include <type_traits>

#include "norm_rope.cuh"
#include "paged_attention.cuh"
#include "paged_codes.cuh"

namespace tkv {
namespace paged {
namespace {

using attn::ex2;
using attn::kFull;
using attn::mma16816;
using attn::smem_addr;
using attn::transpose8x8;

constexpr int kThreads = 128, kWarps = 4, kUnitLog2 = 6, kUnit = 64;
constexpr int kStages = 4;
// An item's setup takes about as long as this many units.  With 0 / 2 / 4 / 8: ragged windows 40.8 /
// 28.5 / 27.8 / 29.1 us, verification 77.7 / 77.3 / 74.3 / 77.4, one of 131k 58.4 / 57.0 / 56.4 / 57.5.
constexpr int kItemCost = 4;
constexpr float kWide = 1024.f;
// Sums of weights times values: 2^15 above them is room for weights of 2^8 times 2^7.
constexpr float kSumUnit = 1.f / 32768.f;
// Parts that the last block to arrive joins by itself; more are left to the join kernel, whose
// rows are spread over the card (one block joined 56 parts of 8 rows in 14 us, it in 3).
constexpr int kOwnParts = 16;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, uint32_t src_size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_size) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Byte offset of 16-byte chunk c of row r in a [16][D] tile.  128-byte lines with their chunks
// exchanged so that both read patterns (rows g, chunks 2 tig + i; rows 2 tig, chunk g) touch
// every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
    else return (r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (r & 6)) << 4);
}

struct Stage {
    float ks, vs;      // the page's scales
    int live;          // 0: no page to read
    int wide;          // the products with its values are formed in fp32
};

// o += P V of 16 keys in fp32: the lane's rows 2 tig, 2 tig + 1 of every row tile and its D / 8 dims,
// which are 16 (8) codes of every key.  p as the products S left it, below 0 where the row does not
// see the key (whose value may be NaN), f the values' factor.
template <int D, int CODE, int NT>
__device__ __forceinline__ void plain_values(uint32_t vt, float f, const float (&p)[NT][4], float (&o)[NT][D / 16][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            uint32_t w[D / 32];
            if constexpr (D == 128) {
                const uint4 u = lds128(vt + chunk_at<D>(j + 8 * half, g));
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            } else {
                const uint2 u = lds64(vt + chunk_at<D>(j + 8 * half, g >> 1) + 8 * (g & 1));
                w[0] = u.x; w[1] = u.y;
            }
            float pj[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) pj[nt][e] = __shfl_sync(kFull, p[nt][e + 2 * half], 4 * j + tig);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t c[2];
                code_pairs<CODE>(w[i], c[0], c[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 v = __half22float2(attn::u32_as_h2(c[k]));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (pj[nt][e] < 0.f) continue;
                            o[nt][2 * i + k][e] = fmaf(pj[nt][e] * f, v.x, o[nt][2 * i + k][e]);
                            o[nt][2 * i + k][e + 2] = fmaf(pj[nt][e] * f, v.y, o[nt][2 * i + k][e + 2]);
                        }
                }
            }
        }
    }
}

// the ring; a block's join of four warps' rows takes no more (32 rows of D fp32)
template <int D>
constexpr int smem_bytes() { return kWarps * kStages * 2 * 16 * D; }

template <typename T, int D, int CODE, int NT>
__global__ void __launch_bounds__(kThreads) rows_kernel(const AttnArgs a) {
    constexpr int kRows = 8 * NT, kSteps = D / 16, kTile = 16 * D, kStageBytes = 2 * kTile;
    constexpr int kPartFloats = kRows * (D + 2);
    extern __shared__ __align__(128) uint8_t ring_all[];
    __shared__ Plan plan;
    __shared__ Stage stage_info[kWarps][kStages];
    __shared__ float sm_m[kWarps][kRows], sm_z[kWarps][kRows];
    __shared__ int sm_last;
    const View &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const uint32_t ring = smem_addr(ring_all) + warp * kStages * kStageBytes;

    // where the lane's chunk of a copy of 512 bytes goes; four rows of 128 bytes on, the exchange
    // of chunks differs in one bit
    const uint32_t lane_at = chunk_at<D>(lane * 16 / D, lane * 16 % D >> 4);
    const uint32_t lane_flip = D == 128 ? (lane_at ^ 64) - lane_at : 0;

    long long begin, share;
    make_plan<kThreads>(a, plan, kUnitLog2, &begin, &share);
    if (tid == 0) a.cut[blockIdx.x] = CutItem{};
    if (begin >= plan.total) return;
    const long long end = min(begin + share, plan.total);
    Cursor k;
    cursor_start(a, plan, begin, kUnitLog2, &k);
    do {
        int u0, nu;
        cursor_units(k, begin, end, &u0, &nu);
        if (nu == 0) continue;
        const int tokens = min(a.tile_tokens, k.s.n - k.i0);
        // ---- the warp's 16 keys of every unit
        const int tok0 = ((k.r.tile0 + u0) << kUnitLog2) + warp * 16;         // first key of the first unit
        // Pages and scales of 32 units at a time, a lane each, the next 32 in flight.
        int id0 = -1, id1 = -1;
        float ks0 = 0.f, vs0 = 0.f, ks1 = 0.f, vs1 = 0.f;
        auto fetch = [&](int i0, int &id, float &ks, float &vs) {
            const int t = tok0 + ((i0 + lane) << kUnitLog2);
            id = -1;
            ks = vs = 0.f;
            if (i0 + lane < nu && t < k.r.hi && t + 15 >= k.r.lo) {
                uint32_t bad = 0;
                id = load_page(c, a.block_table, k.b, t >> c.page_log2, &bad);
                if (id >= 0) {
                    ks = c.k_scale[(size_t)id * c.Hkv + k.h];
                    vs = c.v_scale[(size_t)id * c.Hkv + k.h];
                } else if (k.h == 0) {
                    latch(c, bad);
                }
            }
        };
        fetch(0, id0, ks0, vs0);
        fetch(32, id1, ks1, vs1);
        // the smallest value scale of the units so far, at first of the first 64; that of zeros does
        // not count (a page of zeros would make all others wide)
        float low = INFINITY;
        auto lower = [&](float vs) {
            vs = vs > 0.f && vs != kLeastScale ? vs : INFINITY;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) vs = fminf(vs, __shfl_xor_sync(kFull, vs, s));
            low = fminf(low, vs);
        };
        // The copies of unit i's keys and values, and what its products need of the page.
        auto copy = [&](int i) {
            if (i < nu) {
                if ((i & 31) == 0 && i > 0) {
                    id0 = id1; ks0 = ks1; vs0 = vs1;
                    fetch(i + 32, id1, ks1, vs1);
                    lower(vs0);
                }
                const int id = __shfl_sync(kFull, id0, i & 31);
                const int st = i % kStages, t = tok0 + (i << kUnitLog2);
                const size_t base = ((((size_t)max(id, 0) * c.Hkv + k.h) << c.page_log2) + (t & (c.page - 1))) * D + lane * 16;
                const uint8_t *const ks = c.k_pool + base, *const vs = c.v_pool + base;
                const uint32_t dst = ring + st * kStageBytes + lane_at, dst2 = dst + lane_flip;
                if (id >= 0 && t >= k.r.lo && t + 16 <= k.r.hi) {
#pragma unroll
                    for (int j = 0; j < kTile / 512; ++j) {
                        cp_async16((j & 1 ? dst2 : dst) + j * 512, ks + j * 512);
                        cp_async16((j & 1 ? dst2 : dst) + j * 512 + kTile, vs + j * 512);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kTile / 512; ++j) {
                        // rows that no query sees are zeros, whatever their codes are
                        const int r = t + (j * 512 + lane * 16) / D;
                        const uint32_t n = id >= 0 && r >= k.r.lo && r < k.r.hi ? 16 : 0;
                        cp_async16_or_zero((j & 1 ? dst2 : dst) + j * 512, ks + j * 512, n);
                        cp_async16_or_zero((j & 1 ? dst2 : dst) + j * 512 + kTile, vs + j * 512, n);
                    }
                }
            }
            attn::cp_async_commit();
        };
        auto note = [&](int i) {
            if (i < nu) {
                const int id = __shfl_sync(kFull, id0, i & 31);
                const float ks = __shfl_sync(kFull, ks0, i & 31), vs = __shfl_sync(kFull, vs0, i & 31);
                if (lane == 0) stage_info[warp][i % kStages] = Stage{ks, vs, id >= 0, vs > low * kWide};
            }
        };
        // the first copies go out before the queries are read and before the scales are there
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy(i);
        // ---- the queries, as B fragments (column g of every tile of eight rows)
        uint32_t qf[NT][kSteps][2];
        float qinv[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + g, ti = row / c.G;
            const bool live = ti < tokens;
            const T *src = static_cast<const T *>(a.q.p) + (long long)(k.s.row0 + k.i0 + ti) * a.q.token +
                           (long long)(k.h * c.G + row - ti * c.G) * a.q.head + tig * (D / 4);
            uint2 raw[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                raw[s] = live ? *reinterpret_cast<const uint2 *>(src + 4 * s) : make_uint2(0, 0);
            float inv = 1.f;
            if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
                // bf16 queries: a power of two brings the row's largest element to 2^8
                float mx = 0.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const float2 u = unpack2<T>(raw[s].x), v = unpack2<T>(raw[s].y);
                    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
                }
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                const int e = (int)(__float_as_uint(mx) >> 23) - 127;
                const int sh = e >= 128 ? 0 : min(8 - e, 126);          // not finite: as it is
                const float f = __uint_as_float((uint32_t)(sh + 127) << 23);
                inv = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const float2 u = unpack2<T>(raw[s].x), v = unpack2<T>(raw[s].y);
                    qf[nt][s][0] = attn::f32x2_to_f16x2(u.x * f, u.y * f);
                    qf[nt][s][1] = attn::f32x2_to_f16x2(v.x * f, v.y * f);
                }
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) { qf[nt][s][0] = raw[s].x; qf[nt][s][1] = raw[s].y; }
            }
            // of the columns that this lane's products are for
            qinv[nt][0] = __shfl_sync(kFull, inv, 8 * tig);
            qinv[nt][1] = __shfl_sync(kFull, inv, 8 * tig + 4);
        }
        float o[NT][kSteps][4], m[NT][2], z[NT][2];      // o: in units of kSumUnit
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = attn::kNoMax;
            z[nt][0] = z[nt][1] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) o[nt][s][0] = o[nt][s][1] = o[nt][s][2] = o[nt][s][3] = 0.f;
        }
        const int last_pos = k.r.first + tokens - 1;
        // Is element e of row tile nt's products with the 16 keys from t on outside its row's sight?
        auto hidden = [&](int nt, int e, int t) {
            const int pos = k.r.first + (nt * 8 + 2 * tig + (e & 1)) / c.G, j = t + g + 8 * (e >> 1);
            return j > pos || (a.window && j <= pos - a.window);
        };
        lower(vs0);
        lower(vs1);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) note(i);
        for (int i = 0; i < nu; ++i) {
            copy(i + kStages - 1);
            note(i + kStages - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const int st = i % kStages, t = tok0 + (i << kUnitLog2);
            const Stage info = stage_info[warp][st];
            if (info.live) {
                const uint32_t kt = ring + st * kStageBytes, vt = kt + kTile;
                float x[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const int ch = D == 128 ? 2 * tig + part : tig;
                    const uint4 r0 = lds128(kt + chunk_at<D>(g, ch)), r1 = lds128(kt + chunk_at<D>(g + 8, ch));
                    const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        code_pairs<CODE>(w0[w], a0, a2);
                        code_pairs<CODE>(w1[w], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(x[nt], a0, a1, a2, a3, qf[nt][part * 4 + w][0], qf[nt][part * 4 + w][1]);
                    }
                }
                const float kf = info.ks * a.scale_log2;
                bool up = false;
                const bool edge = t + 15 > k.r.first || (a.window && t <= last_pos - a.window);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float f0 = kf * qinv[nt][0], f1 = kf * qinv[nt][1];
                    x[nt][0] *= f0; x[nt][1] *= f1; x[nt][2] *= f0; x[nt][3] *= f1;
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (hidden(nt, e, t)) x[nt][e] = -INFINITY;
                    }
                    up |= fmaxf(x[nt][0], x[nt][2]) > m[nt][0] + attn::kRescaleSlack ||
                          fmaxf(x[nt][1], x[nt][3]) > m[nt][1] + attn::kRescaleSlack;
                }
                if (__any_sync(kFull, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float n = fmaxf(m[nt][e], fmaxf(x[nt][e], x[nt][e + 2]));
#pragma unroll
                            for (int s = 4; s < 32; s <<= 1) n = fmaxf(n, __shfl_xor_sync(kFull, n, s));
                            const float r = ex2(m[nt][e] - n);
                            m[nt][e] = n;
                            z[nt][e] *= r;
#pragma unroll
                            for (int s = 0; s < kSteps; ++s) { o[nt][s][e] *= r; o[nt][s][e + 2] *= r; }
                        }
                }
                const float vs = info.vs * kSumUnit;
                float p[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[nt][e] = ex2(x[nt][e] - m[nt][e & 1]);
                    z[nt][0] += p[nt][0] + p[nt][2];
                    z[nt][1] += p[nt][1] + p[nt][3];
                }
                bool plain = info.wide;
                if (CODE == TKV_CODE_E4M3 && edge) {
                    // a NaN of a key that some rows do not see: zero times it would be NaN
                    bool nan = false;
#pragma unroll
                    for (int i = 0; i < kTile / 512; ++i) {
                        const uint4 w = lds128(vt + i * 512 + lane * 16);
                        nan |= any_nan_code(w.x) || any_nan_code(w.y) || any_nan_code(w.z) || any_nan_code(w.w);
                    }
                    if (__any_sync(kFull, nan)) {
                        plain = true;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (hidden(nt, e, t)) p[nt][e] = -1.f;
                    }
                }
                if (plain) {
                    plain_values<D, CODE, NT>(vt, vs * 128.f, p, o);
                } else {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        pb[nt][0] = transpose8x8(attn::f32x2_to_f16x2(p[nt][0] * 128.f, p[nt][1] * 128.f));
                        pb[nt][1] = transpose8x8(attn::f32x2_to_f16x2(p[nt][2] * 128.f, p[nt][3] * 128.f));
                    }
                    // V: words of tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
                    constexpr int kWords = D / 32;
                    uint32_t v[4][kWords];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 2 * tig + (r & 1) + 8 * (r >> 1);
                        if constexpr (D == 128) {
                            const uint4 q4 = lds128(vt + chunk_at<D>(row, g));
                            v[r][0] = q4.x; v[r][1] = q4.y; v[r][2] = q4.z; v[r][3] = q4.w;
                        } else {
                            const uint2 q2 = lds64(vt + chunk_at<D>(row, g >> 1) + 8 * (g & 1));
                            v[r][0] = q2.x; v[r][1] = q2.y;
                        }
                    }
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const uint32_t sel = s & 1 ? 0x7362 : 0x5140;
                        uint32_t a0, a1, a2, a3;
                        code_pairs<CODE>(__byte_perm(v[0][s >> 1], v[1][s >> 1], sel), a0, a1);
                        code_pairs<CODE>(__byte_perm(v[2][s >> 1], v[3][s >> 1], sel), a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float t4[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(t4, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][s][e] = fmaf(t4[e], vs, o[nt][s][e]);
                        }
                    }
                }
            }
            __syncwarp();       // the stage is free for the next copies
        }
        cp_async_wait<0>();
        // ---- join the four warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) z[nt][e] += __shfl_xor_sync(kFull, z[nt][e], s);
                if (g == 0) {
                    sm_m[warp][nt * 8 + 2 * tig + e] = m[nt][e];
                    sm_z[warp][nt * 8 + 2 * tig + e] = z[nt][e] * (128.f * kSumUnit);
                }
            }
        __syncthreads();
        float *const obuf = reinterpret_cast<float *>(ring_all);       // [warp][row][D]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * tig + e;
                const float mm = fmaxf(fmaxf(sm_m[0][row], sm_m[1][row]), fmaxf(sm_m[2][row], sm_m[3][row]));
                const float f = ex2(m[nt][e] - mm);
                float *dst = obuf + (warp * kRows + row) * D + g * (D / 8);
#pragma unroll
                for (int s = 0; s < kSteps; s += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * s) = make_float4(o[nt][s][e] * f, o[nt][s][e + 2] * f,
                                                                           o[nt][s + 1][e] * f, o[nt][s + 1][e + 2] * f);
            }
        __syncthreads();
        const Parts cut = item_parts(k, share);
        const int parts = cut.count;
        auto out_at = [&](int row) {
            const int ti = row / c.G;
            return static_cast<T *>(const_cast<void *>(a.out.p)) + (long long)(k.s.row0 + k.i0 + ti) * a.out.token +
                   (long long)(k.h * c.G + row - ti * c.G) * a.out.head;
        };
        auto slot_of = [&](long long blk) { return part_at(a, kPartFloats, cut.first, blk); };
        const int live_rows = tokens * c.G;
        for (int i = tid; i < kRows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), col = i % (D / 4) * 4;
            if (row >= live_rows) break;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            float mm = attn::kNoMax, zz = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 u = *reinterpret_cast<const float4 *>(obuf + (w * kRows + row) * D + col);
                s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
                mm = fmaxf(mm, sm_m[w][row]);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) zz += sm_z[w][row] * ex2(sm_m[w][row] - mm);
            if (parts == 1) {
                const float f = zz > 0.f || zz != zz ? 1.f / zz : 0.f;
                *reinterpret_cast<uint2 *>(out_at(row) + col) =
                    make_uint2(pack2<T>(s.x * f, s.y * f), pack2<T>(s.z * f, s.w * f));
            } else {
                float *p = slot_of(blockIdx.x);
                *reinterpret_cast<float4 *>(p + 2 * kRows + row * D + col) = s;
                if (col == 0) { p[row] = mm; p[kRows + row] = zz; }
            }
        }
        if (parts > kOwnParts) {
            if (tid == 0 && blockIdx.x == cut.first)
                a.cut[blockIdx.x] = CutItem{k.s.row0 + k.i0, k.h * c.G, (int16_t)tokens, (int16_t)parts, 0};
        } else if (parts > 1) {
            __threadfence();
            __syncthreads();
            // the count wraps to zero with the last arrival, ready for the next call
            if (tid == 0) sm_last = atomicInc(a.arrived + cut.first, parts - 1) == (uint32_t)parts - 1;
            __syncthreads();
            if (sm_last) {
                __threadfence();
                float *const wt = reinterpret_cast<float *>(ring_all);   // [part][row] maxima, then weights
                float *const zt = wt + kOwnParts * kRows;                // sums
                for (int i = tid; i < parts * kRows; i += kThreads) {
                    const float *p = slot_of(cut.first + i / kRows) + i % kRows;
                    wt[i] = __ldcg(p);
                    zt[i] = __ldcg(p + kRows);
                }
                __syncthreads();
                if (tid < kRows) {
                    float n = attn::kNoMax, zz = 0.f;
                    for (int i = 0; i < parts; ++i) n = fmaxf(n, wt[i * kRows + tid]);
                    for (int i = 0; i < parts; ++i) {
                        const float w = ex2(wt[i * kRows + tid] - n);
                        zz = fmaf(zt[i * kRows + tid], w, zz);
                        wt[i * kRows + tid] = w;
                    }
                    sm_z[0][tid] = zz > 0.f || zz != zz ? 1.f / zz : 0.f;
                }
                __syncthreads();
                for (int i = tid; i < live_rows * (D / 4); i += kThreads) {
                    const int row = i / (D / 4), col = i % (D / 4) * 4;
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int p = 0; p < parts; ++p) {
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(slot_of(cut.first + p) + 2 * kRows + row * D + col));
                        const float w = wt[p * kRows + row];
                        s.x = fmaf(u.x, w, s.x); s.y = fmaf(u.y, w, s.y); s.z = fmaf(u.z, w, s.z); s.w = fmaf(u.w, w, s.w);
                    }
                    const float f = sm_z[0][row];
                    *reinterpret_cast<uint2 *>(out_at(row) + col) =
                        make_uint2(pack2<T>(s.x * f, s.y * f), pack2<T>(s.z * f, s.w * f));
                }
            }
        }
        __syncthreads();        // the ring and the join's arrays are free
    } while (cursor_next(a, kUnitLog2, end, &k));
}

template <typename T, int D, int CODE, int NT>
cudaError_t run(AttnArgs a, cudaStream_t st, int64_t *launches) {
    static int occupancy[kMaxDevices];
    const auto kernel = rows_kernel<T, D, CODE, NT>;
    int sms = 0, per_sm = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e == cudaSuccess) e = cached_blocks_per_sm(occupancy, reinterpret_cast<const void *>(kernel), kThreads,
                                                   smem_bytes<D>(), &per_sm);
    if (e != cudaSuccess) return e;
    a.tile_tokens = 8 * NT / a.c.G;
    a.item_cost = kItemCost;
    const int blocks = min(sms * per_sm, min(kMaxBlocks, kPartRows / (8 * NT)));
    kernel<<<blocks, kThreads, smem_bytes<D>(), st>>>(a);
    e = cudaGetLastError();
    ++*launches;
    // no item has more units than the block table has room for (key_range)
    if (e == cudaSuccess && ((a.room + kUnit - 1) >> kUnitLog2) + 1 > kOwnParts) {
        e = launch_join(a, blocks, 8 * NT, 8 * NT, st);
        ++*launches;
    }
    return e;
}
template <typename T, int D, int CODE>
cudaError_t run_rows(const AttnArgs &a, long long rows, cudaStream_t st, int64_t *launches) {
    if (rows <= 8) return run<T, D, CODE, 1>(a, st, launches);
    if (rows <= 16) return run<T, D, CODE, 2>(a, st, launches);
    if (rows <= 24) return run<T, D, CODE, 3>(a, st, launches);
    return run<T, D, CODE, 4>(a, st, launches);
}
template <typename T>
cudaError_t run_type(const AttnArgs &a, long long rows, cudaStream_t st, int64_t *launches) {
    if (a.c.code == TKV_CODE_E4M3)
        return a.c.D == 64 ? run_rows<T, 64, TKV_CODE_E4M3>(a, rows, st, launches)
                           : run_rows<T, 128, TKV_CODE_E4M3>(a, rows, st, launches);
    return a.c.D == 64 ? run_rows<T, 64, TKV_CODE_INT8>(a, rows, st, launches)
                       : run_rows<T, 128, TKV_CODE_INT8>(a, rows, st, launches);
}

}  // namespace

size_t rows_workspace_bytes(int D) { return 2ull * kPartRows * (D + 2) * sizeof(float); }

cudaError_t launch_rows(AttnArgs a, long long rows, cudaStream_t st, int64_t *launches) {
    return a.c.dtype == TKV_DTYPE_BF16 ? run_type<__nv_bfloat16>(a, rows, st, launches) : run_type<__half>(a, rows, st, launches);
}

}  // namespace paged
}  // namespace tkv
