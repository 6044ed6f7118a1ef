// paged_attention_tiles.cu -- attention of many query rows (prompt chunks, long verification
// steps) over the paged 8-bit cache, on the 5th-generation tensor cores.
//
// One resident block per SM; an item is up to two tiles of 128 query rows (tokens x the G
// heads of a kv head) against units of 128 keys.  Warpgroups 0 and 1 hold a row a thread and
// do the softmax, warpgroup 2 turns the cache's codes into fp16 operands (exact for both code
// types) in shared memory, one thread of warpgroup 3 issues the matrix instructions:
//   S [128 x 128] = Q K^T   (Q, K in shared memory, K-major, 128-byte swizzle)
//   O [128 x D]  += P V     (P fp16 in tensor memory over S, V in shared memory, MN-major)
// With two tiles of rows the tensor cores work on one while the other is in its softmax, and
// converting a key costs 1/256 of a row's work.
// A page's two scales enter as y = x + log2(value scale) in place of the logit x: P = 2^(y - M)
// carries the value scale, O = sum P code, and the softmax sum is sum P / value scale, so both
// have one running maximum M, which moves only when y passes it by 2^8.  P is fp16 times 2^7:
// 11 bits, more than either output type keeps, and multiples of 2^-31 of the largest.  So an
// attended key of a page with a large scale, even one whose codes are zeros, takes bits from the
// others: 2^10 between an item's scales leave 2^-21 of the largest weight.  Rows of items whose
// scales are further apart are formed in fp32 by the join kernel, which follows anyway, and so are
// those of items with a NaN value that some rows see and others do not (zero times it would be
// NaN); warps of their own look for them (the softmax's or the codes' warps would take 1 to 5 %
// longer).
//
// Measured: two chunks of 2048 rows x 32 heads on 14k and 16k keys, 961 GFLOP, in 888 us = 1.08
// PFLOP/s, 65 % of the library's bf16 product (pages of 16 1037 us, int8 908); with 64-dim heads 734 us;
// four prompts of 4096 without a prefix, 550 GFLOP, 835 us.  Tensor cores and exponentials are each
// busy 46 % of the time: a unit's softmax follows its S and precedes its O, and the second tile of
// rows covers only part of that.  Every instantiation spills (64 to 112 bytes of stack; softmax
// and codes both).  Slower: two threads a row (16 softmax warps), the maximum and P in
// one pass with a second one where the maximum moved, an issuing warp for each tile of rows (its
// products take turns with the other's; 312 -> 380 us on 2048 rows x 16 heads x 8k keys).
#include <climits>

#include <cuda_fp8.h>

#include "f32x2.cuh"
#include "norm_rope.cuh"
#include "paged_attention.cuh"
#include "paged_codes.cuh"
#include "tcgen05.cuh"

namespace tkv {
namespace paged {
namespace {

using attn::ex2;
using attn::kFull;
using attn::mbar_arrive;
using attn::mbar_wait;
using attn::smem_addr;

constexpr int kThreads = 512, kUnitLog2 = kTileUnitLog2, kUnit = 1 << kUnitLog2;
// An item's setup takes about as long as this many units.  With 0 / 1 / 2 / 4: 64 rows on 4 to 8k tokens
// 131.2 / 128.6 / 124.4 / 125.4 us, 33 rows on 1000 17.0 / 17.3 / 16.7 / 16.5, prompt chunks 891 / 890 /
// 887 / 887.
constexpr int kItemCost = 2;
constexpr int kChunks = kUnit / 16;      // groups of keys that share a page
constexpr int kConstSets = 4;
constexpr int kReaders = 3;              // warps that look for what is left to the join kernel's plain rows
// Items whose value scales are further apart, or larger, are.
constexpr float kScaleSpread = 1024.f, kScaleMost = 1048576.f;
constexpr float kTiny = 1e-37f;          // factors of logits stay above zero: -inf times one is -inf
constexpr uint32_t kColS = 0, kColO = 256;      // tensor memory: S of tile s at 128 s, O at 256 + 128 s

template <int D>
struct Layout {
    static constexpr int kTile = 128 * D * 2;                  // a tile of fp16 operands
    static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kBytes = 6 * kTile + 1024;
};

// What the softmax needs of 16 keys: key scale times the softmax scale (log2 units), log2 of
// the value scale, its inverse.
struct __align__(16) ChunkConst {
    float f, lb, iv, pad;
};

struct Barriers {
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];
    uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2];
    uint64_t c_full[kConstSets], drain;
};

// Byte offset of the 16-byte chunk (8 dims) ch of row r in a [128][D] fp16 tile: atoms of 64
// dims, 128-byte swizzle.
__device__ __forceinline__ uint32_t operand_at(int r, int ch) {
    return (ch >> 3) * 16384 + r * 128 + (((ch ^ r) & 7) << 4);
}

// A bounded wait with one answer for the whole warp.
__device__ __forceinline__ bool warp_wait(const uint64_t *bar, uint32_t parity) {
    return __all_sync(kFull, mbar_wait(smem_addr(bar), parity));
}

// Counts in shared memory that a warp each raises: what they did before is seen behind the wait, which
// is bounded as those on barriers are.
__device__ __forceinline__ void store_release(uint32_t *count, uint32_t n) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_addr(count)), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ bool wait_above(const uint32_t (&count)[N], uint32_t n) {
    const uint32_t at = smem_addr(count + (threadIdx.x & 31) % N);
    auto above = [&] {
        uint32_t v;
        asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
        return v > n;
    };
    bool there = above();
    for (const long long t0 = clock64(); !there && clock64() - t0 <= attn::kWaitCycles;) there = above();
    return __all_sync(kFull, there);
}

__device__ __forceinline__ void st128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// SETS: constants of a unit that the softmax reads, one for every 64 keys (pages of 64 tokens or
// more) or every 16.
template <typename T, int D, int CODE, int SETS>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ AttnArgs a) {
    using L = Layout<D>;
    constexpr int kPartFloats = 256 * (D + 2);
    extern __shared__ uint8_t smem_raw[];
    __shared__ Plan plan;
    __shared__ __align__(8) Barriers bar;
    __shared__ ChunkConst consts[kConstSets][kChunks];
    __shared__ uint32_t tmem_base;
    __shared__ int plain_from;                // number of the first item that is left to the join
    __shared__ uint32_t items_read[kReaders]; // items that each reader has looked through
    const View &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int sub_tokens = 128 / c.G;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.k_full[i], 4);
            tc::mbar_init(&bar.v_full[i], 4);
            tc::mbar_init(&bar.k_free[i], 1);
            tc::mbar_init(&bar.v_free[i], 1);
            tc::mbar_init(&bar.q_ready[i], 4);
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_ready[i], 4);
            tc::mbar_init(&bar.o_full[i], 1);
        }
        for (int i = 0; i < kConstSets; ++i) tc::mbar_init(&bar.c_full[i], 4);
        tc::mbar_init(&bar.drain, 1);
        tc::mbar_init_fence();
        plain_from = INT_MAX;
        for (int i = 0; i < kReaders; ++i) items_read[i] = 0;
        a.cut[blockIdx.x] = CutItem{};
    }
    if (warp == 12) tc::alloc(smem_addr(&tmem_base), 512);
    long long begin, share;
    make_plan<kThreads>(a, plan, kUnitLog2, &begin, &share);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tb = tmem_base;
    const long long end = min(begin + share, plan.total);
    bool ok = true;
    if (begin < plan.total) {
        Cursor k;
        cursor_start(a, plan, begin, kUnitLog2, &k);
        uint32_t n_tile = 0, n_item = 0;          // units and items behind
        uint32_t n_tile1 = 0, n_item1 = 0;        // of the second tile of rows
        if (warp < 8) {
            // 176, 104 and 56 registers for the three kinds of warps: the launch's 512 x 128 in all
            asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
            const int sub = warp >> 2, row = tid & 127;
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;
            const uint32_t s_col = tb + lanes + kColS + 128 * sub, o_col = tb + lanes + kColO + 128 * sub;
            const int ti = row / c.G, hd = row - ti * c.G;
            do {
                int u0, nu;
                cursor_units(k, begin, end, &u0, &nu);
                if (nu == 0) continue;
                const int tokens = min(a.tile_tokens, k.s.n - k.i0);
                if (sub == 0 || tokens > sub_tokens) {
                    const int tok = sub * sub_tokens + ti;
                    const bool live = ti < sub_tokens && tok < tokens;
                    // ---- the row's query into the operand tile
                    float qinv = 1.f;
                    {
                        const T *src = static_cast<const T *>(a.q.p) + (long long)(k.s.row0 + k.i0 + tok) * a.q.token +
                                       (long long)(k.h * c.G + hd) * a.q.head;
                        const uint32_t dst = sm + L::kQ + sub * L::kTile;
                        uint2 raw[D / 4];
#pragma unroll
                        for (int i = 0; i < D / 4; ++i)
                            raw[i] = live ? *reinterpret_cast<const uint2 *>(src + 4 * i) : make_uint2(0, 0);
                        float f = 1.f;
                        if constexpr (!std::is_same<T, __half>::value) {
                            // a power of two brings the row's largest element to 2^8
                            float mx = 0.f;
#pragma unroll
                            for (int i = 0; i < D / 4; ++i) {
                                const float2 u = unpack2<T>(raw[i].x), v = unpack2<T>(raw[i].y);
                                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
                            const int e = (int)(__float_as_uint(mx) >> 23) - 127;
                            const int sh = e >= 128 ? 0 : min(8 - e, 126);
                            f = __uint_as_float((uint32_t)(sh + 127) << 23);
                            qinv = __uint_as_float((uint32_t)(127 - sh) << 23);
                        }
                        if (a.scale_log2 < 0.f) f = -f;       // the keys' factors are not negative
#pragma unroll
                        for (int i = 0; i < D / 4; i += 2) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float2 u = unpack2<T>(raw[i + j].x), v = unpack2<T>(raw[i + j].y);
                                w[2 * j] = attn::f32x2_to_f16x2(u.x * f, u.y * f);
                                w[2 * j + 1] = attn::f32x2_to_f16x2(v.x * f, v.y * f);
                            }
                            st128(dst + operand_at(row, i / 2), w[0], w[1], w[2], w[3]);
                        }
                        attn::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&bar.q_ready[sub]));
                    }
                    const int pos = k.r.first + tok;
                    const int sub_first = k.r.first + sub * sub_tokens, sub_last = sub_first + sub_tokens - 1;
                    float M = attn::kNoMax, z = 0.f;
                    const uint32_t base = sub ? n_tile1 : n_tile;       // tiles of this half before the item
                    for (int i = 0; i < nu && ok; ++i) {
                        const uint32_t n = base + i, kt = n_tile + i;
                        // An item without a second tile of rows is passed over by that tile's warps, and
                        // the codes' phases they have not followed are met again with S.
                        if (i == 0) ok = warp_wait(&bar.s_full[sub], n & 1);
                        ok = ok && warp_wait(&bar.c_full[kt & (kConstSets - 1)], (kt / kConstSets) & 1);
                        // read while S is formed: with eight reads behind it a unit took an eighth longer
                        const ChunkConst *cc = consts[kt & (kConstSets - 1)];
                        constexpr int kKeys = kUnit / SETS;
                        float f[SETS], lb[SETS];
#pragma unroll
                        for (int j = 0; j < SETS; ++j) {
                            const ChunkConst w = cc[j * (kKeys / 16)];
                            f[j] = fmaxf(w.f * qinv, kTiny);
                            lb[j] = w.lb;
                        }
                        ok = ok && warp_wait(&bar.s_full[sub], n & 1);
                        if (!ok) break;
                        tc::fence_after();
                        uint32_t s[128];
#pragma unroll
                        for (int j = 0; j < 128; j += 32) tc::ld32(s_col + j, s + j);
                        tc::wait_ld<128>(s);
                        const int t0 = (k.r.tile0 + u0 + i) << kUnitLog2;
                        // (keys without a page are zeros, and S is NaN there if the query is not finite)
                        float least = lb[0];
#pragma unroll
                        for (int j = 1; j < SETS; ++j) least = fminf(least, lb[j]);
                        if (t0 + kUnit - 1 > sub_first || (a.window && t0 <= sub_last - a.window) || least == -INFINITY) {
                            const int hi = pos - t0, lo = a.window ? hi - a.window : -1;      // lo < key <= hi
#pragma unroll
                            for (int j = 0; j < 128; ++j)
                                if (j > hi || j <= lo || lb[j / kKeys] == -INFINITY) s[j] = 0xff800000u;
                        }
                        float ym = -INFINITY;
#pragma unroll
                        for (int j = 0; j < SETS; ++j) {
                            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < kKeys; e += 2)
                                m[(e >> 1) & 3] = max3(m[(e >> 1) & 3], __uint_as_float(s[kKeys * j + e]), __uint_as_float(s[kKeys * j + e + 1]));
                            ym = fmaxf(ym, fmaf(fmaxf(max3(m[0], m[1], m[2]), m[3]), f[j], lb[j]));
                        }
                        if (__any_sync(kFull, ym > M + attn::kRescaleSlack)) {
                            const float n_M = fmaxf(M, ym), r = ex2(M - n_M);
                            M = n_M;
                            z *= r;
                            if (i > 0) {
                                ok = warp_wait(&bar.o_full[sub], (n - 1) & 1);
                                tc::fence_after();
#pragma unroll
                                for (int j = 0; j < D; j += 16) {
                                    uint32_t o[16];
                                    tc::ld16(o_col + j, o);
                                    tc::wait_ld<16>(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                                    tc::st16(o_col + j, o);
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < SETS; ++j) {
                            const float b = lb[j] - M + 7.f;
                            const uint64_t f2 = pack_f2(f[j], f[j]), b2 = pack_f2(b, b);
                            uint64_t sum[2] = {0, 0};
#pragma unroll
                            for (int q = 0; q < kKeys; q += 16) {
                                uint32_t p[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const int at = kKeys * j + q + 2 * e;
                                    float u, v;
                                    unpack_f2(fma_f2(pack_f2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), f2, b2), u, v);
                                    u = ex2(u);
                                    v = ex2(v);
                                    sum[e & 1] = add_f2(sum[e & 1], pack_f2(u, v));
                                    p[e] = attn::f32x2_to_f16x2(u, v);
                                }
                                tc::st8(s_col + (kKeys * j + q) / 2, p);
                            }
                            float su, sv;
                            unpack_f2(add_f2(sum[0], sum[1]), su, sv);
                            z = fmaf(su + sv, cc[j * (kKeys / 16)].iv, z);
                        }
                        tc::wait_st();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&bar.p_ready[sub]));
                    }
                    // ---- the row's output
                    if (ok) ok = warp_wait(&bar.o_full[sub], (base + nu - 1) & 1);
                    tc::fence_after();
                    const Parts cut = item_parts(k, share);
                    const int parts = cut.count;
                    ok = wait_above<kReaders>(items_read, n_item) && ok;
                    const bool plain = *const_cast<volatile int *>(&plain_from) <= (int)n_item;
                    if (parts == 1) {
                        const float f = z > 0.f || z != z ? 1.f / z : 0.f;
                        T *dst = static_cast<T *>(const_cast<void *>(a.out.p)) + (long long)(k.s.row0 + k.i0 + tok) * a.out.token +
                                 (long long)(k.h * c.G + hd) * a.out.head;
#pragma unroll
                        for (int j = 0; j < D; j += 16) {
                            uint32_t o[16];
                            tc::ld16(o_col + j, o);
                            tc::wait_ld<16>(o);
                            if (live && ok && !plain) {
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<uint2 *>(dst + j + e) = make_uint2(
                                        pack2<T>(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f),
                                        pack2<T>(__uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f));
                            }
                        }
                    } else {
                        float *p = part_at(a, kPartFloats, cut.first, blockIdx.x);
                        const int r = sub * 128 + row;
#pragma unroll
                        for (int j = 0; j < D; j += 16) {
                            uint32_t o[16];
                            tc::ld16(o_col + j, o);
                            tc::wait_ld<16>(o);
                            if (live) {
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<uint4 *>(p + 512 + r * D + j + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            }
                        }
                        if (live) { p[r] = M; p[256 + r] = z; }
                        if (tid == 0 && blockIdx.x == cut.first)
                            a.cut[blockIdx.x] = CutItem{k.s.row0 + k.i0, k.h * c.G, (int16_t)tokens, (int16_t)parts, 0};
                    }
                    tc::fence_before();      // the reads of O are behind the next item's products
                }
                if (!ok) break;
                n_tile += nu;
                n_item += 1;
                if (tokens > sub_tokens) { n_tile1 += nu; n_item1 += 1; }
            } while (cursor_next(a, kUnitLog2, end, &k));
        } else if (warp < 12) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
            // ---- codes to operands: a warp's rows are keys 32 w .. 32 w + 31 of every unit, a lane's
            // loads row (lane / 4) of eight, 16 codes
            const int w = warp - 8, r8 = lane >> 2, q4 = lane & 3;
            constexpr int kHalves = D / 64, kLoads = 4 * kHalves;
            const float sl = fabsf(a.scale_log2);
            uint4 kr[kLoads], vr[kLoads];
            do {
                int u0, nu;
                cursor_units(k, begin, end, &u0, &nu);
                if (nu == 0) continue;
                const int t_item = ((k.r.tile0 + u0) << kUnitLog2) + 32 * w;
                // pages and scales of the warp's two groups of 16 keys, 16 units at a time
                int id0 = -1, id1 = -1;
                float ks0 = 0.f, vs0 = 0.f, ks1 = 0.f, vs1 = 0.f;
                auto fetch = [&](int i0, int &id, float &ks, float &vs) {
                    const int u = i0 + (lane >> 1), t = t_item + (u << kUnitLog2) + 16 * (lane & 1);
                    id = -1;
                    ks = vs = 0.f;
                    // (constants read for 64 keys are those of their first 16, visible or not)
                    if (u < nu && t < k.r.hi && (t | (kUnit / SETS - 1)) >= k.r.lo) {
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
                fetch(16, id1, ks1, vs1);
                // loads of unit i: eight rows an instruction
                const uint32_t mine = (uint32_t)(r8 * D + q4 * 16);
                auto load = [&](const uint8_t *pool, int i, const int (&id)[2], uint4 (&x)[kLoads]) {
                    const int t = t_item + (i << kUnitLog2);
                    const uint8_t *src[2];
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch)
                        src[ch] = pool + ((((size_t)max(id[ch], 0) * c.Hkv + k.h) << c.page_log2) + ((t + 16 * ch) & (c.page - 1))) * D + mine;
                    if (id[0] >= 0 && id[1] >= 0 && t >= k.r.lo && t + 32 <= k.r.hi) {
#pragma unroll
                        for (int j = 0; j < kLoads; ++j) {
                            const int grp = j / kHalves, half = j % kHalves;       // eight rows each, two a chunk
                            x[j] = __ldg(reinterpret_cast<const uint4 *>(src[grp >> 1] + (grp & 1) * 8 * D + half * 64));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kLoads; ++j) {
                            const int grp = j / kHalves, half = j % kHalves, row = t + 8 * grp + r8;
                            x[j] = make_uint4(0, 0, 0, 0);      // rows that no query sees, whatever their codes are
                            if (id[grp >> 1] >= 0 && row >= k.r.lo && row < k.r.hi)
                                x[j] = __ldg(reinterpret_cast<const uint4 *>(src[grp >> 1] + (grp & 1) * 8 * D + half * 64));
                        }
                    }
                };
                const uint32_t put0 = operand_at(32 * w + r8, q4 * 2), put1 = operand_at(32 * w + r8, q4 * 2 + 1);
                auto store = [&](uint32_t dst, const uint4 (&x)[kLoads]) {
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        // rows 8 on keep the exchange of chunks, and the second 64 dims are the next atom
                        const uint32_t to = dst + (j / kHalves) * 1024 + (j % kHalves) * 16384;
                        const uint32_t in[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) code_pairs<CODE>(in[e], o[2 * e], o[2 * e + 1]);
                        st128(to + put0, o[0], o[1], o[2], o[3]);
                        st128(to + put1, o[4], o[5], o[6], o[7]);
                    }
                    attn::fence_proxy_async_smem();
                    __syncwarp();
                };
                ChunkConst cc0;
                auto constants = [&] {
                    const float v = vs0 > 0.f ? vs0 : 8.271806e-25f;        // 2^-80, the least: its values are zeros
                    cc0 = id0 >= 0 ? ChunkConst{ks0 * sl, log2f(v), 1.f / v, 0.f} : ChunkConst{0.f, -INFINITY, 0.f, 0.f};
                };
                // a page's two groups of keys; values whose scale is zero are zeros
                int idk[2], idv[2];
                auto ids = [&](int i) {
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        idk[ch] = __shfl_sync(kFull, id0, 2 * (i & 15) + ch);
                        idv[ch] = __shfl_sync(kFull, vs0 > 0.f ? id0 : -1, 2 * (i & 15) + ch);
                    }
                };
                ids(0);
                load(c.k_pool, 0, idk, kr);
                load(c.v_pool, 0, idv, vr);
                constants();
                // keys run one unit ahead of values: unit i's products wait for its keys first
                auto put_keys = [&](int i) {
                    const uint32_t n = n_tile + i, st = n & 1;
                    if (n >= 2) ok = warp_wait(&bar.k_free[st], ((n >> 1) - 1) & 1);
                    if ((lane >> 1) == (i & 15)) consts[n & (kConstSets - 1)][2 * w + (lane & 1)] = cc0;
                    store(sm + L::kK + st * L::kTile, kr);
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&bar.c_full[n & (kConstSets - 1)]));
                        mbar_arrive(smem_addr(&bar.k_full[st]));
                    }
                    if (i + 1 < nu) {
                        if (((i + 1) & 15) == 0) {
                            id0 = id1; ks0 = ks1; vs0 = vs1;
                            fetch(i + 17, id1, ks1, vs1);
                            constants();
                        }
                        ids(i + 1);
                        load(c.k_pool, i + 1, idk, kr);
                    }
                };
                put_keys(0);
                for (int i = 0; i < nu && ok; ++i) {
                    const int idn[2] = {idv[0], idv[1]};                 // of unit i + 1
                    if (i + 1 < nu) put_keys(i + 1);
                    const uint32_t n = n_tile + i, st = n & 1;
                    if (n >= 2) ok = warp_wait(&bar.v_free[st], ((n >> 1) - 1) & 1) && ok;
                    store(sm + L::kV + st * L::kTile, vr);
                    if (lane == 0) mbar_arrive(smem_addr(&bar.v_full[st]));
                    if (i + 1 < nu) load(c.v_pool, i + 1, idn, vr);
                }
                if (!ok) break;
                n_tile += nu;
            } while (cursor_next(a, kUnitLog2, end, &k));
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
            if (warp == 12) {
                constexpr uint32_t kIdS = tc::idesc_f16(kUnit, 0, 0), kIdO = tc::idesc_f16(D, 0, 1);
                const uint64_t dk = tc::sdesc(sm, 16, 1024), dv = tc::sdesc(sm, 16384, 1024);
                // the base is 16-byte units: offsets below 2^14 units never carry out of the field
                auto off = [](uint64_t t, uint32_t bytes) { return t + (uint64_t)(bytes >> 4); };
                auto qk = [&](int sub, uint32_t n) {
                    const uint64_t q = off(dk, L::kQ + sub * L::kTile), kk = off(dk, L::kK + (n & 1) * L::kTile);
                    if (tc::elect()) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            tc::mma_f16(tb + kColS + 128 * sub, off(q, (s >> 2) * 16384 + (s & 3) * 32),
                                        off(kk, (s >> 2) * 16384 + (s & 3) * 32), kIdS, s > 0);
                        tc::commit(smem_addr(&bar.s_full[sub]));
                    }
                    __syncwarp();
                };
                auto pv = [&](int sub, uint32_t n, bool more) {
                    const uint64_t vv = off(dv, L::kV + (n & 1) * L::kTile);
                    if (tc::elect()) {
#pragma unroll
                        for (int s = 0; s < kUnit / 16; ++s)
                            tc::mma_f16_ts(tb + kColO + 128 * sub, tb + kColS + 128 * sub + 8 * s, off(vv, s * 2048), kIdO,
                                           more || s > 0);
                        tc::commit(smem_addr(&bar.o_full[sub]));
                    }
                    __syncwarp();
                };
                auto release = [&](uint64_t *b) {
                    if (tc::elect()) tc::commit(smem_addr(b));
                    __syncwarp();
                };
                do {
                    int u0, nu;
                    cursor_units(k, begin, end, &u0, &nu);
                    if (nu == 0) continue;
                    const int subs = min(a.tile_tokens, k.s.n - k.i0) > sub_tokens ? 2 : 1;
                    ok = warp_wait(&bar.k_full[n_tile & 1], (n_tile >> 1) & 1);
                    for (int s = 0; s < subs && ok; ++s) {
                        ok = warp_wait(&bar.q_ready[s], (s ? n_item1 : n_item) & 1);
                        tc::fence_after();
                        if (ok) qk(s, n_tile);
                    }
                    if (!ok) break;
                    release(&bar.k_free[n_tile & 1]);
                    for (int i = 0; i < nu && ok; ++i) {
                        const uint32_t n = n_tile + i;
                        ok = warp_wait(&bar.v_full[n & 1], (n >> 1) & 1);
                        if (i + 1 < nu) ok = ok && warp_wait(&bar.k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
                        for (int s = 0; s < subs && ok; ++s) {
                            ok = ok && warp_wait(&bar.p_ready[s], ((s ? n_tile1 : n_tile) + i) & 1);
                            if (!ok) break;
                            tc::fence_after();
                            pv(s, n, i > 0);
                            if (s == subs - 1) release(&bar.v_free[n & 1]);
                            if (i + 1 < nu) {
                                qk(s, n + 1);
                            }
                        }
                        if (!ok) break;
                        if (i + 1 < nu) release(&bar.k_free[(n + 1) & 1]);
                    }
                    if (!ok) break;
                    n_tile += nu;
                    n_item += 1;
                    if (subs == 2) { n_tile1 += nu; n_item1 += 1; }
                } while (cursor_next(a, kUnitLog2, end, &k));
                if (!ok) {      // what was issued ends before tensor memory is given back
                    release(&bar.drain);
                    warp_wait(&bar.drain, 0);
                }
            } else {
                // ---- which items the join has to form: the first reader goes through the value scales,
                // all of them through the codes of the keys that not all rows see
                const int reader = warp - 13;
                do {
                    int u0, nu;
                    cursor_units(k, begin, end, &u0, &nu);
                    if (nu == 0) continue;
                    const int t0 = max(k.r.lo, (k.r.tile0 + u0) << kUnitLog2), t1 = min(k.r.hi, (k.r.tile0 + u0 + nu) << kUnitLog2);
                    bool plain = false;
                    if (CODE == TKV_CODE_E4M3) {
                        constexpr int kLanes = D / 16, kStep = 32 * kReaders / kLanes;      // a key's lanes; keys at once
                        const int of = reader * 32 + lane, last = k.r.first + min(a.tile_tokens, k.s.n - k.i0) - 1;
                        auto read = [&](int j0, int j1) {
#pragma unroll 4
                            for (int j = j0 + of / kLanes; j < j1; j += kStep) {
                                uint32_t bad;
                                const int id = load_page(c, a.block_table, k.b, j >> c.page_log2, &bad);
                                if (id < 0) continue;
                                const size_t row = (((size_t)id * c.Hkv + k.h) << c.page_log2) + (j & (c.page - 1));
                                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(c.v_pool + row * D + of % kLanes * 16));
                                plain |= any_nan_code(w.x) || any_nan_code(w.y) || any_nan_code(w.z) || any_nan_code(w.w);
                            }
                        };
                        read(max(t0, k.r.first + 1), t1);
                        if (a.window) read(t0, min(t1, min(last - a.window, k.r.first) + 1));
                    }
                    float least = INFINITY, most = 0.f;
#pragma unroll 4
                    for (int p = reader > 0 ? INT_MAX : (t0 >> c.page_log2) + lane; p < (t1 + c.page - 1) >> c.page_log2; p += 32) {
                        uint32_t bad;
                        const int id = load_page(c, a.block_table, k.b, p, &bad);
                        const float vs = id >= 0 ? c.v_scale[(size_t)id * c.Hkv + k.h] : 0.f;
                        least = fminf(least, vs > 0.f && vs != kLeastScale ? vs : INFINITY);
                        most = fmaxf(most, vs);
                    }
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) {
                        least = fminf(least, __shfl_xor_sync(kFull, least, s));
                        most = fmaxf(most, __shfl_xor_sync(kFull, most, s));
                    }
                    plain = __any_sync(kFull, plain) || most > kScaleSpread * least || most > kScaleMost;
                    if (lane == 0) {
                        if (plain) atomicMin(&plain_from, (int)n_item);
                        store_release(items_read + reader, n_item + 1);
                    }
                    n_item += 1;
                } while (cursor_next(a, kUnitLog2, end, &k));
            }
        }
        if (!ok && lane == 0) raise_error(c.err, kErrTimeout, kWaitTimeout);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (tid == 0 && plain_from != INT_MAX) a.cut[blockIdx.x].plain = plain_from + 1;
    if (warp == 12) tc::dealloc(tb, 512);
}

template <typename T, int D, int CODE, int SETS>
cudaError_t run(AttnArgs a, cudaStream_t st, int *blocks) {
    static int occupancy[kMaxDevices];
    const auto kernel = tiles_kernel<T, D, CODE, SETS>;
    int sms = 0, per_sm = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e == cudaSuccess)
        e = cached_blocks_per_sm(occupancy, reinterpret_cast<const void *>(kernel), kThreads, Layout<D>::kBytes, &per_sm);
    if (e != cudaSuccess) return e;
    *blocks = min(sms, kTileBlocks);
    kernel<<<*blocks, kThreads, Layout<D>::kBytes, st>>>(a);
    return cudaGetLastError();
}
template <typename T, int D, int CODE>
cudaError_t run_page(const AttnArgs &a, cudaStream_t st, int *blocks) {
    return a.c.page >= 64 ? run<T, D, CODE, 2>(a, st, blocks) : run<T, D, CODE, 8>(a, st, blocks);
}
template <typename T>
cudaError_t run_type(const AttnArgs &a, cudaStream_t st, int *blocks) {
    if (a.c.code == TKV_CODE_E4M3)
        return a.c.D == 64 ? run_page<T, 64, TKV_CODE_E4M3>(a, st, blocks) : run_page<T, 128, TKV_CODE_E4M3>(a, st, blocks);
    return a.c.D == 64 ? run_page<T, 64, TKV_CODE_INT8>(a, st, blocks) : run_page<T, 128, TKV_CODE_INT8>(a, st, blocks);
}

}  // namespace

size_t tiles_workspace_bytes(int D) { return 2ull * kTileBlocks * 256 * (D + 2) * sizeof(float); }

cudaError_t launch_tiles(AttnArgs a, cudaStream_t st, int64_t *launches) {
    a.tile_tokens = 2 * (128 / a.c.G);
    a.item_cost = kItemCost;
    int blocks = 0;
    cudaError_t e = a.c.dtype == TKV_DTYPE_BF16 ? run_type<__nv_bfloat16>(a, st, &blocks) : run_type<__half>(a, st, &blocks);
    if (e != cudaSuccess) return e;
    e = launch_join(a, blocks, 256, 128, st);
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace paged
}  // namespace tkv
