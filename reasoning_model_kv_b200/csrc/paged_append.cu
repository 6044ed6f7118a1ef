// paged_append.cu -- new keys (encoded on the way) and values into the paged 8-bit cache.
//
// A unit is one (page, kv head) of the keys or of the values: its threads hold the page's
// new rows in registers (four passes of rows, eight elements a lane), find their largest
// magnitude, settle the scale, round what the page held before if the scale grew, and write
// the codes.  So the rows are read once, a scale has one writer and nothing needs an atomic.
// Units of small pages share a block.  The queries' rows are blocks of the same launch.
// Measured: eight prompt chunks (21 thousand tokens, 475 MB) in 102 us = 4.7 TB/s (int8 codes 112), where
// the queries' part streams and the units wait for memory and their barrier (the two kinds of
// blocks in turn were no faster); one token of 64 sequences in 7.5 us (int8 7.7), a chain of
// dependent reads (lengths, page, scale and rows) by 1152 blocks in two rounds.
#include <climits>

#include <cuda_fp8.h>

#include "encode_rows.cuh"
#include "paged_plan.cuh"

namespace tkv {
namespace paged {
namespace {

constexpr int kPasses = 4;

__device__ __forceinline__ void unit_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The smallest power of two s >= 2^-64 with qmax * s >= amax (amax finite).
template <int CODE>
__device__ __forceinline__ float pow2_scale(float amax) {
    // amax = f * 2^e with f in [1/2, 1); qmax = fq * 2^eq; 2^(e - eq), once more if f > fq
    constexpr int eq = CODE == TKV_CODE_E4M3 ? 9 : 7;
    constexpr uint32_t fq = CODE == TKV_CODE_E4M3 ? 0x600000u : 0x7E0000u;   // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
    const uint32_t u = __float_as_uint(amax);
    int x = (int)(u >> 23) - 126 - eq + ((u & 0x7fffffu) > fq ? 1 : 0);
    x = max(x, -64);
    return __uint_as_float((uint32_t)(x + 127) << 23);
}

// Four codes of x, which are values over the scale.
template <int CODE>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    if constexpr (CODE == TKV_CODE_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    } else {
        // (int)NaN is 0, and values beyond 127 only come from infinities
        auto q = [](float x) { return (uint32_t)(int)fminf(fmaxf(x == x ? rintf(x) : 0.f, -127.f), 127.f) & 0xffu; };
        return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
    }
}
template <int CODE>
__device__ __forceinline__ void values4(uint32_t w, float (&x)[4]) {
    if constexpr (CODE == TKV_CODE_E4M3) {
        const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
        const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
        const float2 a = __half22float2(lo), b = __half22float2(hi);
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    }
}

struct AppendArgs {
    View c;
    tkv_rope rope;
    Rows k, v, q, qo;
    const int32_t *block_table, *kv_len, *cu;
    int T, max_new, slots;         // slots: pages that a sequence's new tokens can touch
    uint32_t units, kv_blocks;
    bool compact;                  // units are numbered over the pages that are touched
    int q_groups, q_per;
};

// The rows and length of sequence b; false for padding (*bad 0) and where they cannot be used.
__device__ __forceinline__ bool append_seq(const AppendArgs &a, int b, Seq *s, uint32_t *bad) {
    if (!load_seq(a.cu, a.kv_len, b, a.T, s, bad)) return false;
    if (s->len == 0) return false;
    if (s->n > a.max_new) *bad = kBadRows;
    else if (s->len < s->n) *bad = kBadLen;
    return *bad == 0;
}

// Threads of a unit (UT = page * D / 32) and of a block.
__host__ __device__ constexpr int block_threads(int ut) { return ut > 256 ? ut : 256; }

// Four blocks an SM (64 registers, a few spilled): the units wait for memory and for each other,
// and with three blocks eight prompt chunks took 109 us for 99.
template <typename T, int D, int CODE, int UT>
__global__ void __launch_bounds__(block_threads(UT), UT > 256 ? 2 : 4) append_kernel(const AppendArgs a) {
    constexpr int kBlock = block_threads(UT);
    const View &c = a.c;
    if (blockIdx.x >= a.kv_blocks) {      // the queries
        const uint32_t w = (blockIdx.x - a.kv_blocks) * (kBlock / 32) + (threadIdx.x >> 5);
        const int t = (int)(w / (uint32_t)a.q_groups), lane = threadIdx.x & 31;
        if (t >= a.T) return;
        int b = t;
        if (a.cu) {     // the first sequence that has row t
            b = c.B;
            for (int i = 0; i < c.B && b == c.B; i += 32) {
                const uint32_t has = __ballot_sync(0xffffffffu, i + lane < c.B && a.cu[i + lane] <= t && t < a.cu[i + lane + 1]);
                if (has) b = i + __ffs(has) - 1;
            }
        }
        Seq s;
        uint32_t bad = 0;
        // what is wrong with a sequence is reported by its keys' units
        if (b >= c.B || !append_seq(a, b, &s, &bad) || t < s.row0 || t >= s.row0 + s.n) return;
        const int h0 = (int)(w - (uint32_t)t * a.q_groups) * a.q_per;
        encode_rows<T, D>(a.rope, a.q, Rows{}, a.qo, Rows{}, t, s.len - s.n + (t - s.row0), h0,
                          min(h0 + a.q_per, c.Hkv * c.G), c.Hkv * c.G);
        return;
    }
    __shared__ float red[kBlock / 32];
    constexpr int kUnits = kBlock / UT;
    const int unit_in_block = threadIdx.x / UT, tid = threadIdx.x % UT;
    const uint32_t unit = blockIdx.x * kUnits + unit_in_block;
    const uint32_t nth = unit / (uint32_t)c.Hkv;              // key or value pages before it
    const int h = (int)(unit - nth * c.Hkv);
    const bool values = nth & 1;
    int b, slot;
    if (a.compact) {
        // One sequence is far longer than most: the page that the unit's number stands for, counted
        // over the sequences.
        __shared__ long long warp_sum[kBlock / 32], behind;
        __shared__ int at[kUnits][2];
        if (threadIdx.x < kUnits) at[threadIdx.x][0] = -1;
        const long long first = blockIdx.x * kUnits / (2 * (uint32_t)c.Hkv);
        const long long last = (blockIdx.x * kUnits + kUnits - 1) / (2 * (uint32_t)c.Hkv);
        long long before = 0;
        for (int b0 = 0; b0 < c.B && (before <= last || blockIdx.x == 0); b0 += kBlock) {
            const int mine = b0 + threadIdx.x;
            long long pages = 0;
            if (mine < c.B) {
                Seq s;
                uint32_t bad = 0;
                if (append_seq(a, mine, &s, &bad) && s.n > 0)
                    pages = ((s.len - 1) >> c.page_log2) - ((s.len - s.n) >> c.page_log2) + 1;
                if (bad && blockIdx.x == 0) latch(c, bad);
            }
            const long long end = before + block_scan<kBlock>(pages, warp_sum);
            for (int u = 0; u < kUnits; ++u) {
                const long long j = (blockIdx.x * kUnits + u) / (2 * (uint32_t)c.Hkv);
                if (j >= first && j >= end - pages && j < end) { at[u][0] = mine; at[u][1] = (int)(j - (end - pages)); }
            }
            if (threadIdx.x == kBlock - 1) behind = end;
            __syncthreads();
            before = behind;
            __syncthreads();
        }
        __syncthreads();
        if (unit >= a.units || at[unit_in_block][0] < 0) return;
        b = at[unit_in_block][0];
        slot = at[unit_in_block][1];
    } else {
        if (unit >= a.units) return;
        b = (int)((nth >> 1) / (uint32_t)a.slots);
        slot = (int)((nth >> 1) - (uint32_t)b * a.slots);
    }
    Seq s;
    uint32_t bad = 0;
    if (!append_seq(a, b, &s, &bad)) {
        if (bad && tid == 0 && slot == 0 && h == 0 && !values) latch(c, bad);
        return;
    }
    const int start = s.len - s.n, p = (start >> c.page_log2) + slot;
    const long long first = (long long)p << c.page_log2;      // the page's first token
    if (s.n == 0 || first >= s.len) return;
    const int id = load_page(c, a.block_table, b, p, &bad);
    if (id < 0) {
        if (tid == 0 && h == 0 && !values) latch(c, bad);
        return;
    }
    constexpr int L = D / 8, kRows = UT / L;                  // rows of a pass
    const int j = tid & (L - 1), r0 = tid / L;
    const int lo = max(0, (int)(start - first)), hi = min(c.page, (int)(s.len - first));
    const Rows &x_in = values ? a.v : a.k;
    const Chunks ch = row_chunks(a.rope, j);
    uint2 in0[kPasses], in1[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + r0;
        in0[i] = in1[i] = make_uint2(0, 0);
        if (r >= lo && r < hi) {
            const T *src = static_cast<const T *>(x_in.p) + (s.row0 + (first + r - start)) * x_in.token + h * x_in.head;
            in0[i] = *reinterpret_cast<const uint2 *>(src + ch.a);
            in1[i] = *reinterpret_cast<const uint2 *>(src + ch.b);
        }
    }
    const size_t ps = (size_t)id * c.Hkv + h;
    float *const scale = (values ? c.v_scale : c.k_scale) + ps;
    const float old = lo > 0 ? *scale : 0.f;
    Row8 x[kPasses];
    const bool norm = !values && a.rope.k_weight != nullptr, turn = !values && ch.turns;
    Row8 w{};
    double f[4];
    if (norm) w = load_weights<T>(a.rope.k_weight, ch);
    load_turns(a.rope, j, turn, f);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + r0;
        x[i] = unpack8<T>(in0[i], in1[i]);
        if (i * kRows < hi && (i + 1) * kRows > lo) {        // the same for all the unit's threads
            if (norm) row_norm<D>(x[i], w, a.rope.eps);
            if (turn) row_turn(x[i], turn_angles(f, (int)(first + r)), a.rope.interleaved);
        }
        if (r >= lo && r < hi) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float u, v;
                unpack_f2(x[i].v[e], u, v);
                u = fabsf(u);
                v = fabsf(v);
                amax = fmaxf(amax, u < __int_as_float(0x7f800000) ? u : 0.f);      // finite ones
                amax = fmaxf(amax, v < __int_as_float(0x7f800000) ? v : 0.f);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (UT > 32) {
        if ((tid & 31) == 0) red[threadIdx.x >> 5] = amax;
        unit_sync(1 + unit_in_block, UT);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < UT / 32; ++i) amax = fmaxf(amax, red[unit_in_block * (UT / 32) + i]);
    }
    const float now = fmaxf(pow2_scale<CODE>(amax), old);     // the same in all the unit's threads
    uint8_t *const pool = (values ? c.v_pool : c.k_pool) + ((ps << c.page_log2) * D);
    const float inv = 1.f / now;
    const bool exact = (__float_as_uint(now) & 0x7fffffu) == 0;    // a power of two: 1 / now is exact
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + r0;
        if (r >= hi) continue;
        uint32_t *const c0 = reinterpret_cast<uint32_t *>(pool + r * D + ch.a);
        uint32_t *const c1 = reinterpret_cast<uint32_t *>(pool + r * D + ch.b);
        if (r < lo) {
            if (now == old) continue;
            const float ratio = old / now;
            float y[4], z[4];
            values4<CODE>(*c0, y);
            values4<CODE>(*c1, z);
            *c0 = codes4<CODE>(y[0] * ratio, y[1] * ratio, y[2] * ratio, y[3] * ratio);
            *c1 = codes4<CODE>(z[0] * ratio, z[1] * ratio, z[2] * ratio, z[3] * ratio);
        } else {
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) unpack_f2(x[i].v[e], y[2 * e], y[2 * e + 1]);
            if (exact) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= inv;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] /= now;
            }
            *c0 = codes4<CODE>(y[0], y[1], y[2], y[3]);
            *c1 = codes4<CODE>(y[4], y[5], y[6], y[7]);
        }
    }
    // every thread of the unit has read the old scale before the barrier above (or is of the
    // one warp that read it together)
    if constexpr (UT == 32) __syncwarp();
    if (tid == 0) *scale = now;
}

template <typename T, int D, int CODE, int UT>
cudaError_t run(AppendArgs a, cudaStream_t st) {
    constexpr int kBlock = block_threads(UT);
    const long long per = kBlock / UT;
    // Every sequence may have `slots` pages; all together touch at most T / page + 2 B.  256 sequences of 1
    // to 2000 new tokens and pages of 16 (6 times as many) take 178 us counted, 215 not; eight prompt
    // chunks (1.6 times) 105.5 and 101.8; short prompts (3 times) 12.0 either way.
    const long long every = (long long)a.c.B * a.slots, touched = (long long)(a.T >> a.c.page_log2) + 2ll * a.c.B;
    a.compact = every > 4 * touched;
    const long long units = 2 * (a.compact ? touched : every) * a.c.Hkv, kv_blocks = (units + per - 1) / per;
    long long q_blocks = 0;
    if (a.q.p != nullptr) {
        const int heads = a.c.Hkv * a.c.G;
        a.q_per = heads_per_warp<D>(a.T, heads);
        a.q_groups = (heads + a.q_per - 1) / a.q_per;
        q_blocks = ((long long)a.T * a.q_groups + kBlock / 32 - 1) / (kBlock / 32);
    }
    if (units > INT_MAX || kv_blocks + q_blocks > INT_MAX / (kBlock / 32)) return cudaErrorInvalidValue;
    a.units = (uint32_t)units;
    a.kv_blocks = (uint32_t)kv_blocks;
    append_kernel<T, D, CODE, UT><<<(unsigned)(kv_blocks + q_blocks), kBlock, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T, int D, int CODE>
cudaError_t run_page(const AppendArgs &a, cudaStream_t st) {
    switch (a.c.page) {
        case 16: return run<T, D, CODE, 16 * D / 32>(a, st);
        case 32: return run<T, D, CODE, 32 * D / 32>(a, st);
        case 64: return run<T, D, CODE, 64 * D / 32>(a, st);
        default: return run<T, D, CODE, 128 * D / 32>(a, st);
    }
}
template <typename T>
cudaError_t run_type(const AppendArgs &a, cudaStream_t st) {
    if (a.c.code == TKV_CODE_E4M3)
        return a.c.D == 64 ? run_page<T, 64, TKV_CODE_E4M3>(a, st) : run_page<T, 128, TKV_CODE_E4M3>(a, st);
    return a.c.D == 64 ? run_page<T, 64, TKV_CODE_INT8>(a, st) : run_page<T, 128, TKV_CODE_INT8>(a, st);
}

}  // namespace

cudaError_t launch_append(const View &c, const tkv_rope &rope, Rows k, Rows v, Rows q, Rows qo, int T,
                          const int32_t *block_table, const int32_t *kv_len, const int32_t *cu, int max_new,
                          cudaStream_t st, int64_t *launches) {
    AppendArgs a{};
    a.c = c;
    a.rope = rope;
    a.k = k; a.v = v; a.q = q; a.qo = qo;
    a.block_table = block_table; a.kv_len = kv_len; a.cu = cu;
    a.T = T; a.max_new = max_new;
    // max_new tokens that begin at a page's last slot
    a.slots = (int)(((long long)max_new + 2 * c.page - 2) >> c.page_log2);
    const cudaError_t e = c.dtype == TKV_DTYPE_BF16 ? run_type<__nv_bfloat16>(a, st) : run_type<__half>(a, st);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace paged
}  // namespace tkv
