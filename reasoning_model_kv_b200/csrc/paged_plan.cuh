// paged_plan.cuh -- the split of the paged attention's work over a resident grid.
//
// An item is one (sequence, kv head, tile of query tokens); its units are the tiles of keys
// that its rows can see, at least one.  All items' units lie on one line, sequence by
// sequence, and every block takes an equal stretch of it: ragged lengths, long sequences and
// small batches all end up balanced without the host knowing a length.  Before its units an
// item has `item_cost` places on the line that stand for its setup (queries, page table, first
// copies, output).  An item whose units are cut leaves partial results (running maximum, sum,
// unnormalised output), which are joined in block order whichever block arrives last.
#pragma once

#include "attn_common.cuh"
#include "paged.cuh"

namespace tkv {
namespace paged {

// What a block leaves to the join: the item that begins in its stretch and goes on in the next
// blocks', and where the items begin whose rows the join has to form by itself.
struct CutItem {
    int row0, head0;
    int16_t tokens;
    int16_t parts;          // blocks that hold a part; below 2: no such item
    int plain;              // 1 + number of the block's first such item (0: none)
};

struct AttnArgs {
    View c;
    Rows q, out;
    const int32_t *block_table, *kv_len, *cu;
    int T, window;
    int room;               // tokens that a row of the block table has pages for
    float scale_log2;       // softmax_scale * log2(e)
    int tile_tokens;        // query tokens of an item
    int item_cost;          // an item's setup in units
    float *part;            // [blocks][2][rows * (D + 2)] partial results: of the item that a
                            // block goes on with, of the one that it begins
    uint32_t *arrived;      // [blocks] blocks that have left their part of the item that begins here
    CutItem *cut;           // [blocks]
};

// Key range of query tokens [i0, i1) of a sequence, and its tiles of `unit` keys.  It ends with
// the block table: a length beyond it (the plan latches it) adds no units, so an item has no more
// of them than the table has room for.
struct KeyRange {
    int first, lo, hi;      // position of token i0; keys [lo, hi) are seen by some row
    int tile0, units;       // units >= 1
};
__device__ __forceinline__ KeyRange key_range(const AttnArgs &a, const Seq &s, int i0, int unit_log2) {
    KeyRange r;
    const int i1 = min(i0 + a.tile_tokens, s.n);
    r.first = s.len - s.n + i0;
    r.hi = min(max(0, s.len - s.n + i1), a.room);
    r.lo = a.window ? max(0, r.first - a.window + 1) : 0;
    r.tile0 = r.lo >> unit_log2;
    r.units = max(1, ((r.hi + (1 << unit_log2) - 1) >> unit_log2) - r.tile0);
    return r;
}

// a / b for a >= 0, b > 0; nearly always in 32 bits, whose division is a fifth as long.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((unsigned long long)a | (unsigned long long)b) >> 32) return a / b;
    return (long long)((uint32_t)a / (uint32_t)b);
}

// A sequence's rows and length for attention: n = 0 where the rows cannot be used, len = 0
// where the length cannot.
__device__ __forceinline__ Seq attention_seq(const AttnArgs &a, int b, uint32_t *bad) {
    Seq s;
    *bad = 0;
    if (!load_seq(a.cu, a.kv_len, b, a.T, &s, bad)) {
        if (*bad == kBadRows) s.n = 0;
        s.len = 0;
    }
    return s;
}

struct Plan {
    long long warp_sum[32];
    long long total, base;
    int b;                  // sequence in which the block's stretch begins
    long long off;          // units of that sequence before it
};

// Places of one kv head of sequence s on the line.
__device__ __forceinline__ long long head_units(const AttnArgs &a, const Seq &s, int unit_log2) {
    long long u = 0;
    for (int i0 = 0; i0 < s.n; i0 += a.tile_tokens) u += a.item_cost + key_range(a, s, i0, unit_log2).units;
    return u;
}

// Inclusive sum of v over the block's threads, in thread order.
template <int NT>
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sum) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) warp_sum[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v += warp_sum[i];
    return v;
}

// Finds the block's stretch: *share places from *begin on (none if begin >= total), and where
// that is.  Block 0 reports sequences that cannot be used, or whose last token (which their last
// row sees) the block table has no room for.  All NT threads take part.
template <int NT, bool REPORT = true>
__device__ __forceinline__ void make_plan(const AttnArgs &a, Plan &p, int unit_log2, long long *begin, long long *share) {
    const int B = a.c.B, tid = threadIdx.x;
    long long sum = 0, mine = 0;
    for (int b = tid; b < B; b += NT) {
        uint32_t bad;
        const Seq s = attention_seq(a, b, &bad);
        if (!bad && s.n > 0 && s.len > a.room) bad = kNoPage;
        if (REPORT && bad && blockIdx.x == 0) latch(a.c, bad);
        mine = head_units(a, s, unit_log2) * a.c.Hkv;
        sum += mine;
    }
    const long long incl = block_scan<NT>(sum, p.warp_sum);
    if (tid == NT - 1) p.total = incl;
    __syncthreads();
    const long long total = p.total;
    *share = quotient(total + gridDim.x - 1, gridDim.x);
    *begin = *share * blockIdx.x;
    if (B <= NT) {
        if (tid < B && *begin >= incl - sum && *begin < incl) { p.b = tid; p.off = *begin - (incl - sum); }
    } else {
        long long base = 0;
        for (int b0 = 0; b0 < B; b0 += NT) {
            const int b = b0 + tid;
            uint32_t bad;
            const long long u = b < B ? head_units(a, attention_seq(a, b, &bad), unit_log2) * a.c.Hkv : 0;
            const long long in = base + block_scan<NT>(u, p.warp_sum);
            if (*begin >= in - u && *begin < in) { p.b = b; p.off = *begin - (in - u); }
            if (tid == NT - 1) p.base = in;
            __syncthreads();
            base = p.base;
            if (base > *begin) break;
            __syncthreads();
        }
    }
    __syncthreads();
}

// The items along a block's stretch.
struct Cursor {
    int b, h, i0;           // sequence, kv head, first query token
    Seq s;
    KeyRange r;
    long long g0;           // the item's first unit on the line (behind its setup)
};
// Units [u0, u0 + nu) of the cursor's item are in the stretch [begin, end); nu may be 0.
__device__ __forceinline__ void cursor_units(const Cursor &k, long long begin, long long end, int *u0, int *nu) {
    const long long lo = max(begin - k.g0, 0ll), hi = min(end - k.g0, (long long)k.r.units);
    *u0 = (int)lo;
    *nu = (int)max(hi - lo, 0ll);
}

__device__ __forceinline__ void cursor_start(const AttnArgs &a, const Plan &p, long long begin, int unit_log2, Cursor *k) {
    uint32_t bad;
    k->b = p.b;
    k->s = attention_seq(a, k->b, &bad);
    const long long per = head_units(a, k->s, unit_log2);
    k->h = (int)quotient(p.off, per);
    long long off = p.off - k->h * per;
    k->i0 = 0;
    for (;;) {
        k->r = key_range(a, k->s, k->i0, unit_log2);
        if (off < a.item_cost + k->r.units) break;
        off -= a.item_cost + k->r.units;
        k->i0 += a.tile_tokens;
    }
    k->g0 = begin - off + a.item_cost;
}
// The next item; false behind the last one and behind the stretch's end.
__device__ __forceinline__ bool cursor_next(const AttnArgs &a, int unit_log2, long long end, Cursor *k) {
    k->g0 += k->r.units + a.item_cost;
    if (k->g0 >= end) return false;
    k->i0 += a.tile_tokens;
    if (k->i0 >= k->s.n) {
        k->i0 = 0;
        if (++k->h == a.c.Hkv) {
            k->h = 0;
            uint32_t bad;
            do {
                if (++k->b >= a.c.B) return false;
                k->s = attention_seq(a, k->b, &bad);
            } while (k->s.n == 0);
        }
    }
    k->r = key_range(a, k->s, k->i0, unit_log2);
    return true;
}

// The blocks whose stretches hold units of the cursor's item, and where block blk's partial
// result of it is.
struct Parts {
    long long first;
    int count;
};
__device__ __forceinline__ Parts item_parts(const Cursor &k, long long share) {
    const long long first = quotient(k.g0, share);
    return {first, (int)(quotient(k.g0 + k.r.units - 1, share) - first) + 1};
}
__device__ __forceinline__ float *part_at(const AttnArgs &a, size_t floats, long long first, long long blk) {
    return a.part + (size_t)(2 * blk + (blk == first)) * floats;
}

}  // namespace paged
}  // namespace tkv
