// paged_codes.cuh -- the cache's 8-bit codes as fp16 pairs (exact for both code types).
#pragma once

#include "attn_common.cuh"
#include "tkv.h"

namespace tkv {
namespace paged {

// Is one of a word's four codes an E4M3 NaN (all bits but the sign's)?
__device__ __forceinline__ bool any_nan_code(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

// Codes 0, 1 (lo) and 2, 3 (hi) of a word: E4M3 through the hardware's conversion, integers as
// 0x6400 | (code + 128), which is 1024 + 128 + code in fp16, less 1152.
template <int CODE>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (CODE == TKV_CODE_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = attn::u32_as_h2(0x64806480u);
        lo = attn::h2_as_u32(__hsub2(attn::u32_as_h2(__byte_perm(u, 0x64646464u, 0x4140)), bias));
        hi = attn::h2_as_u32(__hsub2(attn::u32_as_h2(__byte_perm(u, 0x64646464u, 0x4342)), bias));
    }
}

}  // namespace paged
}  // namespace tkv
