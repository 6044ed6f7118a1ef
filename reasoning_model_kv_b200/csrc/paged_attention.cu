// paged_attention.cu -- attention over the paged 8-bit cache: the choice of the kernel and the
// workspace.
#include <algorithm>

#include "paged.cuh"
#include "paged_attention.cuh"

namespace tkv {
namespace paged {

size_t attention_workspace_bytes(const tkv_paged_config &cfg) {
    return kArrivedBytes + kCutBytes + std::max(rows_workspace_bytes(cfg.D), tiles_workspace_bytes(cfg.D));
}

size_t attention_reset_bytes() { return kArrivedBytes; }

cudaError_t launch_attention(const View &c, Rows q, Rows out, int T, const int32_t *block_table,
                             const int32_t *kv_len, const int32_t *cu, int max_q, int window, float scale,
                             cudaStream_t st, int64_t *launches) {
    AttnArgs a{};
    a.c = c; a.q = q; a.out = out;
    a.block_table = block_table; a.kv_len = kv_len; a.cu = cu;
    a.T = T;
    // a window as long as the longest sequence hides nothing; positions less a shorter one stay
    // within 32 bits
    a.window = window >= kMaxLen ? 0 : window;
    a.room = c.max_pages * c.page;
    a.scale_log2 = scale * kLog2e;
    a.arrived = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(c.err) + 256);
    a.cut = reinterpret_cast<CutItem *>(reinterpret_cast<uint8_t *>(a.arrived) + kArrivedBytes);
    a.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.cut) + kCutBytes);
    // Query rows a kv head, us on 16 sequences of 4 to 8k tokens of 128 (64) dims:
    //           8        16       24       32       40        64        128       256
    //   rows    50 (32)  62 (41)  76       97 (66)  158 (109) 160 (110) 289 (200) 548
    //   tiles  118 (88) 120 (88) 121      122 (90)  123 (90)  125 (92)  132 (96)  165
    // and 33 rows on 1000 tokens 25 and 17.
    const long long rows = (long long)c.G * std::min(cu ? max_q : 1, T);
    if (rows > 32) return launch_tiles(a, st, launches);
    return launch_rows(a, rows, st, launches);
}

}  // namespace paged
}  // namespace tkv
