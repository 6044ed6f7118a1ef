// paged_attention.cuh -- the kernels that tkv_paged_attention chooses from.
#pragma once

#include "paged_plan.cuh"

namespace tkv {
namespace paged {

constexpr int kMaxBlocks = 1024;                       // blocks of a resident grid
constexpr size_t kArrivedBytes = kMaxBlocks * sizeof(uint32_t);
constexpr int kPartRows = 160 * 64;                    // blocks * rows of an item, at most

// Up to 32 rows an item: keys and values from shared memory into registers, converted there,
// warp matrix instructions (paged_attention_rows.cu).
size_t rows_workspace_bytes(int D);
cudaError_t launch_rows(AttnArgs a, long long rows, cudaStream_t st);

}  // namespace paged
}  // namespace tkv
