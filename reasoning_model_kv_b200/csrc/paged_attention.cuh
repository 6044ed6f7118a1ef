// paged_attention.cuh -- the kernels that tkv_paged_attention chooses from.
#pragma once

#include "paged_plan.cuh"

namespace tkv {
namespace paged {

constexpr int kMaxBlocks = 1024;                       // blocks of a resident grid
constexpr size_t kArrivedBytes = kMaxBlocks * sizeof(uint32_t);
constexpr size_t kCutBytes = kMaxBlocks * sizeof(CutItem);
constexpr int kPartRows = 160 * 64;                    // blocks * rows of an item, at most

// Up to 32 rows an item: keys and values from shared memory into registers, converted there,
// warp matrix instructions (paged_attention_rows.cu).
size_t rows_workspace_bytes(int D);
cudaError_t launch_rows(AttnArgs a, long long rows, cudaStream_t st, int64_t *launches);

// More rows: up to 256 an item, tcgen05 matrix instructions (paged_attention_tiles.cu).
constexpr int kTileBlocks = 160;                       // blocks of its grid at most
constexpr int kTileUnitLog2 = 7;                       // its units: 128 keys
size_t tiles_workspace_bytes(int D);
cudaError_t launch_tiles(AttnArgs a, cudaStream_t st, int64_t *launches);

// Joins the partial results of every block's cut item, and forms the rows of items that a block has
// marked (paged_join.cu).  Row of token t and head
// g in a partial result: item_rows rows in tiles of tile_rows.
cudaError_t launch_join(const AttnArgs &a, int blocks, int item_rows, int tile_rows, cudaStream_t st);

}  // namespace paged
}  // namespace tkv
