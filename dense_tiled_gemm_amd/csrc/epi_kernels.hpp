// epi_kernels.hpp -- the kernels with an epilogue, compiled in gemm_epi.hip and
// launched by gemm_bt.hip.
#pragma once

#include "epilogue.hpp"

namespace gbt {

// The twin of dma_variants()[variant] for inputs of in_dtype with an epilogue
// (the gated one), or of its split form; nullptr where there is none.  Any output
// type.
const void* epi_dma_fn(int variant, int in_dtype, bool split, bool gated);
// The streaming kernel for M <= 16 (the first of skinny_variants()).
const void* epi_skinny_fn(int in_dtype, bool gated);
// K == 0: (void* C, int M, int N, EpiArgs), a grid of any size.
const void* epi_fill_fn(bool gated);

// The 8-bit product with scales per block of 128: tiles of blockTile(i) with B's
// scales per 128 rows (tall) or per row, their split form, and the streaming
// kernel for M <= 16.
constexpr int kBlockTiles = 5;
struct BlockTile {
    int bm, bn, bk, threads, stages;
};
constexpr BlockTile kBlockTile[kBlockTiles] = {
    {256, 128, 128, 512, 3}, {128, 128, 128, 256, 4}, {64, 64, 128, 256, 4}, {256, 256, 128, 512, 2}, {64, 64, 256, 256, 4}};  // (3: tall alone)
const void* block_dma_fn(int tile, bool tall, bool split);
const void* block_skinny_fn(bool tall);

// The same epilogue for the rows from m1 on, N columns each (of the kept
// pre-activation, where it is gated).
inline EpiArgs epi_rows(EpiArgs e, int64_t m1, int64_t N) {
    if (e.row_scale) e.row_scale += m1;
    if (e.residual) e.residual = (const char*)e.residual + m1 * N * elem_size(epi_type(e.mode, EPI_RESIDUAL_TYPE));
    if (e.preact) e.preact = (char*)e.preact + m1 * N * elem_size(epi_type(e.mode, EPI_PREACT_TYPE));
    return e;
}

}  // namespace gbt
