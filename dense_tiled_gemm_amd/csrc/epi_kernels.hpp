// epi_kernels.hpp -- the kernels with an epilogue, compiled in gemm_epi.hip and
// launched by gemm_bt.hip.
#pragma once

#include "epilogue.hpp"

namespace gbt {

// The twin of dma_variants()[variant] for inputs of in_dtype with an epilogue,
// or of its split form; nullptr where there is none.  Any output type.
const void* epi_dma_fn(int variant, int in_dtype, bool split);
// The streaming kernel for M <= 16 (the first of skinny_variants()).
const void* epi_skinny_fn(int in_dtype);
// K == 0: (void* C, int M, int N, EpiArgs), a grid of any size.
const void* epi_fill_fn();

// The same epilogue for the rows from m1 on of a product with N columns.
inline EpiArgs epi_rows(EpiArgs e, int64_t m1, int64_t N) {
    if (e.row_scale) e.row_scale += m1;
    if (e.residual) e.residual = (const char*)e.residual + m1 * N * elem_size(epi_type(e.mode, EPI_RESIDUAL_TYPE));
    if (e.preact) e.preact = (char*)e.preact + m1 * N * elem_size(epi_type(e.mode, EPI_PREACT_TYPE));
    return e;
}

}  // namespace gbt
