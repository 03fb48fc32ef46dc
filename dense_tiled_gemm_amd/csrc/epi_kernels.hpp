// epi_kernels.hpp -- the kernels with an epilogue, compiled in gemm_epi.hip and
// launched by gemm_bt.hip.
#pragma once

#include <algorithm>

#include "epilogue.hpp"

namespace gbt {

// The twin of dma_variants()[variant] for inputs of in_dtype with an epilogue
// (the gated one), or of its split form; nullptr where there is none.  Any output
// type.
const void* epi_dma_fn(int variant, int in_dtype, bool split, bool gated);
// The streaming kernel for M <= 16 (the first of skinny_variants()), and the gated
// one in the shape kStream[shape].
const void* epi_skinny_fn(int in_dtype);
const void* gated_skinny_fn(int in_dtype, int shape);

// Shapes of the streaming kernels for M <= 16: rows of B per workgroup, bytes of
// each per stage, stages, and how many workgroups a CU holds.
struct StreamShape {
    int rows, bytes, stages, per_cu;
    double step;  // us per 1000 bytes of a row where latency bounds
};
constexpr int kStreams = 3;
constexpr StreamShape kStream[kStreams] = {{8, 512, 3, 4, 1.55}, {16, 256, 3, 6, 1.92}, {16, 512, 2, 4, 2.2}};

// f(std::integral_constant<int, i>{}) for the shape kStream[i]
template <class F>
inline const void* with_stream(int shape, F&& f) {
    switch (shape) {
        case 0: return f(std::integral_constant<int, 0>{});
        case 1: return f(std::integral_constant<int, 1>{});
        default: return f(std::integral_constant<int, 2>{});
    }
}

// The shape with the shortest estimate for `rows` rows of `bytes` each.  Workgroups
// that fill the CUs stream a round of rows at HBM's rate (5.1 TB/s; the first
// shape, with the fewest rows in flight, 4.1); a round that does not takes 4 us and
// the latencies of its stages if that is longer.  Measured (us, E4M3 with scales per block,
// the three shapes): 8192 rows of 8192 bytes 17.8, 19.5, 22.3; 12288 32.0, 20.5,
// 24.2; 16384 32.8, 26.4, 26.6; 24576 48.4, 40.0, 45.4; 32768 64.7, 58.9, 49.8; 65536
// 131, 105, 98.5; 24576 rows of 2048 19.1, 11.5, 16.5; 16384 of 16384 59.2, 54.9, 47.3.
inline int pick_stream(int64_t rows, int64_t bytes, int num_cu) {
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < kStreams; ++i) {
        const StreamShape& s = kStream[i];
        const int64_t round = (int64_t)num_cu * s.per_cu * s.rows;
        const double rate = (double)bytes / (i == 0 ? 4.1e6 : 5.1e6);  // us a row
        const int64_t rest = rows % round;
        double t = (double)(rows / round * round) * rate;
        if (rest) t += std::max((double)rest * rate, 4.0 + s.step * (double)bytes * 1e-3);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}
// K == 0: (void* C, int M, int N, EpiArgs), a grid of any size.
const void* epi_fill_fn(bool gated);

// The 8-bit product with scales per block of 128: tiles of kBlockTile[i] with B's
// scales per 128 rows (tall) or per row, their split form, and the streaming
// kernel for M <= 16.
constexpr int kBlockTiles = 5;
struct BlockTile {
    int bm, bn, bk, threads, stages;
};
constexpr BlockTile kBlockTile[kBlockTiles] = {
    {256, 128, 128, 512, 3}, {128, 128, 128, 256, 4}, {64, 64, 128, 256, 4}, {256, 256, 128, 512, 2}, {64, 64, 256, 256, 4}};  // (3: tall and not wide alone)
// `wide`: for fp32 results (kBlkWide).
const void* block_dma_fn(int tile, bool tall, bool split, bool wide);
const void* block_skinny_fn(bool tall, int shape, bool wide);

// The same epilogue for the rows from m1 on, N columns each (of the kept
// pre-activation, where it is gated).
inline EpiArgs epi_rows(EpiArgs e, int64_t m1, int64_t N) {
    if (e.row_scale) e.row_scale += m1;
    if (e.residual) e.residual = (const char*)e.residual + m1 * N * elem_size(epi_type(e.mode, EPI_RESIDUAL_TYPE));
    if (e.preact) e.preact = (char*)e.preact + m1 * N * elem_size(epi_type(e.mode, EPI_PREACT_TYPE));
    return e;
}

}  // namespace gbt
