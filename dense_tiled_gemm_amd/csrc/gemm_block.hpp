// gemm_block.hpp -- the kernels of the 8-bit product with scales per block of 128
// (declared in epi_kernels.hpp), compiled with linear_back.hip.
#pragma once

#include "dma_kernel.hpp"
#include "epi_kernels.hpp"
#include "skinny_dma.hpp"

namespace gbt {

template <int BM, int BN, int BK, int S, int WM, int WN, int SCHED, int SK, int BLK>
static const void* block_fn() {
    return (const void*)&dma_kernel<GEMM_BT_FP8_E4M3, GEMM_BT_F32, BM, BN, BK, S, WM, WN, 2, SCHED, 0, 32, 0, 0, SK, 0, 1, BLK>;
}
template <int BLK>
static const void* block_fn_of(int tile, bool split) {
    if (split) return tile == 4 ? block_fn<64, 64, 256, 4, 2, 2, 4, 1, BLK>() : nullptr;
    // (widened, with B's scales per row, the larger tiles do not fit the registers)
    switch (tile) {
        case 0:
            if constexpr (BLK != 2 + kBlkWide) return block_fn<256, 128, 128, 3, 4, 2, 8, 0, BLK>();
            return nullptr;
        case 1:
            if constexpr (BLK != 2 + kBlkWide) return block_fn<128, 128, 128, 4, 2, 2, 8, 0, BLK>();
            return nullptr;
        case 2: return block_fn<64, 64, 128, 4, 2, 2, 4, 0, BLK>();
        case 4: return block_fn<64, 64, 256, 4, 2, 2, 4, 0, BLK>();
        default:
            if constexpr (BLK == 1) return block_fn<256, 256, 128, 2, 2, 4, 6, 0, 1>();
            return nullptr;
    }
}
const void* block_dma_fn(int tile, bool tall, bool split, bool wide) {
    if (wide) return tall ? block_fn_of<1 + kBlkWide>(tile, split) : block_fn_of<2 + kBlkWide>(tile, split);
    return tall ? block_fn_of<1>(tile, split) : block_fn_of<2>(tile, split);
}
const void* block_skinny_fn(bool tall, int shape, bool wide) {
    return with_stream(shape, [&](auto c) {
        constexpr StreamShape s = kStream[c()];
        if (wide)
            return tall ? (const void*)&skinny_block_kernel<true, true, s.rows, s.bytes, s.stages>
                        : (const void*)&skinny_block_kernel<false, true, s.rows, s.bytes, s.stages>;
        return tall ? (const void*)&skinny_block_kernel<true, false, s.rows, s.bytes, s.stages>
                    : (const void*)&skinny_block_kernel<false, false, s.rows, s.bytes, s.stages>;
    });
}

}  // namespace gbt
