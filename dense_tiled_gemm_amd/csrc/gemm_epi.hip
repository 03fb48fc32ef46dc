// gemm_epi.hip -- the product kernels with an epilogue: scales, bias,
// activation and residual applied to the fp32 sums inside the kernel
// (epilogue.hpp).  Every tile shape and schedule is that of the plain product
// (dma_variants() in gemm_bt.hip, by the same index), so one plan serves both.
#include "dma_kernel.hpp"
#include "epi_kernels.hpp"
#include "skinny_dma.hpp"

namespace gbt {

// The fp32 accumulators reach the epilogue unrounded, so the kernels differ
// by input type only (int8: int32 sums).
template <int IN>
constexpr int acc_type() {
    return IN == GEMM_BT_INT8 ? GEMM_BT_INT32 : GEMM_BT_F32;
}

template <int IN, int BM, int BN, int BK, int S, int WM, int WN, int SCHED, int MF, int RING5 = 0, int SK = 0, int PH = 0>
static const void* epi_fn() {
    return (const void*)&dma_kernel<IN, acc_type<IN>(), BM, BN, BK, S, WM, WN, 2, SCHED, 0, MF, 0, RING5, SK, PH, 1>;
}

template <int IN>
static const void* epi_fn16(int variant, bool split) {
    if (split) switch (variant) {
            case 1: return epi_fn<IN, 128, 128, 64, 4, 2, 2, 8, 16, 0, 1>();
            case 10: return epi_fn<IN, 64, 64, 128, 4, 2, 2, 4, 16, 0, 1>();
            case 11: return epi_fn<IN, 32, 64, 128, 4, 2, 2, 2, 16, 0, 1>();
            case 12: return epi_fn<IN, 128, 128, 64, 4, 2, 2, 8, 16, 0, 1, 1>();
            default: return nullptr;
        }
    switch (variant) {
        case 0: return epi_fn<IN, 256, 256, 64, 2, 2, 4, 6, 16, 2>();
        case 1: return epi_fn<IN, 128, 128, 64, 4, 2, 2, 8, 16>();
        case 2: return epi_fn<IN, 64, 64, 64, 4, 2, 2, 4, 16>();
        case 6: return epi_fn<IN, 32, 64, 64, 4, 2, 2, 2, 16>();
        case 7: return epi_fn<IN, 128, 256, 64, 3, 2, 4, 8, 16>();
        case 8: return epi_fn<IN, 96, 128, 64, 4, 2, 2, 6, 16>();
        case 9: return epi_fn<IN, 128, 96, 64, 4, 2, 2, 6, 16>();
        case 12: return epi_fn<IN, 128, 128, 64, 4, 2, 2, 8, 16, 0, 0, 1>();
        case 13: return epi_fn<IN, 96, 128, 64, 4, 2, 2, 6, 16, 0, 0, 1>();
        case 14: return epi_fn<IN, 128, 96, 64, 4, 2, 2, 6, 16, 0, 0, 1>();
        case 15: return epi_fn<IN, 64, 64, 64, 4, 2, 2, 4, 16, 0, 0, 1>();
        default: return nullptr;
    }
}

template <int IN>
static const void* epi_fn8(int variant, bool split) {
    if (split) return variant == 16 ? epi_fn<IN, 64, 64, 256, 4, 2, 2, 4, 32, 0, 1>() : nullptr;
    switch (variant) {
        case 3: return epi_fn<IN, 256, 256, 128, 2, 2, 4, 6, 32, 2>();
        case 4: return epi_fn<IN, 128, 128, 128, 4, 2, 2, 8, 32>();
        case 5: return epi_fn<IN, 64, 64, 128, 4, 2, 2, 4, 32>();
        default: return nullptr;
    }
}

const void* epi_dma_fn(int variant, int in_dtype, bool split) {
    switch (in_dtype) {
        case GEMM_BT_BF16: return epi_fn16<GEMM_BT_BF16>(variant, split);
        case GEMM_BT_F16: return epi_fn16<GEMM_BT_F16>(variant, split);
        case GEMM_BT_FP8_E4M3: return epi_fn8<GEMM_BT_FP8_E4M3>(variant, split);
        case GEMM_BT_FP8_E5M2: return epi_fn8<GEMM_BT_FP8_E5M2>(variant, split);
        case GEMM_BT_INT8: return epi_fn8<GEMM_BT_INT8>(variant, split);
        default: return nullptr;
    }
}

const void* epi_skinny_fn(int in_dtype) {
    switch (in_dtype) {  // 512 bytes of K per row and stage
        case GEMM_BT_BF16: return (const void*)&skinny_epi_kernel<GEMM_BT_BF16, 8, 256, 3, 1>;
        case GEMM_BT_F16: return (const void*)&skinny_epi_kernel<GEMM_BT_F16, 8, 256, 3, 1>;
        case GEMM_BT_FP8_E4M3: return (const void*)&skinny_epi_kernel<GEMM_BT_FP8_E4M3, 8, 512, 3, 1>;
        case GEMM_BT_FP8_E5M2: return (const void*)&skinny_epi_kernel<GEMM_BT_FP8_E5M2, 8, 512, 3, 1>;
        case GEMM_BT_INT8: return (const void*)&skinny_epi_kernel<GEMM_BT_INT8, 8, 512, 3, 1>;
        default: return nullptr;
    }
}

// K == 0: the epilogue of empty sums.
__global__ void epi_fill_kernel(void* C, int M, int N, const EpiArgs e) {
    const size_t n = (size_t)M * N, stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride)
        store_epi4({0.0f, 0.0f, 0.0f, 0.0f}, load_epi4(N, i / N, (int)(i % N), 1, e), C, N, i / N, (int)(i % N), 1, e);
}

const void* epi_fill_fn() { return (const void*)&epi_fill_kernel; }

}  // namespace gbt
