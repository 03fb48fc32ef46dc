// gemm_epi.hip -- the product kernels with an epilogue: scales, bias,
// activation and residual applied to the fp32 sums inside the kernel
// (epilogue.hpp).  Every tile shape and schedule is that of the plain product
// (dma_variants() in gemm_bt.hip, by the same index), so one plan serves both.
// The gated twins (EPI = 2) run the plan of the product with 2 N columns.
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

template <int IN, int EPI, int BM, int BN, int BK, int S, int WM, int WN, int SCHED, int MF, int RING5 = 0, int SK = 0, int PH = 0>
static const void* epi_fn() {
    return (const void*)&dma_kernel<IN, acc_type<IN>(), BM, BN, BK, S, WM, WN, 2, SCHED, 0, MF, 0, RING5, SK, PH, EPI>;
}

template <int IN, int EPI>
static const void* epi_fn16(int variant, bool split) {
    if (split) switch (variant) {
            case 1: return epi_fn<IN, EPI, 128, 128, 64, 4, 2, 2, 8, 16, 0, 1>();
            case 10: return epi_fn<IN, EPI, 64, 64, 128, 4, 2, 2, 4, 16, 0, 1>();
            case 11: return epi_fn<IN, EPI, 32, 64, 128, 4, 2, 2, 2, 16, 0, 1>();
            case 12: return epi_fn<IN, EPI, 128, 128, 64, 4, 2, 2, 8, 16, 0, 1, 1>();
            default: return nullptr;
        }
    switch (variant) {
        case 0: return epi_fn<IN, EPI, 256, 256, 64, 2, 2, 4, 6, 16, 2>();
        case 1: return epi_fn<IN, EPI, 128, 128, 64, 4, 2, 2, 8, 16>();
        case 2: return epi_fn<IN, EPI, 64, 64, 64, 4, 2, 2, 4, 16>();
        case 6: return epi_fn<IN, EPI, 32, 64, 64, 4, 2, 2, 2, 16>();
        case 7: return epi_fn<IN, EPI, 128, 256, 64, 3, 2, 4, 8, 16>();
        case 8: return epi_fn<IN, EPI, 96, 128, 64, 4, 2, 2, 6, 16>();
        case 9: return epi_fn<IN, EPI, 128, 96, 64, 4, 2, 2, 6, 16>();
        case 12: return epi_fn<IN, EPI, 128, 128, 64, 4, 2, 2, 8, 16, 0, 0, 1>();
        case 13: return epi_fn<IN, EPI, 96, 128, 64, 4, 2, 2, 6, 16, 0, 0, 1>();
        case 14: return epi_fn<IN, EPI, 128, 96, 64, 4, 2, 2, 6, 16, 0, 0, 1>();
        case 15: return epi_fn<IN, EPI, 64, 64, 64, 4, 2, 2, 4, 16, 0, 0, 1>();
        default: return nullptr;
    }
}

template <int IN, int EPI>
static const void* epi_fn8(int variant, bool split) {
    if (split) return variant == 16 ? epi_fn<IN, EPI, 64, 64, 256, 4, 2, 2, 4, 32, 0, 1>() : nullptr;
    switch (variant) {
        case 3: return epi_fn<IN, EPI, 256, 256, 128, 2, 2, 4, 6, 32, 2>();
        case 4: return epi_fn<IN, EPI, 128, 128, 128, 4, 2, 2, 8, 32>();
        case 5: return epi_fn<IN, EPI, 64, 64, 128, 4, 2, 2, 4, 32>();
        default: return nullptr;
    }
}

template <int EPI>
static const void* fn_of(int variant, int in_dtype, bool split) {
    switch (in_dtype) {
        case GEMM_BT_BF16: return epi_fn16<GEMM_BT_BF16, EPI>(variant, split);
        case GEMM_BT_F16: return epi_fn16<GEMM_BT_F16, EPI>(variant, split);
        case GEMM_BT_FP8_E4M3: return epi_fn8<GEMM_BT_FP8_E4M3, EPI>(variant, split);
        case GEMM_BT_FP8_E5M2: return epi_fn8<GEMM_BT_FP8_E5M2, EPI>(variant, split);
        case GEMM_BT_INT8: return epi_fn8<GEMM_BT_INT8, EPI>(variant, split);
        default: return nullptr;
    }
}
const void* epi_dma_fn(int variant, int in_dtype, bool split, bool gated) {
    return gated ? fn_of<2>(variant, in_dtype, split) : fn_of<1>(variant, in_dtype, split);
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

template <int IN>
static const void* gated_of(int shape) {
    return with_stream(shape, [](auto c) {
        constexpr StreamShape s = kStream[c()];
        return (const void*)&skinny_gated_kernel<IN, s.rows, s.bytes / in_size(IN), s.stages, 1>;
    });
}
const void* gated_skinny_fn(int in_dtype, int shape) {
    switch (in_dtype) {
        case GEMM_BT_BF16: return gated_of<GEMM_BT_BF16>(shape);
        case GEMM_BT_F16: return gated_of<GEMM_BT_F16>(shape);
        case GEMM_BT_FP8_E4M3: return gated_of<GEMM_BT_FP8_E4M3>(shape);
        case GEMM_BT_FP8_E5M2: return gated_of<GEMM_BT_FP8_E5M2>(shape);
        case GEMM_BT_INT8: return gated_of<GEMM_BT_INT8>(shape);
        default: return nullptr;
    }
}

// K == 0: the epilogue of empty sums.
__global__ void epi_fill_kernel(void* C, int M, int N, const EpiArgs e) {
    const size_t n = (size_t)M * N, stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride)
        store_epi4({0.0f, 0.0f, 0.0f, 0.0f}, load_epi4(N, i / N, (int)(i % N), 1, e), C, N, i / N, (int)(i % N), 1, e);
}

// The gated one: act(bias) times the bias of the second half.
__global__ void gated_fill_kernel(void* C, int M, int N, const EpiArgs e) {
    const size_t n = (size_t)M * N, stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
        const size_t row = i / N, col = i % N;
        const int t = epi_type(e.mode, EPI_BIAS_TYPE), zt = epi_type(e.mode, EPI_PREACT_TYPE);
        float gate = e.mode & EPI_BIAS ? load1(e.bias, t, col) : 0.0f;
        const float up = e.mode & EPI_BIAS ? load1(e.bias, t, N + col) : 0.0f;
        if (e.mode & EPI_PREACT) {
            store1(e.preact, zt, 2 * row * N + col, gate);
            store1(e.preact, zt, (2 * row + 1) * N + col, up);
        }
        with_act(e.mode >> EPI_ACT, [&](auto act) __attribute__((always_inline)) { gate = act_value<decltype(act)::value>(gate); });
        store1(C, epi_type(e.mode, EPI_OUT_TYPE), i, gate * up);
    }
}

const void* epi_fill_fn(bool gated) { return gated ? (const void*)&gated_fill_kernel : (const void*)&epi_fill_kernel; }

}  // namespace gbt
