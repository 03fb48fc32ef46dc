// norm.hip -- the row operators next to the product: root-mean-square norm and
// layer norm with the residual's addition, out in 16 or 32 bits or in 8 bits
// with one scale per row; 8-bit rows with scales of a matrix as it is; the
// norms' backward passes; and the backward pass of an epilogue's activation and
// bias.
//
// All of them are bound by HBM: each reads its inputs once and writes its
// outputs once.  A row is read into registers (8 elements per thread and
// chunk), every statistic is taken from there, and the row leaves from there.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "epilogue.hpp"
#include "rows.hpp"

namespace gbt {

// ---- reductions ----------------------------------------------------------------

struct SumOp {
    __device__ static float zero() { return 0.0f; }
    __device__ static float join(float a, float b) { return a + b; }
};
// largest of the bits of |v|: for finite values the largest magnitude, and
// above every finite value once one of them is infinite or NaN
struct MaxBitsOp {
    __device__ static float zero() { return 0.0f; }
    __device__ static float join(float a, float b) { return as_f32(max(as_u32(a), as_u32(b))); }
};

// The value joined over the threads of a row (WAVE: one wave; else the whole
// workgroup, through `part`), the same for all of them and in an order that
// depends on their number only.
template <class Op, bool WAVE>
__device__ __forceinline__ float row_join(float v, float* part) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = Op::join(v, __shfl_xor(v, m));
    if constexpr (!WAVE) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = Op::zero();
        for (int w = 0; w < (int)blockDim.x >> 6; ++w) v = Op::join(v, part[w]);
    }
    return v;
}

// Layer norm's sums.  Lanes are joined by data-parallel moves of the vector unit
// (a row of 16 lanes, then the rows), a few cycles each where a shuffle goes
// through the LDS unit.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float add_moved(float v) {
    return v + as_f32((u32)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), CTRL, ROWS, 0xF, false));
}
// Lane 15 of each row of 16: the row's sum.
__device__ __forceinline__ float sum16(float v) {
    return add_moved<0x118>(add_moved<0x114>(add_moved<0x112>(add_moved<0x111>(v))));
}
// The sum over a wave, in every lane.
__device__ __forceinline__ float sum64(float v) {
    v = add_moved<0x143, 0xC>(add_moved<0x142, 0xA>(sum16(v)));
    return as_f32((u32)__builtin_amdgcn_readlane((int)as_u32(v), 63));
}
// N sums over the threads of a row at one barrier (at most 16 waves), through N
// rows of `part`, `gap` apart.
template <bool WAVE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[16], int gap) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum64(v[i]);
    if constexpr (!WAVE) {
        const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[i * gap][threadIdx.x >> 6] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = as_f32((u32)__builtin_amdgcn_readlane((int)as_u32(sum16(lane < waves ? part[i * gap][lane & 15] : 0.0f)), 15));
    }
}
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (*part)[16]) {
    float one[1] = {v};
    row_sums<WAVE, 1>(one, part, 0);
    return one[0];
}

// ---- rows in chunks of 8 ---------------------------------------------------------

// Elements i .. i+7 of a row of d that starts at element `base` of p.  RAGGED
// (d >= 8, no multiple of 8): the last chunk is loaded from element d - 8 on and
// moved into place when it is decoded.  WHOLE: every chunk is known to be 8 elements.
// A load is then one instruction for every lane, and nothing waits for it before its
// use, where a branch that put single elements together waits for everything in
// flight.  Rows of whole chunks have kernels without the moves.
template <bool RAGGED, bool WHOLE = false>
__device__ __forceinline__ Raw8 load_chunk(const void* p, int t, long long base, int i, int d, bool nt = false) {
    if constexpr (WHOLE) return load_raw8(p, t, (size_t)base + i, 8, nt);
    if constexpr (RAGGED) return load_raw8(p, t, (size_t)(base + min(i, d - 8)), 8, nt);
    return load_raw8(p, t, (size_t)base + i, min(8, d - i), nt);
}
template <bool RAGGED>
__device__ __forceinline__ void decode_chunk(const Raw8& r, int t, int i, int d, float (&v)[8]) {
    decode8(r, t, v);
    if constexpr (RAGGED) {
        const int k = i + 8 - d;  // v holds k elements before the chunk's first
        if (k > 0)
#pragma unroll
            for (int b = 4; b > 0; b >>= 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = k & b ? (e + b < 8 ? v[e + b] : 0.0f) : v[e];
    }
}

// ---- 8-bit codes ---------------------------------------------------------------

typedef u32x2 u32x2_byte __attribute__((aligned(1)));
typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// Four values (|v| <= 448 or 127 up to rounding, or NaN) in 8 bits, to nearest even.
template <int QT>
__device__ __forceinline__ u32 quant4(float a, float b, float c, float d) {
    if constexpr (QT == GEMM_BT_FP8_E4M3) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (u32)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        // (a NaN becomes -127 in the comparisons: a code without a value, whose row's scale is NaN)
        auto code = [](float v) { return (u32)(int)__builtin_fminf(__builtin_fmaxf(__builtin_rintf(v), -127.0f), 127.0f) & 255u; };
        return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
    }
}
__device__ __forceinline__ void store_codes(void* p, int qt, size_t i, int n, const float (&v)[8]) {
    u32x2 w;
    if (qt == GEMM_BT_FP8_E4M3)
        w = u32x2{quant4<GEMM_BT_FP8_E4M3>(v[0], v[1], v[2], v[3]), quant4<GEMM_BT_FP8_E4M3>(v[4], v[5], v[6], v[7])};
    else
        w = u32x2{quant4<GEMM_BT_INT8>(v[0], v[1], v[2], v[3]), quant4<GEMM_BT_INT8>(v[4], v[5], v[6], v[7])};
    unsigned char* s = (unsigned char*)p + i;
    if (n >= 8) {
        __builtin_nontemporal_store(w, (u32x2_byte*)s);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) s[e] = (unsigned char)(w[e >> 2] >> (8 * (e & 3)));
    }
}

// Rows in 8 bits are taken from t = (h p) w instead of y = h rstd w, p the power
// of two below rstd: t has one rounding where y has two, the factor that y has
// more, rstd / p, is one of the whole row, and codes do not depend on it.
__device__ __forceinline__ float power_below(float rstd) {
    return __builtin_fmaxf(as_f32(as_u32(rstd) & 0x7F800000u), 0x1p-126f);
}

// The scale of a row of values t * rest, and what t is multiplied by for its
// codes, from the largest |t|: scale = amax rest / Q, Q = 448 (E4M3) or 127
// (int8), kept above 2^-100 so that its reciprocal is finite; NaN for a row that
// holds an infinity or a NaN, one that t * rest overflows to included.
struct RowScale {
    float scale, code;
};
__device__ __forceinline__ RowScale row_scale_of(float amax, float rest, int qt) {
    const float q = qt == GEMM_BT_FP8_E4M3 ? 448.0f : 127.0f, nan = as_f32(0x7FC00000u);
    const float top = amax * rest;
    if (as_u32(top) >= 0x7F800000u) return {nan, nan};
    const float s = top / q;
    if (!(s >= 0x1p-100f)) return {0x1p-100f, rest * 0x1p100f};
    return {s, q / amax};
}

// ---- norm and quantisation, forward ----------------------------------------------

// 1 / sqrt(ss / d + eps) of a row whose squares sum to ss in fp32.  Where that
// sum left fp32's range (|h| above 2^64 / sqrt d, or below 2^-45 with next to
// no eps) the squares are summed once more, of the row scaled by a power of
// two that brings its largest magnitude near 1.  each(f) calls f on every
// value of h that the thread holds; `part` has two more rows for the joins.
// An infinity gives 0, a NaN NaN.
template <bool WAVE, class Each>
__device__ __forceinline__ float rstd_of(float ss, int d, float eps, float (*part)[16], int flip, Each&& each) {
    const float mean = ss / (float)d + eps;
    if (__builtin_expect(!(mean > 0x1p-90f && mean < __builtin_inff()), 0)) {
        float amax = 0.0f;
        each([&](float v) __attribute__((always_inline)) { amax = MaxBitsOp::join(amax, __builtin_fabsf(v)); });
        amax = row_join<MaxBitsOp, WAVE>(amax, part[flip]);
        if (amax == 0.0f) return 1.0f / __builtin_sqrtf(eps);  // (of layer norm, whose ss may hold what its mean left out)
        if (amax < __builtin_inff()) {
            const float s = as_f32((254u - min(as_u32(amax) >> 23, 253u)) << 23);
            float sq = 0.0f;
            each([&](float v) __attribute__((always_inline)) { sq = __builtin_fmaf(v * s, v * s, sq); });
            sq = row_join<SumOp, WAVE>(sq, part[2 + flip]);
            const float e = eps * s * s;
            return e < __builtin_inff() ? s / __builtin_sqrtf(sq / (float)d + e) : 1.0f / __builtin_sqrtf(eps);
        }
    }
    return 1.0f / __builtin_sqrtf(mean);
}

struct NormArgs {
    const void* x;
    const void* residual;  // nullptr: none
    const void* weight;    // nullptr: the rows as they are (quantisation alone)
    void* y;
    void* h;               // x + residual rounded, nullptr: not kept
    float* scale;          // 8-bit y
    float* rstd;           // nullptr: not kept
    long long rows, ldx, ldr;
    int d;
    float eps;
    int y_type;
    const void* bias;      // layer norm alone, in weight's type; nullptr: none
    float* mean;           // layer norm alone; nullptr: not kept
};

__host__ __device__ inline bool is_code_type(int t) { return t == GEMM_BT_FP8_E4M3 || t == GEMM_BT_INT8; }

// The mean of a row of d values whose sum in fp32 is `sum`.  Where that, or a part of
// it on the way, left fp32's range the values are summed once more, 2^-27 of each
// (d <= 2^26).  NaN where a value is infinite.
template <bool WAVE, class Each>
__device__ __forceinline__ float mean_of(float sum, int d, float* part, Each&& each) {
    float mean = sum / (float)d;
    if (__builtin_expect(!(__builtin_fabsf(mean) < __builtin_inff()), 0)) {
        float s = 0.0f;
        each([&](float v) __attribute__((always_inline)) { s = __builtin_fmaf(v, 0x1p-27f, s); });
        mean = row_join<SumOp, WAVE>(s, part) / (float)d * 0x1p27f;
        mean += mean - mean;
    }
    return mean;
}

// h = x + residual; y = h rstd w: one pass over x and the residual, whose row
// stays in registers between its statistics and its results.  Bound by HBM:
// 8192 x 8192 bf16 with residual 92 us (5.8 TB/s; a plain copy reaches 5.1),
// to E4M3 83 us, 4096 x 4096 quantised alone 11.4 us; one row of 4096 2.8 us, a
// launch.  Inputs are read through the caches, where the kernel before may have
// left them (8192 x 8192 without residual 43 us against 50 past them).
// The T threads that hold a row, U chunks of 8 elements each (T * U * 8 >= d),
// are a wave (WAVE; a workgroup is up to 4 of them, each with rows of its own) or
// the whole workgroup, of as many waves as the row fills.
// CENTER: layer norm, y = (h - mean) rstd w + b.  The sum of h gives m0; then off,
// the mean of h - m0, which is what the rounding of m0 left out, comes with the
// squares of h - m0, d off^2 above those of h - m0 - off.  So the centred values do
// not depend on how well the first sum came out, and rows of nearly equal entries
// keep what distinguishes them.  Bound by HBM: 8192 x 8192 bf16 with residual 96 us
// (5.6 TB/s), 8192 x 4096 49, 16384 x 1024 23.  Two joins over the row's threads where
// the other norm has one: with shuffles and three barriers they cost 113 us, with
// two 108, with moves in the vector unit (row_sums) 96.
template <int XT, int WT, int U, bool WAVE, bool RAGGED, bool CENTER = false>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(const NormArgs a) {
    constexpr bool WHOLE = !RAGGED && !WAVE;  // every chunk is 8 elements of the row (rows below 8 have a wave each)
    // layer norm of two chunks per thread fetches w and b after the statistics: held
    // through them they cost a third workgroup's registers
    constexpr bool LATE = CENTER && U > 1;
    __shared__ float part[CENTER ? 14 : 8][16];
    const int T = WAVE ? 64 : blockDim.x, RB = WAVE ? blockDim.x >> 6 : 1;
    const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int d = a.d;
    int flip = 0;
    for (long long row = (long long)blockIdx.x * RB + (WAVE ? threadIdx.x >> 6 : 0); row < a.rows;
         row += (long long)gridDim.x * RB) {
        Raw8 xr[U], rr[U], wr[U], br[CENTER ? U : 1];
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                xr[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.x, XT, row * a.ldx, i, d);
                if (a.residual) rr[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.residual, XT, row * a.ldr, i, d);
                if (!LATE && a.weight) wr[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.weight, WT, 0, i, d);
                if constexpr (CENTER && !LATE)
                    if (a.bias) br[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.bias, WT, 0, i, d);
            }
        });
        float h[U][8], ss = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                decode_chunk<RAGGED>(xr[u], XT, i, d, h[u]);
                if (a.residual) {
                    float v[8];
                    decode_chunk<RAGGED>(rr[u], XT, i, d, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[u][e] += v[e];
                }
                if (a.h) store8(a.h, XT, (size_t)(row * d) + i, CENTER && WHOLE ? 8 : min(8, d - i), h[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[u][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = CENTER ? ss + h[u][e] : __builtin_fmaf(h[u][e], h[u][e], ss);
        });
        auto each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) f(h[u][e]);
        };
        if constexpr (CENTER) {
            float sums[2] = {0.0f, 0.0f};
            const float m0 = mean_of<WAVE>(row_sum<WAVE>(ss, part + 8 + flip), d, part[10 + flip], each);
            // (elements past the row's end stay 0)
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int n = d - (u * T + renew(t)) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if ((WHOLE ? 0 : e) < n) h[u][e] -= m0;
                    sums[0] += h[u][e];
                    sums[1] = __builtin_fmaf(h[u][e], h[u][e], sums[1]);
                }
            });
            row_sums<WAVE, 2>(sums, part + flip, 12);
            const float off = mean_of<WAVE>(sums[0], d, part[10 + flip], each);
            if (a.mean && t == 0) a.mean[row] = m0 + off;
            // squares outside fp32's range stay infinite, for rstd_of, which takes those of h - m0 - off; a NaN stays one
            ss = sums[1] < __builtin_inff() ? __builtin_fmaxf(__builtin_fmaf(-off * off, (float)d, sums[1]), 0.0f)
                                            : sums[1] + (off - off);
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int n = d - (u * T + renew(t)) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((WHOLE ? 0 : e) < n) h[u][e] -= off;
            });
        }
        float rstd = 1.0f;
        if (a.weight) {
            if constexpr (!CENTER) ss = row_join<SumOp, WAVE>(ss, part[flip]);
            rstd = rstd_of<WAVE>(ss, d, a.eps, part + 4, flip, each);
            if (a.rstd && t == 0) a.rstd[row] = rstd;
        }
        const bool codes = !CENTER && is_code_type(a.y_type);
        const float factor = codes && a.weight ? power_below(rstd) : rstd;
        float amax = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                if constexpr (LATE) {
                    wr[u] = load_chunk<RAGGED, WHOLE>(a.weight, WT, 0, i, d);
                    if (a.bias) br[u] = load_chunk<RAGGED, WHOLE>(a.bias, WT, 0, i, d);
                }
                if (a.weight) {
                    float w[8];
                    decode_chunk<RAGGED>(wr[u], WT, i, d, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[u][e] = h[u][e] * factor * w[e];
                }
                if constexpr (CENTER)
                    if (a.bias) {
                        float b[8];
                        decode_chunk<RAGGED>(br[u], WT, i, d, b);
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[u][e] += b[e];
                    }
                if constexpr (!CENTER)
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = MaxBitsOp::join(amax, __builtin_fabsf(h[u][e]));
                if (!codes) store8(a.y, a.y_type, (size_t)(row * d) + i, CENTER && WHOLE ? 8 : min(8, d - i), h[u]);
            }
        });
        if (codes) {
            amax = row_join<MaxBitsOp, WAVE>(amax, part[2 + flip]);
            const RowScale s = row_scale_of(amax, rstd / factor, a.y_type);
            if (t == 0) a.scale[row] = s.scale;
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int i = (u * T + renew(t)) * 8;
                if (i < d) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[u][e] *= s.code;
                    store_codes(a.y, a.y_type, (size_t)(row * d) + i, min(8, d - i), h[u]);
                }
            });
        }
        flip ^= 1;  // the next row's joins use other words: no thread may still read these
    }
}

// Rows too long for a workgroup's registers: read once per statistic.  h is
// written in the last pass, so that it may replace x or the residual.
template <int XT, int WT, bool CENTER = false>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a) {
    constexpr int T = 1024;
    __shared__ float part[CENTER ? 14 : 8][16];
    const int t = threadIdx.x;
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        auto load_h = [&](int i, int n, float (&h)[8]) __attribute__((always_inline)) {
            decode8(load_raw8(a.x, XT, (size_t)(row * a.ldx) + i, n), XT, h);
            if (a.residual) {
                float v[8];
                decode8(load_raw8(a.residual, XT, (size_t)(row * a.ldr) + i, n), XT, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] += v[e];
            }
        };
        float m0 = 0.0f, off = 0.0f;
        // h, and without its mean
        auto load_c = [&](int i, int n, float (&h)[8]) __attribute__((always_inline)) {
            load_h(i, n, h);
            if constexpr (CENTER) {
                const int m = renew(n);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = e < m ? h[e] - m0 - off : 0.0f;
            }
        };
        auto load_y = [&](int i, int n, float factor, float (&h)[8]) __attribute__((always_inline)) {
            load_c(i, n, h);
            if (a.weight) {
                float w[8];
                decode8(load_raw8(a.weight, WT, (size_t)i, n), WT, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = h[e] * factor * w[e];
            }
            if constexpr (CENTER)
                if (a.bias) {
                    float b[8];
                    decode8(load_raw8(a.bias, WT, (size_t)i, n), WT, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] += b[e];
                }
        };
        const bool codes = !CENTER && is_code_type(a.y_type);
        float rstd = 1.0f, code = 1.0f, h[8];
        auto each = [&](auto&& f) __attribute__((always_inline)) {
            for (long long i = t * 8; i < a.d; i += T * 8) {
                load_c((int)i, min(8, a.d - (int)i), h);
#pragma unroll
                for (int e = 0; e < 8; ++e) f(h[e]);
            }
        };
        if constexpr (CENTER) {
            float sum = 0.0f;
            each([&](float v) __attribute__((always_inline)) { sum += v; });
            // (m0 is still 0 while the mean is taken, off while its rest is)
            m0 = mean_of<false>(row_join<SumOp, false>(sum, part[8 + flip]), a.d, part[10 + flip], each);
            sum = 0.0f;
            each([&](float v) __attribute__((always_inline)) { sum += v; });
            off = mean_of<false>(row_join<SumOp, false>(sum, part[12 + flip]), a.d, part[10 + flip], each);
            if (a.mean && t == 0) a.mean[row] = m0 + off;
        }
        if (a.weight) {
            float ss = 0.0f;
            each([&](float v) __attribute__((always_inline)) { ss = __builtin_fmaf(v, v, ss); });
            ss = row_join<SumOp, false>(ss, part[flip]);
            rstd = rstd_of<false>(ss, a.d, a.eps, part + 4, flip, each);
            if (a.rstd && t == 0) a.rstd[row] = rstd;
        }
        const float factor = codes && a.weight ? power_below(rstd) : rstd;
        if (codes) {
            float amax = 0.0f;
            for (long long i = t * 8; i < a.d; i += T * 8) {
                load_y((int)i, min(8, a.d - (int)i), factor, h);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = MaxBitsOp::join(amax, __builtin_fabsf(h[e]));
            }
            amax = row_join<MaxBitsOp, false>(amax, part[2 + flip]);
            const RowScale s = row_scale_of(amax, rstd / factor, a.y_type);
            code = s.code;
            if (t == 0) a.scale[row] = s.scale;
        }
        for (long long i = t * 8; i < a.d; i += T * 8) {
            const int n = min(8, a.d - (int)i);
            const size_t at = (size_t)(row * a.d) + i;
            if (a.h) {
                load_h((int)i, n, h);
                float y[8];
                load_y((int)i, n, factor, y);
                store8(a.h, XT, at, n, h);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = y[e];
            } else {
                load_y((int)i, n, factor, h);
            }
            if (codes) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] *= code;
                store_codes(a.y, a.y_type, at, n, h);
            } else {
                store8(a.y, a.y_type, at, n, h);
            }
        }
        flip ^= 1;
    }
}

// ---- layer norm in 8 bits --------------------------------------------------------

// Sums, and largest magnitudes, over a row's threads in fp64, as row_sums has them in
// fp32.
struct Sum64Op {
    __device__ static double join(double a, double b) { return a + b; }
};
struct MaxBits64Op {  // MaxBitsOp of values that are not negative
    __device__ static double join(double a, double b) {
        return __builtin_bit_cast(double, max(__builtin_bit_cast(uint64_t, a), __builtin_bit_cast(uint64_t, b)));
    }
};
// f of both halves' bits
template <class F>
__device__ __forceinline__ double halves(double v, F&& f) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(u32)f((int)(b >> 32)) << 32 | (u32)f((int)(u32)b));
}
template <class Op, int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double join_moved(double v) {
    return Op::join(v, halves(v, [](int w) __attribute__((always_inline)) {
                        return __builtin_amdgcn_update_dpp(0, w, CTRL, ROWS, 0xF, false);
                    }));
}
template <class Op>
__device__ __forceinline__ double join16(double v) {
    return join_moved<Op, 0x118>(join_moved<Op, 0x114>(join_moved<Op, 0x112>(join_moved<Op, 0x111>(v))));
}
template <class Op, bool WAVE, int N>
__device__ __forceinline__ void row_joins(double (&v)[N], double (*part)[16]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = halves(join_moved<Op, 0x143, 0xC>(join_moved<Op, 0x142, 0xA>(join16<Op>(v[i]))),
                      [](int w) __attribute__((always_inline)) { return __builtin_amdgcn_readlane(w, 63); });
    if constexpr (!WAVE) {
        const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[i][threadIdx.x >> 6] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = halves(join16<Op>(lane < waves ? part[i][lane & 15] : 0.0),
                          [](int w) __attribute__((always_inline)) { return __builtin_amdgcn_readlane(w, 15); });
    }
}

// A row's mean and 1 / sqrt(var + eps) from the sums of h - m0 and of their squares
// (fp64 holds the squares of every fp32 value).
struct RowStats {
    double mean, rstd;
};
__device__ __forceinline__ RowStats row_stats(const double (&sums)[2], float m0, double per, const NormArgs& a, long long row, bool keep) {
    const double off = sums[0] * per;  // (per: 1 / d)
    const double var = sums[1] * per - off * off;
    // (a NaN stays one)
    const RowStats s = {m0 + off, 1.0 / __builtin_sqrt((var < 0.0 ? 0.0 : var) + (double)a.eps)};
    if (keep) {
        if (a.mean) a.mean[row] = (float)s.mean;
        if (a.rstd) a.rstd[row] = (float)s.rstd;
    }
    return s;
}
// What a row's values are multiplied by for their codes, from the largest magnitude;
// the scale as row_scale_of has it.
__device__ __forceinline__ double row_code(double amax, const NormArgs& a, long long row, bool keep) {
    const bool e4m3 = a.y_type == GEMM_BT_FP8_E4M3;
    const double q = e4m3 ? 448.0 : 127.0, s = amax * (e4m3 ? 1.0 / 448.0 : 1.0 / 127.0);
    const bool fine = as_u32((float)amax) < 0x7F800000u, tiny = !(s >= 0x1p-100);
    if (keep) a.scale[row] = !fine ? as_f32(0x7FC00000u) : tiny ? 0x1p-100f : (float)s;
    return !fine ? (double)as_f32(0x7FC00000u) : tiny ? 0x1p100 : q / amax;
}
// The largest magnitude of 8 values, a NaN above all.
__device__ __forceinline__ double largest8(const double (&y)[8]) {
    double amax = 0.0;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        amax = __builtin_fmax(amax, __builtin_fabs(y[e]));
        nan |= y[e] != y[e];
    }
    return nan ? __builtin_nan("") : amax;
}
// y = (h - mean) rstd w + b of 8 elements.  Past the row's end w and b are 0, and so is
// y, or the row's mean is not finite and all of it NaN.
__device__ __forceinline__ void normed8(const float (&h)[8], const RowStats& s, const float (&w)[8], const float (&b)[8], double (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fma(((double)h[e] - s.mean) * s.rstd, (double)w[e], (double)b[e]);
}
// v in fp32, cut toward zero, its last bit set where that left anything out: what is then
// rounded to fewer bits comes out as if it had been rounded once (v is 0 or far above
// fp32's smallest normal, or its code 0 either way).
__device__ __forceinline__ float to_odd(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const u32 low = (u32)b, left = (low & 0x1FFFFFFFu) + 0x1FFFFFFFu;
    return (float)__builtin_bit_cast(double, (b >> 32) << 32 | ((low | left) & 0xE0000000u));
}
__device__ __forceinline__ void store_codes64(const NormArgs& a, size_t i, int n, const double (&y)[8], double code) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_odd(y[e] * code);
    store_codes(a.y, a.y_type, i, n, v);
}

// Layer norm to E4M3 or int8 codes.  A code is a step function of y: each rounding of
// y in fp32 moves the codes of those values that lie within it of a step's edge by a
// whole step, 1/16 of an E4M3 value, about one value in 2^21.  With a bias the
// row's factors do not cancel in y / amax as they do for the other norm, so
// everything from the centred values to y / scale is kept in fp64 (the vector unit
// needs as many instructions as in fp32 and the conversions) and the codes are those of
// one rounding.  Bound by that work between a row's loads and its stores, of
// which the two workgroups that fit a CU cover a part: 8192 x 8192 bf16 with residual to
// E4M3 129 us (3.6 TB/s; 150 with y made twice; one chunk per thread 185; the other
// norm, in fp32, 83), 8192 x 4096 61, 16384 x 1024 29; one row of 4096 11 to 14 us, bound by
// the call.  Rows that end inside a chunk cost most: 8191 x 4097 128 us (to 16 bits 68), x,
// the residual, w and b each moved into place.  Rows as in norm_kernel.
template <int XT, int U, bool WAVE, bool RAGGED>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_codes_kernel(const NormArgs a, int w_type) {
    constexpr bool WHOLE = !RAGGED && !WAVE;  // as in norm_kernel
    // y stays in registers where a workgroup of 1024 threads has enough, else it is made
    // twice (w and b come from a cache then)
    constexpr bool HOLD = U == 1 || XT != GEMM_BT_F32;
    __shared__ float part[4][16];
    __shared__ double part64[6][16];
    const int T = WAVE ? 64 : blockDim.x, RB = WAVE ? blockDim.x >> 6 : 1;
    const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int d = a.d;
    const double per = 1.0 / (double)d;
    int flip = 0;
    for (long long row = (long long)blockIdx.x * RB + (WAVE ? threadIdx.x >> 6 : 0); row < a.rows;
         row += (long long)gridDim.x * RB) {
        float h[U][8], sum = 0.0f;
        {
            Raw8 xr[U], rr[U];
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int i = (u * T + renew(t)) * 8;
                if (i < d) {
                    xr[u] = load_chunk<RAGGED, WHOLE>(a.x, XT, row * a.ldx, i, d);
                    if (a.residual) rr[u] = load_chunk<RAGGED, WHOLE>(a.residual, XT, row * a.ldr, i, d);
                }
            });
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int i = (u * T + renew(t)) * 8;
                if (i < d) {
                    decode_chunk<RAGGED>(xr[u], XT, i, d, h[u]);
                    if (a.residual) {
                        float v[8];
                        decode_chunk<RAGGED>(rr[u], XT, i, d, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[u][e] += v[e];
                    }
                    if (a.h) store8(a.h, XT, (size_t)(row * d) + i, WHOLE ? 8 : min(8, d - i), h[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[u][e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += h[u][e];
            });
        }
        const float m0 = mean_of<WAVE>(row_sum<WAVE>(sum, part + flip), d, part[2 + flip], [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) f(h[u][e]);
        });
        double sums[2] = {0.0, 0.0};
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int n = d - (u * T + renew(t)) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double c = (WHOLE ? 0 : e) < n ? (double)h[u][e] - (double)m0 : 0.0;
                sums[0] += c;
                sums[1] = __builtin_fma(c, c, sums[1]);
            }
        });
        row_joins<Sum64Op, WAVE>(sums, part64 + 2 * flip);
        const RowStats s = row_stats(sums, m0, per, a, row, t == 0);
        double y[HOLD ? U : 1][8], amax[1] = {0.0};
        auto load_y = [&](int i, const float (&h)[8], double (&y)[8]) __attribute__((always_inline)) {
            float w[8], b[8];
            decode_chunk<RAGGED>(load_chunk<RAGGED, WHOLE>(a.weight, w_type, 0, i, d), w_type, i, d, w);
            if (a.bias)
                decode_chunk<RAGGED>(load_chunk<RAGGED, WHOLE>(a.bias, w_type, 0, i, d), w_type, i, d, b);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = 0.0f;
            normed8(h, s, w, b, y);
        };
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value, v = HOLD ? u : 0;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                load_y(i, h[u], y[v]);
                amax[0] = MaxBits64Op::join(amax[0], largest8(y[v]));
            }
        });
        row_joins<MaxBits64Op, WAVE>(amax, part64 + 4 + flip);
        const double code = row_code(amax[0], a, row, t == 0);
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value, v = HOLD ? u : 0;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                if constexpr (!HOLD) load_y(i, h[u], y[v]);
                store_codes64(a, (size_t)(row * d) + i, WHOLE ? 8 : min(8, d - i), y[v], code);
            }
        });
        flip ^= 1;  // the next row's joins use other words
    }
}

// Rows too long for registers: read once per statistic, h written in the last pass.
template <int XT, int WT>
__global__ __launch_bounds__(1024) void norm_codes_long_kernel(const NormArgs a) {
    constexpr int T = 1024;
    __shared__ float part[4][16];
    __shared__ double part64[6][16];
    const int t = threadIdx.x;
    const double per = 1.0 / (double)a.d;
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        // f(first element, elements, their h)
        auto each8 = [&](auto&& f) __attribute__((always_inline)) {
            for (long long i = renew(t) * 8; i < a.d; i += T * 8) {
                const int n = min(8, a.d - (int)i);
                float h[8];
                decode8(load_raw8(a.x, XT, (size_t)(row * a.ldx) + i, n), XT, h);
                if (a.residual) {
                    float v[8];
                    decode8(load_raw8(a.residual, XT, (size_t)(row * a.ldr) + i, n), XT, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] += v[e];
                }
                f((int)i, n, h);
            }
        };
        float sum = 0.0f;
        auto each = [&](auto&& f) __attribute__((always_inline)) {
            each8([&](int, int, float (&h)[8]) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f(h[e]);  // (0 past the row's end)
            });
        };
        each([&](float v) __attribute__((always_inline)) { sum += v; });
        const float m0 = mean_of<false>(row_sum<false>(sum, part + flip), a.d, part[2 + flip], each);
        double sums[2] = {0.0, 0.0};
        each8([&](int, int n, float (&h)[8]) __attribute__((always_inline)) {
            n = renew(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double c = e < n ? (double)h[e] - (double)m0 : 0.0;
                sums[0] += c;
                sums[1] = __builtin_fma(c, c, sums[1]);
            }
        });
        row_joins<Sum64Op, false>(sums, part64 + 2 * flip);
        const RowStats s = row_stats(sums, m0, per, a, row, renew(t) == 0);
        auto load_y = [&](int i, int n, const float (&h)[8], double (&y)[8]) __attribute__((always_inline)) {
            float w[8], b[8];
            decode8(load_raw8(a.weight, WT, (size_t)i, n), WT, w);
            if (a.bias)
                decode8(load_raw8(a.bias, WT, (size_t)i, n), WT, b);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = 0.0f;
            normed8(h, s, w, b, y);
        };
        double amax[1] = {0.0};
        each8([&](int i, int n, float (&h)[8]) __attribute__((always_inline)) {
            double y[8];
            load_y(i, n, h, y);
            amax[0] = MaxBits64Op::join(amax[0], largest8(y));
        });
        row_joins<MaxBits64Op, false>(amax, part64 + 4 + flip);
        const double code = row_code(amax[0], a, row, renew(t) == 0);
        each8([&](int i, int n, float (&h)[8]) __attribute__((always_inline)) {
            double y[8];
            load_y(i, n, h, y);
            if (a.h) store8(a.h, XT, (size_t)(row * a.d) + i, n, h);
            store_codes64(a, (size_t)(row * a.d) + i, renew(n), y, code);
        });
        flip ^= 1;
    }
}

// Rows of no elements: their squares' mean is 0, and so is their largest
// magnitude.
__global__ __launch_bounds__(256) void empty_rows_kernel(float* scale, float* rstd, float* mean, long long rows, float eps) {
    const long long step = (long long)gridDim.x * 256;
    for (long long row = (long long)blockIdx.x * 256 + threadIdx.x; row < rows; row += step) {
        if (scale) scale[row] = 0x1p-100f;
        if (rstd) rstd[row] = 1.0f / __builtin_sqrtf(eps);
        if (mean) mean[row] = 0.0f;
    }
}

// ---- 8-bit blocks --------------------------------------------------------------------

struct BlockArgs {
    const void* x;
    void* q;
    float* scale;
    long long rows, ldx, pitch;  // of x; pitch of q's rows in bytes
    int d;
    long long tiles_d, tiles;    // 128 x 128 tiles of x: per row of them, and all
};

// v / scale of a block's values, from the largest magnitude: 448 / amax in two parts.
// With 16-bit inputs v 448 / amax often lies on the edge between two codes, else well
// off it; with 448 / amax in one part 1 in 400 of their codes fell on the wrong side.  Of
// fp32 inputs it may lie anywhere: ODD sets the last bit of a rounded value, so that the
// code comes out as if it had been rounded once.
struct BlockCode {
    float high, low;
    template <bool ODD>
    __device__ __forceinline__ float of(float v) const {
#pragma clang fp contract(off)  // p is the rounded product in f and in what is left
        const float p = v * high, q = __builtin_fmaf(v, low, __builtin_fmaf(v, high, -p)), f = p + q;
        if constexpr (!ODD) return f;
        const float left = q - (f - p);
        const u32 b = as_u32(f);  // (toward what is left: up in magnitude where the signs agree)
        return as_f32(left == 0.0f || (b & 1) ? b : b + (u32)(((int)(as_u32(left) ^ b) >> 31) | 1));
    }
};
__device__ __forceinline__ BlockCode block_code(float amax, float* scale) {
    const RowScale s = row_scale_of(amax, 1.0f, GEMM_BT_FP8_E4M3);
    *scale = s.scale;
    // (a scale kept at 2^-100 has a reciprocal of one part)
    return {s.code, s.scale == 0x1p-100f ? 0.0f : __builtin_fmaf(-s.code, amax, 448.0f) * (s.code * (1.0f / 448.0f))};
}

// V = x, or x transposed (TRANS), in E4M3 with one scale per 1 x 128 block of V, or
// per 128 x 128 block (TALL): scale = max(amax / 448, 2^-100), code = RNE(v / scale).
// Bound by HBM: 8192 x 8192 bf16 38 us (5.3 TB/s), transposed 44; 1000 x 2000 f16
// transposed 5.6, 128 workgroups of one tile each.  A workgroup takes a 128 x 128 tile
// of x, thread (tr, tc) = (t / 16, t % 16) its rows 8 tr .. 8 tr + 7 and columns 8 tc ..
// 8 tc + 7: the 16 lanes of a row of x are one row of the vector unit's data moves, a
// column's rows lie in 8 registers, and the 8 x 8 codes of a thread turn in registers
// for the transposed result, which leaves through LDS as whole 128-byte rows.  Scales lie block by
// block, those of consecutive rows of V next to each other, as the product's
// tiles read them.
template <int XT, bool TALL, bool TRANS>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const BlockArgs a) {
    __shared__ float part[4][128];
    __shared__ __attribute__((aligned(16))) unsigned char turned[TRANS ? 128 * 128 : 16];
    const int t = threadIdx.x, tr = t >> 4, tc = t & 15, wave = t >> 6;
    for (long long tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const long long ti = tile / a.tiles_d, tj = tile - ti * a.tiles_d;
        const long long row0 = ti * 128 + 8 * tr;
        const int col0 = (int)(tj * 128) + 8 * tc;
        const int cols = min(8, a.d - col0), rows = (int)max(0LL, min(8LL, a.rows - row0));
        Raw8 raw[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            raw[r] = Raw8{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
            if (r < rows && cols > 0) raw[r] = load_raw8(a.x, XT, (size_t)((row0 + r) * a.ldx) + col0, cols);
        }
        float v[8][8];
#pragma unroll
        for (int r = 0; r < 8; ++r) decode8(raw[r], XT, v[r]);
        auto larger = [](float p, float x) __attribute__((always_inline)) { return MaxBitsOp::join(p, __builtin_fabsf(x)); };
        // what each row (TRANS: each column; TALL: every one) of the thread's part is multiplied by
        BlockCode code[8];
        if constexpr (TALL) {
            float top = 0.0f;
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) top = larger(top, v[r][c]);
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) top = MaxBitsOp::join(top, __shfl_xor(top, m));
            if ((t & 63) == 0) part[wave][0] = top;
            __syncthreads();
            top = MaxBitsOp::join(MaxBitsOp::join(part[0][0], part[1][0]), MaxBitsOp::join(part[2][0], part[3][0]));
            float scale;
            const BlockCode one = block_code(top, &scale);
#pragma unroll
            for (int r = 0; r < 8; ++r) code[r] = one;
            if (t == 0) {
                const long long high = (a.rows + 127) / 128;  // row blocks of x
                a.scale[TRANS ? ti * a.tiles_d + tj : tj * high + ti] = scale;
            }
        } else if constexpr (!TRANS) {
            float scale[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) top = larger(top, v[r][c]);
                // the largest of 16 lanes, in each of them: rotations by 8, 4, 2 and 1
                auto moved = [&](auto ctrl) __attribute__((always_inline)) {
                    top = MaxBitsOp::join(top, as_f32((u32)__builtin_amdgcn_update_dpp(0, (int)as_u32(top), decltype(ctrl)::value, 0xF, 0xF, false)));
                };
                moved(std::integral_constant<int, 0x128>{});
                moved(std::integral_constant<int, 0x124>{});
                moved(std::integral_constant<int, 0x122>{});
                moved(std::integral_constant<int, 0x121>{});
                code[r] = block_code(top, &scale[r]);
            }
            if (tc == 0)
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < rows) a.scale[tj * a.rows + row0 + r] = scale[r];
        } else {
            float tops[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float top = 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r) top = larger(top, v[r][c]);
                top = MaxBitsOp::join(top, __shfl_xor(top, 16));
                tops[c] = MaxBitsOp::join(top, __shfl_xor(top, 32));
            }
            if ((t & 63) < 16) {
                *(f32x4*)&part[wave][8 * tc] = f32x4{tops[0], tops[1], tops[2], tops[3]};
                *(f32x4*)&part[wave][8 * tc + 4] = f32x4{tops[4], tops[5], tops[6], tops[7]};
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float top = part[0][8 * tc + c];
#pragma unroll
                for (int w = 1; w < 4; ++w) top = MaxBitsOp::join(top, part[w][8 * tc + c]);
                float scale;
                code[c] = block_code(top, &scale);
                if (tr == 0 && c < cols) a.scale[ti * a.d + col0 + c] = scale;
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c) v[r][c] = code[TRANS ? c : r].template of<XT == GEMM_BT_F32>(v[r][c]);
        if constexpr (!TRANS) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < rows && cols > 0) store_codes(a.q, GEMM_BT_FP8_E4M3, (size_t)((row0 + r) * a.pitch) + col0, cols, v[r]);
            if constexpr (TALL) __syncthreads();  // `part` is written again
        } else {
            // column c of the tile is 128 bytes of `turned`, its 16-byte chunk k at place k ^ (c / 8 % 8)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const u32x2 w = {quant4<GEMM_BT_FP8_E4M3>(v[0][c], v[1][c], v[2][c], v[3][c]),
                                 quant4<GEMM_BT_FP8_E4M3>(v[4][c], v[5][c], v[6][c], v[7][c])};
                *(u32x2*)(turned + (8 * tc + c) * 128 + (((tr >> 1) ^ (tc & 7)) * 16) + (tr & 1) * 8) = w;
            }
            __syncthreads();
            const int wide = (int)min(128LL, a.pitch - ti * 128);  // a multiple of 16: zeros behind the last row of x
            const int high = min(128, a.d - (int)(tj * 128));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = i * 32 + (t >> 3), k = t & 7;
                if (c < high && 16 * k < wide) {
                    const u32x4 w = *(const u32x4*)(turned + c * 128 + ((k ^ (c >> 3 & 7)) * 16));
                    __builtin_nontemporal_store(w, (u32x4_byte*)((unsigned char*)a.q + (size_t)((tj * 128 + c) * a.pitch) + ti * 128 + 16 * k));
                }
            }
            __syncthreads();  // `part` and `turned` are written again
        }
    }
}

// ---- norm, backward --------------------------------------------------------------

struct NormBackArgs {
    const void* dy;
    const void* h;
    const void* weight;
    const float* rstd;
    const void* dh;   // nullptr: none
    void* dx;
    float* partials;  // gridDim.x rows of d sums of dy * xhat
    long long rows, ld_dy, ldh, ld_dh;
    int d;
    const float* mean;    // layer norm alone
    float* bias_parts;    // layer norm alone: gridDim.x rows of d sums of dy, nullptr: not wanted
    // rows of whole 16-byte chunks: dy, h and dh are read past the caches (8192
    // x 8192 bf16 100.3 -> 93.6 us).  Elsewhere neighbouring chunks share lines, and
    // it makes no difference (8191 x 4097 80.5 against 80.9).
    int nt;
};

// Bound by HBM: 8192 x 4096 bf16 with dh 49 us for this kernel and 4 for the
// fold of its partial sums (5.1 TB/s in all).
// With xhat = h rstd and g = dy w:  dx = rstd (g - xhat mean(g xhat)) + dh, and
// dw = sum over rows of dy xhat.  Layout as in norm_kernel; each thread sums
// dw of its own columns over the workgroup's rows in registers, and the
// workgroup leaves one row of partial sums.  AHEAD: the next row is fetched
// while this one is worked on, and the weight stays in registers; without it
// (rows that fill the registers) both are read when they are needed.
// CENTER: layer norm (8192 x 4096 bf16 with dh and db 57 us in all: this kernel 49, 5.4
// TB/s, the fold of dw and db 7; with a dh that stays in the caches 50, by shuffles
// 53).  xhat = (h - mean) rstd, dx = rstd (g - mean(g) - xhat mean(g
// xhat)) + dh, and db = sum over rows of dy, summed and left like dw.
template <int XT, int WT, int U, bool WAVE, bool AHEAD, int MOST, bool RAGGED, bool CENTER = false>
__global__ __launch_bounds__(MOST) void norm_back_kernel(const NormBackArgs a) {
    constexpr int RB = WAVE ? MOST / 64 : 1;
    constexpr int S = CENTER ? 2 : 1;  // sums over rows: dw, db
    constexpr bool WHOLE = !RAGGED && !WAVE;  // every chunk is 8 elements of the row (rows below 8 have a wave each)
    __shared__ float part[2 * S][16];
    __shared__ float joined[WAVE ? MOST * U * 8 : 1];
    const int T = WAVE ? 64 : blockDim.x;
    const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int d = a.d;
    float dw[S * U][8];  // with db after it
    Raw8 wr[U];
    if constexpr (AHEAD)
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) wr[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.weight, WT, 0, i, d);
        });
#pragma unroll
    for (int u = 0; u < S * U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = 0.0f;
    const long long step = (long long)gridDim.x * RB;
    struct Row {
        Raw8 dy[U], h[U], dh[U];
        float rstd, mean;
    };
    auto fetch = [&](long long row, Row& r) __attribute__((always_inline)) {
        if (row >= a.rows) return;
        r.rstd = a.rstd[row];
        if constexpr (CENTER) r.mean = a.mean[row];
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                r.dy[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.dy, XT, row * a.ld_dy, i, d, a.nt);
                r.h[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.h, XT, row * a.ldh, i, d, a.nt);
                if (AHEAD && a.dh) r.dh[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.dh, XT, row * a.ld_dh, i, d, a.nt);
            }
        });
    };
    int flip = 0;
    long long row = (long long)blockIdx.x * RB + (WAVE ? threadIdx.x >> 6 : 0);
    Row now;
    if constexpr (AHEAD) fetch(row, now);
    for (; row < a.rows; row += step) {
        Row next;
        if constexpr (AHEAD) {
            fetch(row + step, next);
        } else {
            fetch(row, now);
        }
        float xhat[U][8], g[U][8], c = 0.0f, m = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float w[8];
                if constexpr (!AHEAD) wr[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.weight, WT, 0, i, d);
                decode_chunk<RAGGED>(now.h[u], XT, i, d, xhat[u]);
                decode_chunk<RAGGED>(now.dy[u], XT, i, d, g[u]);
                decode_chunk<RAGGED>(wr[u], WT, i, d, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (CENTER) {
                        // (0 past the row's end: 0 g stays 0 however far the mean is)
                        xhat[u][e] = WHOLE || i + e < d ? (xhat[u][e] - now.mean) * now.rstd : 0.0f;
                        dw[U + u][e] += g[u][e];
                    } else {
                        xhat[u][e] *= now.rstd;
                    }
                    dw[u][e] = __builtin_fmaf(g[u][e], xhat[u][e], dw[u][e]);
                    g[u][e] *= w[e];
                    c = __builtin_fmaf(g[u][e], xhat[u][e], c);
                    if constexpr (CENTER) m += g[u][e];
                }
            }
        });
        if constexpr (CENTER) {
            float sums[2] = {c, m};
            row_sums<WAVE, 2>(sums, part + flip, 2);
            c = sums[0];
            m = sums[1] / (float)d;
        } else {
            c = row_join<SumOp, WAVE>(c, part[flip]);
        }
        c /= (float)d;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = now.rstd * __builtin_fmaf(-xhat[u][e], c, CENTER ? g[u][e] - m : g[u][e]);
                if (a.dh) {
                    float v[8];
                    if constexpr (!AHEAD) now.dh[u] = load_chunk<RAGGED, CENTER && WHOLE>(a.dh, XT, row * a.ld_dh, i, d);
                    decode_chunk<RAGGED>(now.dh[u], XT, i, d, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += v[e];
                }
                store8(a.dx, XT, (size_t)(row * d) + i, CENTER && WHOLE ? 8 : min(8, d - i), o);
            }
        });
        if constexpr (AHEAD) now = next;
        flip ^= 1;
    }
    if constexpr (RB > 1) {
        // join the waves' sums, in wave order
        const int wave = threadIdx.x >> 6;
        static_for<0, S>([&](auto sc) __attribute__((always_inline)) {
            constexpr int s = decltype(sc)::value;
            if constexpr (s > 0) __syncthreads();
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
#pragma unroll
                for (int e = 0; e < 8; ++e) joined[(wave * U * 8 + u * 8 + e) * 64 + t] = dw[s * U + u][e];
            });
            __syncthreads();
            if (wave == 0)
                static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                    constexpr int u = decltype(uc)::value;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int w = 1; w < RB; ++w) dw[s * U + u][e] += joined[(w * U * 8 + u * 8 + e) * 64 + t];
                });
        });
        if (wave != 0) return;
    }
    static_for<0, S * U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        const int i = (u % U * T + t) * 8;
        float* const sums = u < U ? a.partials : a.bias_parts;
        if (i < d && (u < U || sums)) {
            float* p = sums + (size_t)blockIdx.x * d + i;
            if (i + 8 <= d) {
                *(u32x4_any*)p = u32x4{as_u32(dw[u][0]), as_u32(dw[u][1]), as_u32(dw[u][2]), as_u32(dw[u][3])};
                *(u32x4_any*)(p + 4) = u32x4{as_u32(dw[u][4]), as_u32(dw[u][5]), as_u32(dw[u][6]), as_u32(dw[u][7])};
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (i + e < d) p[e] = dw[u][e];
            }
        }
    });
}

// Few rows: the first a.rows workgroups (WAVE: a wave each) make dx, one row
// each; the others make dw itself, 64 columns each over all rows, from dy and
// h as the caches hold them.  One launch, no partial sums.
// CENTER: layer norm, with db (dbias, nullptr: not wanted) beside dw.
template <int XT, int WT, int U, bool WAVE, bool RAGGED, bool CENTER = false>
__global__ __launch_bounds__(1024) void norm_back_few_kernel(const NormBackArgs a, int row_blocks, void* dweight, void* dbias) {
    constexpr int S = CENTER ? 2 : 1;
    constexpr bool WHOLE = !RAGGED && !WAVE;
    __shared__ float part[S][16];
    __shared__ float joined[S][128][65];
    const int d = a.d;
    if ((int)blockIdx.x < row_blocks) {
        const int T = WAVE ? 64 : blockDim.x;
        const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
        const long long row = WAVE ? (long long)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : blockIdx.x;
        if (row >= a.rows) return;
        Raw8 dyr[U], hr[U], dhr[U], wr[U];
        const float rstd = a.rstd[row], mean = CENTER ? a.mean[row] : 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                dyr[u] = load_chunk<RAGGED>(a.dy, XT, row * a.ld_dy, i, d);
                hr[u] = load_chunk<RAGGED>(a.h, XT, row * a.ldh, i, d);
                wr[u] = load_chunk<RAGGED>(a.weight, WT, 0, i, d);
                if (a.dh) dhr[u] = load_chunk<RAGGED>(a.dh, XT, row * a.ld_dh, i, d);
            }
        });
        float xhat[U][8], g[U][8], c = 0.0f, m = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float w[8];
                decode_chunk<RAGGED>(wr[u], WT, i, d, w);
                decode_chunk<RAGGED>(hr[u], XT, i, d, xhat[u]);
                decode_chunk<RAGGED>(dyr[u], XT, i, d, g[u]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (CENTER)
                        xhat[u][e] = WHOLE || i + e < d ? (xhat[u][e] - mean) * rstd : 0.0f;
                    else
                        xhat[u][e] *= rstd;
                    g[u][e] *= w[e];
                    c = __builtin_fmaf(g[u][e], xhat[u][e], c);
                    if constexpr (CENTER) m += g[u][e];
                }
            }
        });
        if constexpr (CENTER) {
            float sums[2] = {c, m};
            row_sums<WAVE, 2>(sums, part, 1);
            c = sums[0];
            m = sums[1] / (float)d;
        } else {
            c = row_join<SumOp, WAVE>(c, part[0]);
        }
        c /= (float)d;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = rstd * __builtin_fmaf(-xhat[u][e], c, CENTER ? g[u][e] - m : g[u][e]);
                if (a.dh) {
                    float v[8];
                    decode_chunk<RAGGED>(dhr[u], XT, i, d, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += v[e];
                }
                store8(a.dx, XT, (size_t)(row * d) + i, min(8, d - i), o);
            }
        });
        return;
    }
    // dw of 64 columns: 8 lanes of 8 columns, blockDim / 8 groups of them over the rows
    const int G = blockDim.x >> 3, l = threadIdx.x & 7, k = threadIdx.x >> 3;
    const int j = ((int)blockIdx.x - row_blocks) * 64 + l * 8;
    float sum[S][8];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[s][e] = 0.0f;
    if (j < d) {
        for (int r = k; r < a.rows; r += 4 * G) {
            Raw8 dyr[4], hr[4];
            float rs[4], mean[4];
            static_for<0, 4>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const long long row = r + u * G;
                if (row < a.rows) {
                    rs[u] = a.rstd[row];
                    if constexpr (CENTER) mean[u] = a.mean[row];
                    dyr[u] = load_chunk<RAGGED>(a.dy, XT, row * a.ld_dy, j, d);
                    hr[u] = load_chunk<RAGGED>(a.h, XT, row * a.ldh, j, d);
                }
            });
            static_for<0, 4>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                if (r + u * G < a.rows) {
                    float y[8], h[8];
                    decode_chunk<RAGGED>(dyr[u], XT, j, d, y);
                    decode_chunk<RAGGED>(hr[u], XT, j, d, h);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum[0][e] = __builtin_fmaf(y[e], CENTER ? (h[e] - mean[u]) * rs[u] : h[e] * rs[u], sum[0][e]);
                        if constexpr (CENTER) sum[S - 1][e] += y[e];
                    }
                }
            });
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) joined[s][k][l * 8 + e] = sum[s][e];
    __syncthreads();
    // the groups' sums, halved in number until one is left
    for (int half = G >> 1; half > 0; half >>= 1) {
        for (int i = threadIdx.x; i < half * 64; i += blockDim.x)
#pragma unroll
            for (int s = 0; s < S; ++s) joined[s][i >> 6][i & 63] += joined[s][(i >> 6) + half][i & 63];
        __syncthreads();
    }
    const int col = ((int)blockIdx.x - row_blocks) * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < d) {
        store1(dweight, WT, (size_t)col, joined[0][0][threadIdx.x]);
        if (CENTER && dbias) store1(dbias, WT, (size_t)col, joined[S - 1][0][threadIdx.x]);
    }
}

// Rows too long for a workgroup's registers: dw is summed in the workgroup's
// row of partial sums itself, each word by one thread.
template <int XT, int WT, bool CENTER = false>
__global__ __launch_bounds__(1024) void norm_back_long_kernel(const NormBackArgs a) {
    constexpr int T = 1024;
    __shared__ float part[CENTER ? 4 : 2][16];
    const int t = threadIdx.x;
    float* sums = a.partials + (size_t)blockIdx.x * a.d;
    float* bsums = CENTER && a.bias_parts ? a.bias_parts + (size_t)blockIdx.x * a.d : nullptr;
    for (long long i = t; i < a.d; i += T) {
        sums[i] = 0.0f;
        if (bsums) bsums[i] = 0.0f;
    }
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row], mean = CENTER ? a.mean[row] : 0.0f;
        auto load1x = [&](const void* p, long long ld, long long i) { return load1(p, XT, (size_t)(row * ld + i)); };
        auto load_xhat = [&](long long i) { return (CENTER ? load1x(a.h, a.ldh, i) - mean : load1x(a.h, a.ldh, i)) * rstd; };
        float c = 0.0f, m = 0.0f;
        for (long long i = t; i < a.d; i += T) {
            const float g = load1x(a.dy, a.ld_dy, i) * load1(a.weight, WT, i);
            c = __builtin_fmaf(g, load_xhat(i), c);
            if constexpr (CENTER) m += g;
        }
        c = row_join<SumOp, false>(c, part[flip]) / (float)a.d;
        if constexpr (CENTER) m = row_join<SumOp, false>(m, part[2 + flip]) / (float)a.d;
        for (long long i = t; i < a.d; i += T) {
            const float dy = load1x(a.dy, a.ld_dy, i), xhat = load_xhat(i), g = dy * load1(a.weight, WT, i);
            float o = rstd * __builtin_fmaf(-xhat, c, CENTER ? g - m : g);
            if (a.dh) o += load1x(a.dh, a.ld_dh, i);
            store1(a.dx, XT, (size_t)(row * a.d + i), o);
            sums[i] = __builtin_fmaf(dy, xhat, sums[i]);
            if (bsums) bsums[i] += dy;
        }
        flip ^= 1;
    }
}

// ---- column sums: the last step ---------------------------------------------------

__global__ __launch_bounds__(512) void fold_kernel(const FoldArgs a) {
    __shared__ float sums[512 / 16][17];
    fold_columns<512>(a, blockIdx.x, sums);
}
// Two at once, the grid's second axis.
__global__ __launch_bounds__(512) void fold2_kernel(const FoldArgs a, const FoldArgs b) {
    __shared__ float sums[512 / 16][17];
    fold_columns<512>(blockIdx.y ? b : a, blockIdx.x, sums);
}

// ---- activation and bias, backward -------------------------------------------------

// Bound by HBM: 4096 x 4096 bf16 22 us (4.6 TB/s), 8192 x 8192 77 (5.2).
// dz = dy act'(z), and the sums of dz over a block of rows.  L lanes hold 8
// columns each; a workgroup's 256 / L groups of lanes take its rows in turn.
template <int L, bool RAGGED>
__global__ __launch_bounds__(256) void act_back_kernel(const ActBackArgs a) {
    constexpr int G = 256 / L;
    __shared__ float joined[G][L * 8];
    const int l = threadIdx.x % L, g = threadIdx.x / L;
    const int j = (blockIdx.x * L + l) * 8;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    const long long first = (long long)blockIdx.y * a.rows_per_block;
    const long long last = min(a.rows, first + a.rows_per_block);
    if (j < a.n)
        with_act(a.preact ? a.act : GEMM_BT_ACT_NONE, [&](auto act) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            auto one = [&](const Raw8& dyr, const Raw8& zr, long long row) __attribute__((always_inline)) {
                float v[8];
                decode_chunk<RAGGED>(dyr, a.type, j, a.n, v);
                if constexpr (ACT != GEMM_BT_ACT_NONE) {
                    float z[8];
                    decode_chunk<RAGGED>(zr, a.preact_type, j, a.n, z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= act_slope<ACT>(z[e]);
                }
                if (a.dz) store8(a.dz, a.type, (size_t)(row * a.ldz) + j, min(8, a.ldz - j), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += v[e];
            };
            auto load = [&](long long row, Raw8& dyr, Raw8& zr) __attribute__((always_inline)) {
                dyr = load_chunk<RAGGED>(a.dy, a.type, row * a.n, j, a.n, a.nt);
                if constexpr (ACT != GEMM_BT_ACT_NONE) zr = load_chunk<RAGGED>(a.preact, a.preact_type, row * a.n, j, a.n, a.nt);
            };
            // four rows in flight: each is fetched again as soon as it is used
            Raw8 dyr[4], zr[4];
            long long row = first + g;
            static_for<0, 4>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                if (row + u * G < last) load(row + u * G, dyr[u], zr[u]);
            });
            for (; row < last; row += 4 * G)
                static_for<0, 4>([&](auto uc) __attribute__((always_inline)) {
                    constexpr int u = decltype(uc)::value;
                    if (row + u * G < last) {
                        one(dyr[u], zr[u], row + u * G);
                        if (row + (u + 4) * G < last) load(row + (u + 4) * G, dyr[u], zr[u]);
                    }
                });
        });
    if (!a.partials) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[g][l * 8 + e] = sum[e];
    __syncthreads();
    float* p = a.partials + (size_t)blockIdx.y * a.n;
    for (int c = threadIdx.x; c < L * 8; c += 256) {
        const long long col = (long long)blockIdx.x * L * 8 + c;
        if (col >= a.n) continue;
        float s = joined[0][c];
#pragma unroll
        for (int i = 1; i < G; ++i) s += joined[i][c];
        p[col] = s;
    }
}

// act(z) and act'(z), which share their exponential.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
    if constexpr (ACT == GEMM_BT_ACT_GELU) {
        float gauss;
        const float p = normal_cdf(z, gauss);
        value = z * p;
        slope = __builtin_fmaf(z * 0.3989422804014327f, gauss, p);
    } else if constexpr (ACT == GEMM_BT_ACT_SILU) {
        const float p = sigmoid_f(z);
        value = z * p;
        slope = p * __builtin_fmaf(z, 1.0f - p, 1.0f);
    } else {
        value = act_value<ACT>(z);
        slope = act_slope<ACT>(z);
    }
}

// Bound by HBM: reads dy and both halves of z, writes both halves of dz (4096 x
// 4096 bf16, 168 MB, 33 us, 5.0 TB/s).  Layout as in act_back_kernel, two rows in
// flight (each is three chunks).
template <int L, bool RAGGED>
__global__ __launch_bounds__(256) void gated_back_kernel(const ActBackArgs a) {
    constexpr int G = 256 / L;
    __shared__ float joined[2][G][L * 8];
    const int l = threadIdx.x % L, g = threadIdx.x / L;
    const int n = a.n, j = (blockIdx.x * L + l) * 8;
    float sum[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[s][e] = 0.0f;
    const long long first = (long long)blockIdx.y * a.rows_per_block;
    const long long last = min(a.rows, first + a.rows_per_block);
    if (j < n)
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            struct Row {
                Raw8 dy, gate, up;
            };
            auto load = [&](long long row, Row& r) __attribute__((always_inline)) {
                r.dy = load_chunk<RAGGED>(a.dy, a.type, row * n, j, n, a.nt);
                r.gate = load_chunk<RAGGED>(a.preact, a.preact_type, row * 2 * n, j, n, a.nt);
                r.up = load_chunk<RAGGED>(a.preact, a.preact_type, (row * 2 + 1) * n, j, n, a.nt);
            };
            auto one = [&](const Row& r, long long row) __attribute__((always_inline)) {
                float dy[8], dg[8], du[8];
                decode_chunk<RAGGED>(r.dy, a.type, j, n, dy);
                decode_chunk<RAGGED>(r.gate, a.preact_type, j, n, dg);
                decode_chunk<RAGGED>(r.up, a.preact_type, j, n, du);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float value, slope;
                    act_both<ACT>(dg[e], value, slope);
                    dg[e] = dy[e] * du[e] * slope;
                    du[e] = dy[e] * value;
                    sum[0][e] += dg[e];
                    sum[1][e] += du[e];
                }
                if (a.dz) {
                    const size_t at = (size_t)(row * a.ldz) + j;
                    store8(a.dz, a.type, at, min(8, n - j), dg);
                    store8(a.dz, a.type, at + n, min(8, a.ldz - n - j), du);  // with zeros behind the row, up to ldz:
                    if (j + 8 >= n)  // at most 3 more, past the last chunk (n = 5, 6 or 7 mod 8)
                        for (int c = n + j + 8; c < a.ldz; ++c) store1(a.dz, a.type, (size_t)(row * a.ldz) + c, 0.0f);
                }
            };
            Row r[2];
            long long row = first + g;
            static_for<0, 2>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                if (row + u * G < last) load(row + u * G, r[u]);
            });
            for (; row < last; row += 2 * G)
                static_for<0, 2>([&](auto uc) __attribute__((always_inline)) {
                    constexpr int u = decltype(uc)::value;
                    if (row + u * G < last) {
                        one(r[u], row + u * G);
                        if (row + (u + 2) * G < last) load(row + (u + 2) * G, r[u]);
                    }
                });
        });
    if (!a.partials) return;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) joined[s][g][l * 8 + e] = sum[s][e];
    __syncthreads();
    float* p = a.partials + (size_t)blockIdx.y * 2 * n;
    for (int c = threadIdx.x; c < 2 * L * 8; c += 256) {
        const int s = c / (L * 8), k = c % (L * 8);
        const long long col = (long long)blockIdx.x * L * 8 + k;
        if (col >= n) continue;
        float v = joined[s][0][k];
#pragma unroll
        for (int i = 1; i < G; ++i) v += joined[s][i][k];
        p[s * (long long)n + col] = v;
    }
}

// ---- host ------------------------------------------------------------------------

// One thread per 16 columns and row group of the fold, in a grid of at most 2^32
// threads; int offsets inside a row.
constexpr int64_t kMaxColumns = 1 << 26;
// Rows `ld` elements apart that all start on a 16-byte boundary.
static bool whole_chunks(const void* p, int64_t ld, int t) { return (uintptr_t)p % 16 == 0 && ld * elem_size(t) % 16 == 0; }
static bool stride_ok(int64_t ld, int64_t d) { return ld >= d && ld < (1LL << 40); }

struct RowPlan {
    const void* fn;
    int threads, rows_per_block;
};

// Whole waves that hold `chunks` groups of 8 elements, U of them per thread.
static int threads_for(int64_t chunks, int U) { return (int)((chunks + 64 * U - 1) / (64 * U) * 64); }

// fn(chunks per thread, whether a wave holds a row) for rows in registers, else far.
template <class F>
static RowPlan rows_plan(int64_t rows, int64_t d, int num_cu, const void* far, F&& fn) {
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    const int64_t chunks = (d + 7) / 8;
    // Few rows (at most two per CU): one chunk per thread, so that one load's
    // latency is all that is waited for.
    const bool few = rows <= 2 * num_cu;
    if (chunks <= 64) return few ? RowPlan{fn(One{}, std::true_type{}), 64, 1} : RowPlan{fn(One{}, std::true_type{}), 256, 4};
    if (chunks <= 128 && !few) return {fn(Two{}, std::true_type{}), 256, 4};
    if (chunks <= 256 || (few && chunks <= 1024)) return {fn(One{}, std::false_type{}), threads_for(chunks, 1), 1};
    if (chunks <= 2048) return {fn(Two{}, std::false_type{}), threads_for(chunks, 2), 1};
    return {far, 1024, 1};
}
template <int XT, int WT, bool R, bool C>
static RowPlan norm_plan(int64_t rows, int64_t d, int num_cu) {
    return rows_plan(rows, d, num_cu, (const void*)&norm_long_kernel<XT, WT, C>,
                     [](auto u, auto wave) { return (const void*)&norm_kernel<XT, WT, u(), wave(), R, C>; });
}
// Layer norm in 8 bits: the kernels that hold a row take w's type as an argument.
template <int XT, int WT, bool R>
static RowPlan norm_codes_plan(int64_t rows, int64_t d, int num_cu) {
    return rows_plan(rows, d, num_cu, (const void*)&norm_codes_long_kernel<XT, WT>,
                     [](auto u, auto wave) { return (const void*)&norm_codes_kernel<XT, u(), wave(), R>; });
}

template <int XT, int WT, bool R, bool C>
static RowPlan norm_back_plan(int64_t d) {
    const int64_t chunks = (d + 7) / 8;
    if (chunks <= 64) return {(const void*)&norm_back_kernel<XT, WT, 1, true, true, 256, R, C>, 256, 4};
    if (chunks <= 128) return {(const void*)&norm_back_kernel<XT, WT, 2, true, true, 256, R, C>, 256, 4};
    if (chunks <= 256) return {(const void*)&norm_back_kernel<XT, WT, 1, false, true, 256, R, C>, threads_for(chunks, 1), 1};
    if (chunks <= 1024) return {(const void*)&norm_back_kernel<XT, WT, 2, false, true, 512, R, C>, threads_for(chunks, 2), 1};
    if (chunks <= 2048) return {(const void*)&norm_back_kernel<XT, WT, 2, false, false, 1024, R, C>, threads_for(chunks, 2), 1};
    return {(const void*)&norm_back_long_kernel<XT, WT, C>, 1024, 1};
}

// Rows that end inside a chunk of 8 (those below 8 have no chunk to load from).
// Kernels of their own for them, against one kernel that puts the last chunk
// together element by element (us, bf16): norm 32768 x 511 57 -> 29 (512: 22),
// backward 139 -> 37 (28), 16384 x 1023 77 -> 33 (29), 8191 x 4097 114 -> 80
// (54), activation backward 16384 x 1023 61 -> 31 (25).  With the moves in the
// kernels for whole chunks too, those lost: 32768 x 512 backward 28 -> 47.
static bool ragged(int64_t d) { return d >= 8 && d % 8 != 0; }

static bool weight_type_ok(int x_type, int w_type) { return w_type == x_type || w_type == GEMM_BT_F32; }
// f(x_type, w_type, ragged) for the weight types there are kernels for (x's own
// and fp32) and rows of d elements.
template <class F>
static RowPlan with_types(int x_type, int w_type, int64_t d, F&& f) {
    auto g = [&](auto x, auto w) { return ragged(d) ? f(x, w, std::true_type{}) : f(x, w, std::false_type{}); };
    typedef std::integral_constant<int, GEMM_BT_F32> F32;
    typedef std::integral_constant<int, GEMM_BT_F16> F16;
    typedef std::integral_constant<int, GEMM_BT_BF16> BF16;
    if (x_type == GEMM_BT_F32) return g(F32{}, F32{});
    if (x_type == GEMM_BT_F16) return w_type == GEMM_BT_F32 ? g(F16{}, F32{}) : g(F16{}, F16{});
    return w_type == GEMM_BT_F32 ? g(BF16{}, F32{}) : g(BF16{}, BF16{});
}

template <bool C = false>
static int launch_norm(NormArgs& a, int x_type, int w_type, void* stream) {
    int num_cu = 0;
    const int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    const RowPlan p = with_types(x_type, w_type, a.d, [&](auto x, auto w, auto r) {
        if constexpr (C)
            if (is_code_type(a.y_type)) return norm_codes_plan<x(), w(), r()>(a.rows, a.d, num_cu);
        return norm_plan<x(), w(), r(), C>(a.rows, a.d, num_cu);
    });
    const int64_t grid = std::min<int64_t>((a.rows + p.rows_per_block - 1) / p.rows_per_block, 1 << 20);
    void* args[] = {&a, &w_type};  // (norm_codes_kernel has both)
    return launch(p.fn, dim3((unsigned)grid), p.threads, args, stream);
}

// Rows of no elements leave their scales and rstd, where there are any.
static int empty_rows(float* scale, float* rstd, float* mean, long long rows, float eps, void* stream) {
    if (!aligned(scale, GEMM_BT_F32) || !aligned(rstd, GEMM_BT_F32) || !aligned(mean, GEMM_BT_F32)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!scale && !rstd && !mean) return GEMM_BT_OK;
    int num_cu = 0;
    const int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    void* args[] = {&scale, &rstd, &mean, &rows, &eps};
    return launch((const void*)&empty_rows_kernel, dim3((unsigned)std::min<int64_t>((rows + 255) / 256, 8 * num_cu)), 256, args,
                  stream);
}

template <bool C = false>
static RowPlan norm_back_plan_of(int x_type, int w_type, int64_t d) {
    return with_types(x_type, w_type, d, [&](auto x, auto w, auto r) { return norm_back_plan<x(), w(), r(), C>(d); });
}
// The kernel for few rows, or none: while dy and h stay in the caches, reading
// them twice costs less than a second launch and its partial sums, as long as
// each group of lanes has at most 8 rows to sum (us, bf16, two launches vs
// one: 1 x 4096 5.4 vs 3.2, 128 x 8192 10.4 vs 5.3, 512 x 4096 15.3 vs 8.8, 512 x
// 8192 17.5 vs 13.7; with 16 rows to a group 1000 x 2050 fp32 13.1 vs 14.3, 400 x
// 1023 bf16 7.0 vs 9.2, with 32 1000 x 2048 11.3 vs 19.8, 2048 x 4096 22.5 vs 27.0).  Threads in a power of two: the
// last step halves their groups.
template <int XT, int WT, bool R, bool C>
static RowPlan norm_back_few(int64_t rows, int64_t d) {
    const int64_t chunks = (d + 7) / 8;
    auto pow2 = [](int64_t n) {
        int t = 256;
        while (t < n) t *= 2;
        return t;
    };
    if (chunks > 2048 || rows * d > (4 << 20)) return {nullptr, 0, 0};
    RowPlan p;
    if (chunks <= 64) p = {(const void*)&norm_back_few_kernel<XT, WT, 1, true, R, C>, 256, 4};
    else if (chunks <= 1024) p = {(const void*)&norm_back_few_kernel<XT, WT, 1, false, R, C>, pow2(chunks), 1};
    else p = {(const void*)&norm_back_few_kernel<XT, WT, 2, false, R, C>, 1024, 1};
    if (rows > p.threads) return {nullptr, 0, 0};
    return p;
}

// Workgroups of the backward pass, each of which leaves one row of partial
// sums: about 512 threads per CU (all of them resident), and the same number
// of rows for all but the last ones.  (8192 x 4096 bf16, us: 512 threads per CU 53.6, 768 59.0,
// 1024 63.6; 16384 x 1024 28.3, 29.6, 32.6: more workgroups do not read faster,
// and each leaves d fp32 sums more to write and fold.  Workgroups of 192, two or
// three per CU: 16384 x 2560 72.7, 64.3, 16384 x 1536 46.4, 41.5, 4000 x 2056 21.2,
// 20.1, 8192 x 3000 42.2, 43.5; of 320, one or two: 8192 x 5120 65.5, 69.4, 8191 x
// 4104 59.4, 61.5, 8191 x 4097 80.3, 72.6.)
static int64_t norm_back_grid(const RowPlan& p, int64_t rows, int num_cu) {
    const int per_cu = p.threads <= 256 ? (512 + p.threads / 2) / p.threads : 1;
    const int64_t most = (int64_t)num_cu * per_cu * p.rows_per_block;
    const int64_t per = (rows + most - 1) / most * p.rows_per_block;  // rows of a workgroup
    return per > 0 ? (rows + per - 1) / per : 0;
}

// Row blocks of the activation's backward pass (the grid's second axis).
struct ActBackPlan {
    const void* fn;
    int64_t strips, blocks;
    int rows_per_block;
};
static ActBackPlan act_back_plan(int64_t rows, int64_t n, int num_cu, bool gated = false) {
    ActBackPlan p;
    int lanes = 64;
    const bool r = ragged(n);
    auto kernel = [&](auto l) {
        lanes = l();
        if (gated) p.fn = r ? (const void*)&gated_back_kernel<l(), true> : (const void*)&gated_back_kernel<l(), false>;
        else p.fn = r ? (const void*)&act_back_kernel<l(), true> : (const void*)&act_back_kernel<l(), false>;
    };
    if (n <= 64) kernel(std::integral_constant<int, 8>{});
    else if (n <= 128) kernel(std::integral_constant<int, 16>{});
    else if (n <= 256) kernel(std::integral_constant<int, 32>{});
    else kernel(std::integral_constant<int, 64>{});
    const int groups = 256 / lanes;  // rows a workgroup takes at a time
    p.strips = (n + lanes * 8 - 1) / (lanes * 8);
    // as many workgroups as run at once, four per CU, each with whole rounds of its
    // groups (4096 x 4096 bf16, gelu_tanh, us: two per CU 34.1, four 26.3, eight
    // 28.5, which also leave twice the partial sums); the kernels for ragged rows
    // take 150 registers and run three (8191 x 4097: three 60.2, four 75.6; 16384 x
    // 1023: 30.7, 35.6)
    const int64_t want = std::max<int64_t>(1, (r ? 3 : 4) * num_cu / p.strips);
    int64_t per = (rows + want - 1) / want;
    per = std::max<int64_t>(groups, (per + groups - 1) / groups * groups);
    p.blocks = (rows + per - 1) / per;
    while (p.blocks > 32768) {  // the grid's second axis ends at 65535
        per *= 2;
        p.blocks = (rows + per - 1) / per;
    }
    p.rows_per_block = (int)per;
    return p;
}

static int fold(const float* partials, void* out, int out_type, int64_t parts, int64_t d, void* stream) {
    FoldArgs a = {partials, out, d, (int)parts, out_type};
    void* args[] = {&a};
    return launch((const void*)&fold_kernel, dim3(fold_blocks(d)), 512, args, stream);
}

int64_t act_back_parts(int64_t rows, int64_t n, int num_cu) { return act_back_plan(rows, n, num_cu).blocks; }

int launch_act_back(ActBackArgs a, int num_cu, void* stream) {
    const ActBackPlan p = act_back_plan(a.rows, a.n, num_cu);
    a.rows_per_block = p.rows_per_block;
    a.nt = whole_chunks(a.dy, a.n, a.type) && whole_chunks(a.preact, a.n, a.preact_type);
    void* args[] = {&a};
    return launch(p.fn, dim3((unsigned)p.strips, (unsigned)p.blocks), 256, args, stream);
}

// ---- the norms' backward passes: checks and launches ---------------------------------

// Layer norm (C) leaves the partial sums of dbias after those of dweight.
template <bool C>
static int norm_back_workspace(int64_t rows, int64_t d, size_t* bytes) {
    if (!bytes) return GEMM_BT_ERR_INVALID_VALUE;
    *bytes = 0;
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    // (the plans' grids do not depend on the types, nor on whole chunks)
    if (norm_back_few<GEMM_BT_BF16, GEMM_BT_BF16, false, C>(rows, d).fn) return GEMM_BT_OK;
    *bytes = (size_t)(norm_back_grid(norm_back_plan_of<C>(GEMM_BT_BF16, GEMM_BT_BF16, d), rows, plan_cus()) * d * (C ? 8 : 4));
    return GEMM_BT_OK;
}

template <bool C>
static int norm_backward(NormBackArgs a, int64_t d, void* dweight, void* dbias, int x_dtype, int w_dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const int64_t rows = a.rows;
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (!float_type(x_dtype) || !weight_type_ok(x_dtype, w_dtype)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d == 0) return GEMM_BT_OK;
    if (!dweight || !aligned(dweight, w_dtype) || !aligned(dbias, w_dtype)) return GEMM_BT_ERR_INVALID_VALUE;
    if (rows > 0) {
        // (the few-rows kernel's sums for dweight read dy and h while dx is written)
        if (!a.dy || !a.h || !a.weight || !a.rstd || (C && !a.mean) || !a.dx || a.dx == a.dy || a.dx == a.h)
            return GEMM_BT_ERR_INVALID_VALUE;
        if (!stride_ok(a.ld_dy, d) || !stride_ok(a.ldh, d) || (a.dh && !stride_ok(a.ld_dh, d))) return GEMM_BT_ERR_INVALID_VALUE;
        if (!aligned(a.dy, x_dtype) || !aligned(a.h, x_dtype) || !aligned(a.dh, x_dtype) || !aligned(a.dx, x_dtype) ||
            !aligned(a.weight, w_dtype) || !aligned(a.rstd, GEMM_BT_F32) || !aligned(a.mean, GEMM_BT_F32) ||
            !aligned(workspace, GEMM_BT_F32))
            return GEMM_BT_ERR_INVALID_VALUE;
    }
    int num_cu = 0;
    int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    a.d = (int)d;
    int64_t grid = 0;
    if (rows > 0) {
        const RowPlan few = with_types(
            x_dtype, w_dtype, d, [&](auto x, auto w, auto r) { return norm_back_few<x(), w(), r(), C>(rows, d); });
        if (few.fn) {
            int row_blocks = (int)((rows + few.rows_per_block - 1) / few.rows_per_block);
            void* args[] = {&a, &row_blocks, &dweight, &dbias};
            return launch(few.fn, dim3((unsigned)(row_blocks + (d + 63) / 64)), few.threads, args, stream);
        }
        const RowPlan p = norm_back_plan_of<C>(x_dtype, w_dtype, d);
        grid = norm_back_grid(p, rows, num_cu);
        if (!workspace || workspace_bytes < (size_t)(grid * d * (C ? 8 : 4))) return GEMM_BT_ERR_INVALID_VALUE;
        a.partials = (float*)workspace;
        if (dbias) a.bias_parts = a.partials + grid * d;
        a.nt = whole_chunks(a.dy, a.ld_dy, x_dtype) && whole_chunks(a.h, a.ldh, x_dtype) && whole_chunks(a.dh, a.ld_dh, x_dtype);
        void* args[] = {&a};
        st = launch(p.fn, dim3((unsigned)grid), p.threads, args, stream);
        if (st != GEMM_BT_OK) return st;
    }
    if (!dbias) return fold((const float*)workspace, dweight, w_dtype, grid, d, stream);
    FoldArgs fw = {(const float*)workspace, dweight, d, (int)grid, w_dtype}, fb = {fw.partials + grid * d, dbias, d, (int)grid, w_dtype};
    void* args[] = {&fw, &fb};
    return launch((const void*)&fold2_kernel, dim3(fold_blocks(d), 2), 512, args, stream);
}

int64_t gated_back_parts(int64_t rows, int64_t n, int num_cu) { return act_back_plan(rows, n, num_cu, true).blocks; }

int launch_gated_back(ActBackArgs a, int num_cu, void* stream) {
    const ActBackPlan p = act_back_plan(a.rows, a.n, num_cu, true);
    a.rows_per_block = p.rows_per_block;
    a.nt = whole_chunks(a.dy, a.n, a.type) && whole_chunks(a.preact, a.n, a.preact_type);
    void* args[] = {&a};
    return launch(p.fn, dim3((unsigned)p.strips, (unsigned)p.blocks), 256, args, stream);
}

}  // namespace gbt

using namespace gbt;

extern "C" {

int gemm_bt_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* y, void* h,
                     float* scale, float* rstd, int64_t rows, int64_t d, float eps, int x_dtype, int w_dtype, int y_dtype,
                     void* stream) {
    if (rows < 0 || d < 0 || !(eps >= 0.0f)) return GEMM_BT_ERR_INVALID_VALUE;
    const bool codes = y_dtype == GEMM_BT_FP8_E4M3 || y_dtype == GEMM_BT_INT8;
    if (!float_type(x_dtype) || !weight_type_ok(x_dtype, w_dtype) || !(codes || float_type(y_dtype))) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_BT_OK;
    if (codes && !scale) return GEMM_BT_ERR_INVALID_VALUE;
    if (d == 0) return empty_rows(codes ? scale : nullptr, rstd, nullptr, rows, eps, stream);
    if (!x || !weight || !y) return GEMM_BT_ERR_INVALID_VALUE;
    if (!stride_ok(ldx, d) || (residual && !stride_ok(ldr, d))) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(residual, x_dtype) || !aligned(h, x_dtype) || !aligned(weight, w_dtype) ||
        (!codes && !aligned(y, y_dtype)) || !aligned(scale, GEMM_BT_F32) || !aligned(rstd, GEMM_BT_F32))
        return GEMM_BT_ERR_INVALID_VALUE;
    NormArgs a = {x, residual, weight, y, h, scale, rstd, rows, ldx, ldr, (int)d, eps, y_dtype, nullptr, nullptr};
    return launch_norm(a, x_dtype, w_dtype, stream);
}

int gemm_bt_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, const void* bias,
                       void* y, void* h, float* scale, float* mean, float* rstd, int64_t rows, int64_t d, float eps, int x_dtype,
                       int w_dtype, int y_dtype, void* stream) {
    if (rows < 0 || d < 0 || !(eps >= 0.0f)) return GEMM_BT_ERR_INVALID_VALUE;
    const bool codes = y_dtype == GEMM_BT_FP8_E4M3 || y_dtype == GEMM_BT_INT8;
    if (!float_type(x_dtype) || !weight_type_ok(x_dtype, w_dtype) || !(codes || float_type(y_dtype))) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_BT_OK;
    if (codes && !scale) return GEMM_BT_ERR_INVALID_VALUE;
    if (d == 0) return empty_rows(codes ? scale : nullptr, rstd, mean, rows, eps, stream);
    if (!x || !weight || !y) return GEMM_BT_ERR_INVALID_VALUE;
    if (!stride_ok(ldx, d) || (residual && !stride_ok(ldr, d))) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(residual, x_dtype) || !aligned(h, x_dtype) || !aligned(weight, w_dtype) ||
        !aligned(bias, w_dtype) || (!codes && !aligned(y, y_dtype)) || !aligned(scale, GEMM_BT_F32) || !aligned(mean, GEMM_BT_F32) ||
        !aligned(rstd, GEMM_BT_F32))
        return GEMM_BT_ERR_INVALID_VALUE;
    NormArgs a = {x, residual, weight, y, h, scale, rstd, rows, ldx, ldr, (int)d, eps, y_dtype, bias, mean};
    return launch_norm<true>(a, x_dtype, w_dtype, stream);
}

int gemm_bt_quantize_rows(const void* x, int64_t ldx, void* q, float* scale, int64_t rows, int64_t d, int x_dtype,
                          int q_dtype, void* stream) {
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (!float_type(x_dtype) || (q_dtype != GEMM_BT_FP8_E4M3 && q_dtype != GEMM_BT_INT8)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_BT_OK;
    if (!scale) return GEMM_BT_ERR_INVALID_VALUE;
    if (d == 0) return empty_rows(scale, nullptr, nullptr, rows, 0.0f, stream);
    if (!x || !q || !stride_ok(ldx, d)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(scale, GEMM_BT_F32)) return GEMM_BT_ERR_INVALID_VALUE;
    NormArgs a = {x, nullptr, nullptr, q, nullptr, scale, nullptr, rows, ldx, 0, (int)d, 0.0f, q_dtype, nullptr, nullptr};
    return launch_norm(a, x_dtype, x_dtype, stream);
}

int gemm_bt_quantize_blocks(const void* x, int64_t ldx, void* q, float* scale, int64_t rows, int64_t d, int block_rows,
                            int transpose, int x_dtype, int q_dtype, void* stream) {
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if ((block_rows != 1 && block_rows != 128) || (transpose != 0 && transpose != 1)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!float_type(x_dtype) || q_dtype != GEMM_BT_FP8_E4M3) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows == 0 || d == 0) return GEMM_BT_OK;
    if (!x || !q || !scale || !stride_ok(ldx, d)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(scale, GEMM_BT_F32)) return GEMM_BT_ERR_INVALID_VALUE;
    int num_cu = 0;
    const int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    const int64_t wide = (d + 127) / 128;
    BlockArgs a = {x, q, scale, rows, ldx, transpose ? (rows + 15) / 16 * 16 : d, (int)d, wide, (rows + 127) / 128 * wide};
    const void* fn = nullptr;
    auto pick = [&](auto t) {
        constexpr int XT = decltype(t)::value;
        if (block_rows == 128)
            fn = transpose ? (const void*)&quantize_blocks_kernel<XT, true, true> : (const void*)&quantize_blocks_kernel<XT, true, false>;
        else
            fn = transpose ? (const void*)&quantize_blocks_kernel<XT, false, true> : (const void*)&quantize_blocks_kernel<XT, false, false>;
    };
    if (x_dtype == GEMM_BT_F32) pick(std::integral_constant<int, GEMM_BT_F32>{});
    else if (x_dtype == GEMM_BT_F16) pick(std::integral_constant<int, GEMM_BT_F16>{});
    else pick(std::integral_constant<int, GEMM_BT_BF16>{});
    void* args[] = {&a};
    return launch(fn, dim3((unsigned)std::min<int64_t>(a.tiles, 1 << 20)), 256, args, stream);
}

int gemm_bt_rms_norm_backward_workspace(int64_t rows, int64_t d, size_t* bytes) {
    return norm_back_workspace<false>(rows, d, bytes);
}

int gemm_bt_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const void* weight,
                              const float* rstd, const void* dh, int64_t ld_dh, void* dx, void* dweight, int64_t rows,
                              int64_t d, int x_dtype, int w_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    NormBackArgs a = {dy, h, weight, rstd, dh, dx, nullptr, rows, ld_dy, ldh, ld_dh, 0, nullptr, nullptr, 0};
    return norm_backward<false>(a, d, dweight, nullptr, x_dtype, w_dtype, workspace, workspace_bytes, stream);
}

int gemm_bt_layer_norm_backward_workspace(int64_t rows, int64_t d, size_t* bytes) {
    return norm_back_workspace<true>(rows, d, bytes);
}

int gemm_bt_layer_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const void* weight, const float* mean,
                                const float* rstd, const void* dh, int64_t ld_dh, void* dx, void* dweight, void* dbias,
                                int64_t rows, int64_t d, int x_dtype, int w_dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
    NormBackArgs a = {dy, h, weight, rstd, dh, dx, nullptr, rows, ld_dy, ldh, ld_dh, 0, mean, nullptr, 0};
    return norm_backward<true>(a, d, dweight, dbias, x_dtype, w_dtype, workspace, workspace_bytes, stream);
}

int gemm_bt_act_backward_workspace(int64_t rows, int64_t n, size_t* bytes) {
    if (!bytes) return GEMM_BT_ERR_INVALID_VALUE;
    *bytes = 0;
    if (rows < 0 || n < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (n > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows > 0 && n > 0) *bytes = (size_t)(act_back_plan(rows, n, plan_cus()).blocks * n * 4);
    return GEMM_BT_OK;
}

int gemm_bt_act_backward(const void* dy, const void* preact, void* dz, void* dbias, int64_t rows, int64_t n,
                         int activation, int dtype, int preact_dtype, int bias_dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (rows < 0 || n < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (activation < GEMM_BT_ACT_NONE || activation > GEMM_BT_ACT_SILU) return GEMM_BT_ERR_INVALID_VALUE;
    const bool act = activation != GEMM_BT_ACT_NONE;
    if (!float_type(dtype) || (act && !float_type(preact_dtype)) || (dbias && !float_type(bias_dtype)))
        return GEMM_BT_ERR_UNSUPPORTED;
    if (n > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (n == 0) return GEMM_BT_OK;
    if (dbias && !aligned(dbias, bias_dtype)) return GEMM_BT_ERR_INVALID_VALUE;
    if (rows > 0) {
        if (!dy || (act && !preact) || (dbias && !workspace)) return GEMM_BT_ERR_INVALID_VALUE;
        if (!aligned(dy, dtype) || !aligned(dz, dtype) || (act && !aligned(preact, preact_dtype)) ||
            !aligned(workspace, GEMM_BT_F32))
            return GEMM_BT_ERR_INVALID_VALUE;
    }
    if (!dbias && (!dz || rows == 0)) return GEMM_BT_OK;
    int num_cu = 0;
    int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    int64_t parts = 0;
    if (rows > 0) {
        parts = act_back_parts(rows, n, num_cu);
        if (dbias && workspace_bytes < (size_t)(parts * n * 4)) return GEMM_BT_ERR_INVALID_VALUE;
        st = launch_act_back({dy, act ? preact : nullptr, dz, dbias ? (float*)workspace : nullptr, rows, (int)n, (int)n, 0, dtype,
                              preact_dtype, activation},
                             num_cu, stream);
        if (st != GEMM_BT_OK) return st;
    }
    return dbias ? fold((const float*)workspace, dbias, bias_dtype, parts, n, stream) : GEMM_BT_OK;
}

}  // extern "C"
