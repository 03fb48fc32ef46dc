// norm.hip -- the row operators next to the product: root-mean-square norm
// with the residual's addition, out in 16 or 32 bits or in 8 bits with one
// scale per row; 8-bit rows with scales of a matrix as it is; the norm's
// backward pass; and the backward pass of an epilogue's activation and bias.
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

// ---- rows in chunks of 8 ---------------------------------------------------------

// Elements i .. i+7 of a row of d that starts at element `base` of p.  RAGGED
// (d >= 8, no multiple of 8): the last chunk is loaded from element d - 8 on and
// moved into place when it is decoded.  A load is then one instruction for
// every lane, and nothing waits for it before its use, where a branch that put
// single elements together waits for everything in flight.  Rows of whole
// chunks have kernels without the moves.
template <bool RAGGED>
__device__ __forceinline__ Raw8 load_chunk(const void* p, int t, long long base, int i, int d, bool nt = false) {
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
        if (amax > 0.0f && amax < __builtin_inff()) {
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
};

__device__ inline bool is_code_type(int t) { return t == GEMM_BT_FP8_E4M3 || t == GEMM_BT_INT8; }

// h = x + residual; y = h rstd w: one pass over x and the residual, whose row
// stays in registers between its statistics and its results.  Bound by HBM:
// 8192 x 8192 bf16 with residual 92 us (5.8 TB/s; a plain copy reaches 5.1),
// to E4M3 83 us, 4096 x 4096 quantised alone 11.4 us; one row of 4096 2.8 us, a
// launch.  Inputs are read through the caches, where the kernel before may have
// left them (8192 x 8192 without residual 43 us against 50 past them).
// The T threads that hold a row, U chunks of 8 elements each (T * U * 8 >= d),
// are a wave (WAVE; a workgroup is up to 4 of them, each with rows of its own) or
// the whole workgroup, of as many waves as the row fills.
template <int XT, int WT, int U, bool WAVE, bool RAGGED>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(const NormArgs a) {
    __shared__ float part[8][16];
    const int T = WAVE ? 64 : blockDim.x, RB = WAVE ? blockDim.x >> 6 : 1;
    const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int d = a.d;
    int flip = 0;
    for (long long row = (long long)blockIdx.x * RB + (WAVE ? threadIdx.x >> 6 : 0); row < a.rows;
         row += (long long)gridDim.x * RB) {
        Raw8 xr[U], rr[U], wr[U];
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                xr[u] = load_chunk<RAGGED>(a.x, XT, row * a.ldx, i, d);
                if (a.residual) rr[u] = load_chunk<RAGGED>(a.residual, XT, row * a.ldr, i, d);
                if (a.weight) wr[u] = load_chunk<RAGGED>(a.weight, WT, 0, i, d);
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
                if (a.h) store8(a.h, XT, (size_t)(row * d) + i, min(8, d - i), h[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[u][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[u][e], h[u][e], ss);
        });
        float rstd = 1.0f;
        if (a.weight) {
            ss = row_join<SumOp, WAVE>(ss, part[flip]);
            rstd = rstd_of<WAVE>(ss, d, a.eps, part + 4, flip, [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f(h[u][e]);
            });
            if (a.rstd && t == 0) a.rstd[row] = rstd;
        }
        const bool codes = is_code_type(a.y_type);
        const float factor = codes && a.weight ? power_below(rstd) : rstd;
        float amax = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                if (a.weight) {
                    float w[8];
                    decode_chunk<RAGGED>(wr[u], WT, i, d, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[u][e] = h[u][e] * factor * w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = MaxBitsOp::join(amax, __builtin_fabsf(h[u][e]));
                if (!codes) store8(a.y, a.y_type, (size_t)(row * d) + i, min(8, d - i), h[u]);
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
template <int XT, int WT>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a) {
    constexpr int T = 1024;
    __shared__ float part[8][16];
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
        auto load_y = [&](int i, int n, float factor, float (&h)[8]) __attribute__((always_inline)) {
            load_h(i, n, h);
            if (a.weight) {
                float w[8];
                decode8(load_raw8(a.weight, WT, (size_t)i, n), WT, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = h[e] * factor * w[e];
            }
        };
        const bool codes = is_code_type(a.y_type);
        float rstd = 1.0f, code = 1.0f, h[8];
        if (a.weight) {
            float ss = 0.0f;
            for (long long i = t * 8; i < a.d; i += T * 8) {
                load_h((int)i, min(8, a.d - (int)i), h);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[e], h[e], ss);
            }
            ss = row_join<SumOp, false>(ss, part[flip]);
            rstd = rstd_of<false>(ss, a.d, a.eps, part + 4, flip, [&](auto&& f) __attribute__((always_inline)) {
                for (long long i = t * 8; i < a.d; i += T * 8) {
                    load_h((int)i, min(8, a.d - (int)i), h);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f(h[e]);
                }
            });
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

// Rows of no elements: their squares' mean is 0, and so is their largest
// magnitude.
__global__ __launch_bounds__(256) void empty_rows_kernel(float* scale, float* rstd, long long rows, float eps) {
    const long long step = (long long)gridDim.x * 256;
    for (long long row = (long long)blockIdx.x * 256 + threadIdx.x; row < rows; row += step) {
        if (scale) scale[row] = 0x1p-100f;
        if (rstd) rstd[row] = 1.0f / __builtin_sqrtf(eps);
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
template <int XT, int WT, int U, bool WAVE, bool AHEAD, int MOST, bool RAGGED>
__global__ __launch_bounds__(MOST) void norm_back_kernel(const NormBackArgs a) {
    constexpr int RB = WAVE ? MOST / 64 : 1;
    __shared__ float part[2][16];
    __shared__ float joined[WAVE ? MOST * U * 8 : 1];
    const int T = WAVE ? 64 : blockDim.x;
    const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int d = a.d;
    float dw[U][8];
    Raw8 wr[U];
    if constexpr (AHEAD)
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) wr[u] = load_chunk<RAGGED>(a.weight, WT, 0, i, d);
        });
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = 0.0f;
    const long long step = (long long)gridDim.x * RB;
    struct Row {
        Raw8 dy[U], h[U], dh[U];
        float rstd;
    };
    auto fetch = [&](long long row, Row& r) __attribute__((always_inline)) {
        if (row >= a.rows) return;
        r.rstd = a.rstd[row];
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                r.dy[u] = load_chunk<RAGGED>(a.dy, XT, row * a.ld_dy, i, d, a.nt);
                r.h[u] = load_chunk<RAGGED>(a.h, XT, row * a.ldh, i, d, a.nt);
                if (AHEAD && a.dh) r.dh[u] = load_chunk<RAGGED>(a.dh, XT, row * a.ld_dh, i, d, a.nt);
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
        float xhat[U][8], g[U][8], c = 0.0f;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float w[8];
                if constexpr (!AHEAD) wr[u] = load_chunk<RAGGED>(a.weight, WT, 0, i, d);
                decode_chunk<RAGGED>(now.h[u], XT, i, d, xhat[u]);
                decode_chunk<RAGGED>(now.dy[u], XT, i, d, g[u]);
                decode_chunk<RAGGED>(wr[u], WT, i, d, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xhat[u][e] *= now.rstd;
                    dw[u][e] = __builtin_fmaf(g[u][e], xhat[u][e], dw[u][e]);
                    g[u][e] *= w[e];
                    c = __builtin_fmaf(g[u][e], xhat[u][e], c);
                }
            }
        });
        c = row_join<SumOp, WAVE>(c, part[flip]) / (float)d;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = now.rstd * __builtin_fmaf(-xhat[u][e], c, g[u][e]);
                if (a.dh) {
                    float v[8];
                    if constexpr (!AHEAD) now.dh[u] = load_chunk<RAGGED>(a.dh, XT, row * a.ld_dh, i, d);
                    decode_chunk<RAGGED>(now.dh[u], XT, i, d, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += v[e];
                }
                store8(a.dx, XT, (size_t)(row * d) + i, min(8, d - i), o);
            }
        });
        if constexpr (AHEAD) now = next;
        flip ^= 1;
    }
    if constexpr (RB > 1) {
        // join the waves' sums, in wave order
        const int wave = threadIdx.x >> 6;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
#pragma unroll
            for (int e = 0; e < 8; ++e) joined[(wave * U * 8 + u * 8 + e) * 64 + t] = dw[u][e];
        });
        __syncthreads();
        if (wave != 0) return;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int w = 1; w < RB; ++w) dw[u][e] += joined[(w * U * 8 + u * 8 + e) * 64 + t];
        });
    }
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        const int i = (u * T + t) * 8;
        if (i < d) {
            float* p = a.partials + (size_t)blockIdx.x * d + i;
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
template <int XT, int WT, int U, bool WAVE, bool RAGGED>
__global__ __launch_bounds__(1024) void norm_back_few_kernel(const NormBackArgs a, int row_blocks, void* dweight) {
    __shared__ float part[16];
    __shared__ float joined[128][65];
    const int d = a.d;
    if ((int)blockIdx.x < row_blocks) {
        const int T = WAVE ? 64 : blockDim.x;
        const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
        const long long row = WAVE ? (long long)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : blockIdx.x;
        if (row >= a.rows) return;
        Raw8 dyr[U], hr[U], dhr[U], wr[U];
        const float rstd = a.rstd[row];
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
        float xhat[U][8], g[U][8], c = 0.0f;
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
                    xhat[u][e] *= rstd;
                    g[u][e] *= w[e];
                    c = __builtin_fmaf(g[u][e], xhat[u][e], c);
                }
            }
        });
        c = row_join<SumOp, WAVE>(c, part) / (float)d;
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            const int i = (u * T + renew(t)) * 8;
            if (i < d) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = rstd * __builtin_fmaf(-xhat[u][e], c, g[u][e]);
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
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    if (j < d) {
        for (int r = k; r < a.rows; r += 4 * G) {
            Raw8 dyr[4], hr[4];
            float rs[4];
            static_for<0, 4>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const long long row = r + u * G;
                if (row < a.rows) {
                    rs[u] = a.rstd[row];
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
                    for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(y[e], h[e] * rs[u], sum[e]);
                }
            });
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[k][l * 8 + e] = sum[e];
    __syncthreads();
    // the groups' sums, halved in number until one is left
    for (int half = G >> 1; half > 0; half >>= 1) {
        for (int i = threadIdx.x; i < half * 64; i += blockDim.x) joined[i >> 6][i & 63] += joined[(i >> 6) + half][i & 63];
        __syncthreads();
    }
    const int col = ((int)blockIdx.x - row_blocks) * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < d) store1(dweight, WT, (size_t)col, joined[0][threadIdx.x]);
}

// Rows too long for a workgroup's registers: dw is summed in the workgroup's
// row of partial sums itself, each word by one thread.
template <int XT, int WT>
__global__ __launch_bounds__(1024) void norm_back_long_kernel(const NormBackArgs a) {
    constexpr int T = 1024;
    __shared__ float part[2][16];
    const int t = threadIdx.x;
    float* sums = a.partials + (size_t)blockIdx.x * a.d;
    for (long long i = t; i < a.d; i += T) sums[i] = 0.0f;
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        auto load1x = [&](const void* p, long long ld, long long i) { return load1(p, XT, (size_t)(row * ld + i)); };
        float c = 0.0f;
        for (long long i = t; i < a.d; i += T)
            c = __builtin_fmaf(load1x(a.dy, a.ld_dy, i) * load1(a.weight, WT, i), load1x(a.h, a.ldh, i) * rstd, c);
        c = row_join<SumOp, false>(c, part[flip]) / (float)a.d;
        for (long long i = t; i < a.d; i += T) {
            const float dy = load1x(a.dy, a.ld_dy, i), xhat = load1x(a.h, a.ldh, i) * rstd;
            float o = rstd * __builtin_fmaf(-xhat, c, dy * load1(a.weight, WT, i));
            if (a.dh) o += load1x(a.dh, a.ld_dh, i);
            store1(a.dx, XT, (size_t)(row * a.d + i), o);
            sums[i] = __builtin_fmaf(dy, xhat, sums[i]);
        }
        flip ^= 1;
    }
}

// ---- column sums: the last step ---------------------------------------------------

__global__ __launch_bounds__(512) void fold_kernel(const FoldArgs a) {
    __shared__ float sums[512 / 16][17];
    fold_columns<512>(a, blockIdx.x, sums);
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

template <int XT, int WT, bool R>
static RowPlan norm_plan(int64_t rows, int64_t d, int num_cu) {
    const int64_t chunks = (d + 7) / 8;
    // Few rows (at most two per CU): one chunk per thread, so that one load's
    // latency is all that is waited for.
    const bool few = rows <= 2 * num_cu;
    if (chunks <= 64)
        return few ? RowPlan{(const void*)&norm_kernel<XT, WT, 1, true, R>, 64, 1}
                   : RowPlan{(const void*)&norm_kernel<XT, WT, 1, true, R>, 256, 4};
    if (chunks <= 128 && !few) return {(const void*)&norm_kernel<XT, WT, 2, true, R>, 256, 4};
    if (chunks <= 256 || (few && chunks <= 1024))
        return {(const void*)&norm_kernel<XT, WT, 1, false, R>, threads_for(chunks, 1), 1};
    if (chunks <= 2048) return {(const void*)&norm_kernel<XT, WT, 2, false, R>, threads_for(chunks, 2), 1};
    return {(const void*)&norm_long_kernel<XT, WT>, 1024, 1};
}

template <int XT, int WT, bool R>
static RowPlan norm_back_plan(int64_t d) {
    const int64_t chunks = (d + 7) / 8;
    if (chunks <= 64) return {(const void*)&norm_back_kernel<XT, WT, 1, true, true, 256, R>, 256, 4};
    if (chunks <= 128) return {(const void*)&norm_back_kernel<XT, WT, 2, true, true, 256, R>, 256, 4};
    if (chunks <= 256) return {(const void*)&norm_back_kernel<XT, WT, 1, false, true, 256, R>, threads_for(chunks, 1), 1};
    if (chunks <= 1024) return {(const void*)&norm_back_kernel<XT, WT, 2, false, true, 512, R>, threads_for(chunks, 2), 1};
    if (chunks <= 2048) return {(const void*)&norm_back_kernel<XT, WT, 2, false, false, 1024, R>, threads_for(chunks, 2), 1};
    return {(const void*)&norm_back_long_kernel<XT, WT>, 1024, 1};
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

static int launch_norm(NormArgs& a, int x_type, int w_type, void* stream) {
    int num_cu = 0;
    const int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    const RowPlan p = with_types(
        x_type, w_type, a.d, [&](auto x, auto w, auto r) { return norm_plan<x(), w(), r()>(a.rows, a.d, num_cu); });
    const int64_t grid = std::min<int64_t>((a.rows + p.rows_per_block - 1) / p.rows_per_block, 1 << 20);
    void* args[] = {&a};
    return launch(p.fn, dim3((unsigned)grid), p.threads, args, stream);
}

// Rows of no elements leave their scales and rstd, where there are any.
static int empty_rows(float* scale, float* rstd, long long rows, float eps, void* stream) {
    if (!aligned(scale, GEMM_BT_F32) || !aligned(rstd, GEMM_BT_F32)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!scale && !rstd) return GEMM_BT_OK;
    int num_cu = 0;
    const int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    void* args[] = {&scale, &rstd, &rows, &eps};
    return launch((const void*)&empty_rows_kernel, dim3((unsigned)std::min<int64_t>((rows + 255) / 256, 8 * num_cu)), 256, args,
                  stream);
}

static RowPlan norm_back_plan_of(int x_type, int w_type, int64_t d) {
    return with_types(x_type, w_type, d, [&](auto x, auto w, auto r) { return norm_back_plan<x(), w(), r()>(d); });
}
// The kernel for few rows, or none: while dy and h stay in the caches, reading
// them twice costs less than a second launch and its partial sums, as long as
// each group of lanes has at most 8 rows to sum (us, bf16, two launches vs
// one: 1 x 4096 5.4 vs 3.2, 128 x 8192 10.4 vs 5.3, 512 x 4096 15.3 vs 8.8, 512 x
// 8192 17.5 vs 13.7; with 16 rows to a group 1000 x 2050 fp32 13.1 vs 14.3, 400 x
// 1023 bf16 7.0 vs 9.2, with 32 1000 x 2048 11.3 vs 19.8, 2048 x 4096 22.5 vs 27.0).  Threads in a power of two: the
// last step halves their groups.
template <int XT, int WT, bool R>
static RowPlan norm_back_few(int64_t rows, int64_t d) {
    const int64_t chunks = (d + 7) / 8;
    auto pow2 = [](int64_t n) {
        int t = 256;
        while (t < n) t *= 2;
        return t;
    };
    if (chunks > 2048 || rows * d > (4 << 20)) return {nullptr, 0, 0};
    RowPlan p;
    if (chunks <= 64) p = {(const void*)&norm_back_few_kernel<XT, WT, 1, true, R>, 256, 4};
    else if (chunks <= 1024) p = {(const void*)&norm_back_few_kernel<XT, WT, 1, false, R>, pow2(chunks), 1};
    else p = {(const void*)&norm_back_few_kernel<XT, WT, 2, false, R>, 1024, 1};
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
static ActBackPlan act_back_plan(int64_t rows, int64_t n, int num_cu) {
    ActBackPlan p;
    int lanes = 64;
    const bool r = ragged(n);
    auto kernel = [&](auto l) {
        lanes = l();
        p.fn = r ? (const void*)&act_back_kernel<l(), true> : (const void*)&act_back_kernel<l(), false>;
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
    if (d == 0) return empty_rows(codes ? scale : nullptr, rstd, rows, eps, stream);
    if (!x || !weight || !y) return GEMM_BT_ERR_INVALID_VALUE;
    if (!stride_ok(ldx, d) || (residual && !stride_ok(ldr, d))) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(residual, x_dtype) || !aligned(h, x_dtype) || !aligned(weight, w_dtype) ||
        (!codes && !aligned(y, y_dtype)) || !aligned(scale, GEMM_BT_F32) || !aligned(rstd, GEMM_BT_F32))
        return GEMM_BT_ERR_INVALID_VALUE;
    NormArgs a = {x, residual, weight, y, h, scale, rstd, rows, ldx, ldr, (int)d, eps, y_dtype};
    return launch_norm(a, x_dtype, w_dtype, stream);
}

int gemm_bt_quantize_rows(const void* x, int64_t ldx, void* q, float* scale, int64_t rows, int64_t d, int x_dtype,
                          int q_dtype, void* stream) {
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (!float_type(x_dtype) || (q_dtype != GEMM_BT_FP8_E4M3 && q_dtype != GEMM_BT_INT8)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_BT_OK;
    if (!scale) return GEMM_BT_ERR_INVALID_VALUE;
    if (d == 0) return empty_rows(scale, nullptr, rows, 0.0f, stream);
    if (!x || !q || !stride_ok(ldx, d)) return GEMM_BT_ERR_INVALID_VALUE;
    if (!aligned(x, x_dtype) || !aligned(scale, GEMM_BT_F32)) return GEMM_BT_ERR_INVALID_VALUE;
    NormArgs a = {x, nullptr, nullptr, q, nullptr, scale, nullptr, rows, ldx, 0, (int)d, 0.0f, q_dtype};
    return launch_norm(a, x_dtype, x_dtype, stream);
}

int gemm_bt_rms_norm_backward_workspace(int64_t rows, int64_t d, size_t* bytes) {
    if (!bytes) return GEMM_BT_ERR_INVALID_VALUE;
    *bytes = 0;
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    // (the plans' grids do not depend on the types, nor on whole chunks)
    if (norm_back_few<GEMM_BT_BF16, GEMM_BT_BF16, false>(rows, d).fn) return GEMM_BT_OK;
    *bytes = (size_t)(norm_back_grid(norm_back_plan_of(GEMM_BT_BF16, GEMM_BT_BF16, d), rows, plan_cus()) * d * 4);
    return GEMM_BT_OK;
}

int gemm_bt_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const void* weight,
                              const float* rstd, const void* dh, int64_t ld_dh, void* dx, void* dweight, int64_t rows,
                              int64_t d, int x_dtype, int w_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows < 0 || d < 0) return GEMM_BT_ERR_INVALID_VALUE;
    if (!float_type(x_dtype) || !weight_type_ok(x_dtype, w_dtype)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d > kMaxColumns || rows > (1LL << 31)) return GEMM_BT_ERR_UNSUPPORTED;
    if (d == 0) return GEMM_BT_OK;
    if (!dweight || !aligned(dweight, w_dtype)) return GEMM_BT_ERR_INVALID_VALUE;
    if (rows > 0) {
        // (the few-rows kernel's sums for dweight read dy and h while dx is written)
        if (!dy || !h || !weight || !rstd || !dx || dx == dy || dx == h) return GEMM_BT_ERR_INVALID_VALUE;
        if (!stride_ok(ld_dy, d) || !stride_ok(ldh, d) || (dh && !stride_ok(ld_dh, d))) return GEMM_BT_ERR_INVALID_VALUE;
        if (!aligned(dy, x_dtype) || !aligned(h, x_dtype) || !aligned(dh, x_dtype) || !aligned(dx, x_dtype) ||
            !aligned(weight, w_dtype) || !aligned(rstd, GEMM_BT_F32) || !aligned(workspace, GEMM_BT_F32))
            return GEMM_BT_ERR_INVALID_VALUE;
    }
    int num_cu = 0;
    int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    int64_t grid = 0;
    if (rows > 0) {
        const RowPlan few = with_types(
            x_dtype, w_dtype, d, [&](auto x, auto w, auto r) { return norm_back_few<x(), w(), r()>(rows, d); });
        if (few.fn) {
            NormBackArgs a = {dy, h, weight, rstd, dh, dx, nullptr, rows, ld_dy, ldh, ld_dh, (int)d, 0};
            int row_blocks = (int)((rows + few.rows_per_block - 1) / few.rows_per_block);
            void* args[] = {&a, &row_blocks, &dweight};
            return launch(few.fn, dim3((unsigned)(row_blocks + (d + 63) / 64)), few.threads, args, stream);
        }
        const RowPlan p = norm_back_plan_of(x_dtype, w_dtype, d);
        grid = norm_back_grid(p, rows, num_cu);
        if (!workspace || workspace_bytes < (size_t)(grid * d * 4)) return GEMM_BT_ERR_INVALID_VALUE;
        NormBackArgs a = {dy, h, weight, rstd, dh, dx, (float*)workspace, rows, ld_dy, ldh, ld_dh, (int)d,
                          whole_chunks(dy, ld_dy, x_dtype) && whole_chunks(h, ldh, x_dtype) && whole_chunks(dh, ld_dh, x_dtype)};
        void* args[] = {&a};
        st = launch(p.fn, dim3((unsigned)grid), p.threads, args, stream);
        if (st != GEMM_BT_OK) return st;
    }
    return fold((const float*)workspace, dweight, w_dtype, grid, d, stream);
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
