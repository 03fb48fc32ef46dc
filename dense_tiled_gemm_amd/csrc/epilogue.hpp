// epilogue.hpp -- what follows a product inside its kernel: scales, bias,
// activation and residual, with one rounding at the end (gfx950).
//
//   Z[i][j] = row_scale[i] * col_scale[j] * sum_k A[i][k] B[j][k] + bias[j]
//   C[i][j] = act(Z[i][j]) + residual[i][j]
//
// Z and everything after it is held in fp32 and rounded once into C (and once
// into the kept pre-activation, if there is one).  All operands but the sum
// are optional.  Element types are run-time values that are the same for the
// whole launch, so each is one scalar branch per group of 8 outputs and one
// kernel serves every combination of them.
#pragma once

#include "common.hpp"

namespace gbt {

// The run-time arguments of an epilogue.  `mode` holds which terms there are,
// the element types and the activation, packed: the kernels test its bits
// where they need them, since one condition held per term and type for the
// length of the tile would not fit the scalar registers.
struct EpiArgs {
    const float* row_scale;
    const float* col_scale;
    const void* bias;
    const void* residual;
    void* preact;
    int mode;
};
enum {
    EPI_ROW_SCALE = 1,
    EPI_COL_SCALE = 2,
    EPI_BIAS = 4,
    EPI_RESIDUAL = 8,
    EPI_PREACT = 16,
    EPI_BIAS_TYPE = 8,  // shifts of the 2-bit types (GEMM_BT_F32, GEMM_BT_F16 or GEMM_BT_BF16) ...
    EPI_RESIDUAL_TYPE = 10,
    EPI_PREACT_TYPE = 12,
    EPI_OUT_TYPE = 14,
    EPI_ACT = 16  // ... and of the activation
};
__host__ __device__ inline int epi_type(int mode, int shift) { return (mode >> shift) & 3; }

// 16 bytes at any element alignment (the target's unaligned access mode).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

__device__ __forceinline__ u32x4 load16(const void* p, bool nt = false) {
    return nt ? __builtin_nontemporal_load((const u32x4_any*)p) : *(const u32x4_any*)p;
}
__device__ __forceinline__ void store16_nt(void* p, u32x4 v) { __builtin_nontemporal_store(v, (u32x4_any*)p); }

__host__ __device__ inline int elem_size(int t) { return t == GEMM_BT_F32 ? 4 : 2; }

// A per-thread value that the compiler takes for new: conditions on it are
// then made where they are used.  Kept for the length of a tile, each would
// hold a lane mask in two scalar registers.
__device__ __forceinline__ int renew(int n) {
    asm volatile("" : "+v"(n));
    return n;
}

// Eight consecutive elements as they lie in memory: 16-bit ones in `a`, fp32
// ones in `a` and `b`.
struct Raw8 {
    u32x4 a, b;
};

// Elements i .. i+n-1 (n in 1..8) of an array of type t; the rest are zero.
// nt: read once, not kept in the caches.
__device__ __forceinline__ Raw8 load_raw8(const void* p, int t, size_t i, int n, bool nt = false) {
    Raw8 r = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    if (t == GEMM_BT_F32) {
        const u32* s = (const u32*)p + i;
        if (n >= 8) {
            r.a = load16(s, nt);
            r.b = load16(s + 4, nt);
        } else {
            n = renew(n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e < n) r.a[e] = s[e];
                if (e + 4 < n) r.b[e] = s[e + 4];
            }
        }
    } else {
        const u16* s = (const u16*)p + i;
        if (n >= 8) {
            r.a = load16(s, nt);
        } else {
            n = renew(n);
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) r.a[e >> 1] |= (u32)s[e] << (16 * (e & 1));
        }
    }
    return r;
}

__device__ __forceinline__ void decode8(const Raw8& r, int t, float (&v)[8]) {
    if (t == GEMM_BT_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 x = r.a[e], y = r.b[e];
            v[e] = as_f32(x);
            v[e + 4] = as_f32(y);
        }
    } else if (t == GEMM_BT_BF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 x = r.a[e];
            v[2 * e] = as_f32(x << 16);
            v[2 * e + 1] = as_f32(x & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 x = r.a[e];
            v[2 * e] = decode16<GEMM_BT_F16>(x & 0xFFFFu);
            v[2 * e + 1] = decode16<GEMM_BT_F16>(x >> 16);
        }
    }
}

// v rounded to nearest even into type t, at elements i .. i+n-1 (n in 1..8).
// Non-temporal: written once and not read back by the kernel.
__device__ __forceinline__ void store8(void* p, int t, size_t i, int n, const float (&v)[8]) {
    if (t == GEMM_BT_F32) {
        u32* s = (u32*)p + i;
        if (n >= 8) {
            store16_nt(s, u32x4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])});
            store16_nt(s + 4, u32x4{as_u32(v[4]), as_u32(v[5]), as_u32(v[6]), as_u32(v[7])});
        } else {
            n = renew(n);
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) s[e] = as_u32(v[e]);
        }
    } else {
        u32x4 w;
        if (t == GEMM_BT_BF16)
            w = u32x4{pack2<GEMM_BT_BF16>(v[0], v[1]), pack2<GEMM_BT_BF16>(v[2], v[3]), pack2<GEMM_BT_BF16>(v[4], v[5]),
                      pack2<GEMM_BT_BF16>(v[6], v[7])};
        else
            w = u32x4{pack2<GEMM_BT_F16>(v[0], v[1]), pack2<GEMM_BT_F16>(v[2], v[3]), pack2<GEMM_BT_F16>(v[4], v[5]),
                      pack2<GEMM_BT_F16>(v[6], v[7])};
        u16* s = (u16*)p + i;
        if (n >= 8) {
            store16_nt(s, w);
        } else {
            n = renew(n);
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) s[e] = (u16)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// One element of type t.
__device__ inline float load1(const void* p, int t, size_t i) {
    if (t == GEMM_BT_F32) return ((const float*)p)[i];
    const u32 x = ((const u16*)p)[i];
    return t == GEMM_BT_BF16 ? decode16<GEMM_BT_BF16>(x) : decode16<GEMM_BT_F16>(x);
}
__device__ inline void store1(void* p, int t, size_t i, float v) {
    if (t == GEMM_BT_F32) ((float*)p)[i] = v;
    else if (t == GEMM_BT_BF16) ((u16*)p)[i] = (u16)pack2<GEMM_BT_BF16>(v, 0.0f);
    else ((u16*)p)[i] = (u16)pack2<GEMM_BT_F16>(v, 0.0f);
}

// ---- activations -------------------------------------------------------------

// exp(x) and 1/x of the hardware, which are within 1 ulp; x log2(e) is rounded
// before the exponential, so exp(x) is off by up to 1.25 |x| + 2 units of 2^-24,
// relative.  Carried to the results (units of 2^-24, relative): silu 8 + 1.5 |z|,
// gelu 24 + 1.25 z^2, gelu_tanh 8 + 6 |argument of its exponential|.  z is a
// rounded fp32 value itself, which moves a tail by half as much or so, and
// 16-bit results are rounded at 2^-9 or 2^-12; two or more operations per output
// for the low part of the product would lie open in the epilogue, which nothing
// covers.
__device__ inline float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ inline float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + exp(-x)); exp overflowing to infinity gives 0, underflowing 1.
__device__ inline float sigmoid_f(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

// Phi(-x) = exp(-x^2/2) t p(t), t = 1 / (1 + x/4), for x >= 0: p is a least
// largest relative error fit (4.7e-8 with these fp32 coefficients) of exp(x^2/2)
// Phi(-x) / t on 0 < t <= 1, highest power first, so the tail keeps the relative
// accuracy that the exponential has.
constexpr int kPhiTerms = 10;
__device__ constexpr float kPhi[kPhiTerms] = {1.978199370e-02f, -8.087722957e-02f, 9.559692442e-02f, -3.171735257e-02f,
                                              6.369900703e-02f, 5.897518620e-02f,  8.160310239e-02f, 9.346635640e-02f,
                                              9.973642975e-02f, 9.973556548e-02f};

// The normal distribution's function Phi(z), and exp(-z^2/2).
__device__ inline float normal_cdf(float z, float& gauss) {
    const float x = __builtin_fabsf(z);
    const float t = fast_rcp(__builtin_fmaf(x, 0.25f, 1.0f));
    gauss = fast_exp(-0.5f * x * x);
    float p = kPhi[0];
#pragma unroll
    for (int i = 1; i < kPhiTerms; ++i) p = __builtin_fmaf(p, t, kPhi[i]);
    const float tail = gauss * p * t;
    return z > 0.0f ? 1.0f - tail : tail;
}

// gelu_tanh(z) = z (1 + tanh u) / 2 = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGeluA = 1.5957691216057308f;             // 2 sqrt(2/pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

template <int ACT>
__device__ inline float act_value(float z) {
    if constexpr (ACT == GEMM_BT_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    } else if constexpr (ACT == GEMM_BT_ACT_GELU) {
        float gauss;
        return z * normal_cdf(z, gauss);
    } else if constexpr (ACT == GEMM_BT_ACT_GELU_TANH) {
        return z * sigmoid_f(z * __builtin_fmaf(kGeluB, z * z, kGeluA));
    } else if constexpr (ACT == GEMM_BT_ACT_SILU) {
        return z * sigmoid_f(z);
    } else {
        return z;
    }
}

// The derivative act'(z).
template <int ACT>
__device__ inline float act_slope(float z) {
    if constexpr (ACT == GEMM_BT_ACT_RELU) {
        return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);  // NaN stays NaN
    } else if constexpr (ACT == GEMM_BT_ACT_GELU) {
        float gauss;
        const float p = normal_cdf(z, gauss);
        return __builtin_fmaf(z * 0.3989422804014327f, gauss, p);
    } else if constexpr (ACT == GEMM_BT_ACT_GELU_TANH) {
        const float p = sigmoid_f(z * __builtin_fmaf(kGeluB, z * z, kGeluA));
        // past |z| = 30 p is 0 or 1 and the second term is 0: without the
        // bound z^3 would overflow there and give 0 * infinity
        const float c = __builtin_fminf(__builtin_fmaxf(z, -30.0f), 30.0f);
        return __builtin_fmaf(c * p * (1.0f - p), __builtin_fmaf(3.0f * kGeluB, c * c, kGeluA), p);
    } else if constexpr (ACT == GEMM_BT_ACT_SILU) {
        const float p = sigmoid_f(z);
        return p * __builtin_fmaf(z, 1.0f - p, 1.0f);
    } else {
        return 1.0f;
    }
}

// f(std::integral_constant<int, activation>{}) for a run-time activation: one
// scalar branch around code that is specialised for it.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case GEMM_BT_ACT_RELU: f(std::integral_constant<int, GEMM_BT_ACT_RELU>{}); break;
        case GEMM_BT_ACT_GELU: f(std::integral_constant<int, GEMM_BT_ACT_GELU>{}); break;
        case GEMM_BT_ACT_GELU_TANH: f(std::integral_constant<int, GEMM_BT_ACT_GELU_TANH>{}); break;
        case GEMM_BT_ACT_SILU: f(std::integral_constant<int, GEMM_BT_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, GEMM_BT_ACT_NONE>{}); break;
    }
}

// ---- the tile's epilogue -------------------------------------------------------

// Store the workgroup's BM x BN tile with the epilogue applied.  As in
// store_tile_lds the tile goes through LDS so that global accesses run along
// rows, but it is parked as fp32 sums: the residual, the kept pre-activation
// and C are then each read or written as 8 consecutive elements per thread (a
// wave covers 1 KiB of consecutive bytes of one or more rows), and every
// output is rounded once, after all of its terms.  The residual's loads go out
// before the tile is parked, so that their latency passes behind it.  With NT
// a multiple of the groups per row a thread keeps the same 8 columns
// throughout and holds their bias and scales in registers.  With one tile per
// CU nothing covers it, so its bytes and its arithmetic add to the product's
// time (4096^3 bf16, us: plain kernel 94, bias 100, with gelu_tanh 102, gelu 107,
// and residual 105, and z kept 108: 67 MB more of the residual and z).  INT: the sums are
// int32 bits.  Rows >= M and columns >= N are neither read nor written; the
// caller guarantees that no wave still reads or fills `lds`.
template <bool INT, int FN, int FM, int BM, int BN, int WM, int NT, int LDS_BYTES, int MF>
__device__ __forceinline__ void store_tile_epi(const typename AccBlock<MF>::type (&acc)[FN][FM], unsigned char* lds, void* C,
                                      int M, int N, int m0, int n0, int mw, int nw, int wm, int tid, const EpiArgs& e) {
    typedef AccBlock<MF> AB;
    constexpr int ROWB = BN * 4, CPR = ROWB / 16;
    constexpr int P = BM * ROWB <= LDS_BYTES ? 1 : WM;
    constexpr int RP = BM / P;    // tile rows per pass
    constexpr int GPR = BN / 8;   // groups of 8 columns per row
    constexpr int IT = RP * GPR / NT;
    constexpr bool FIXED = NT % GPR == 0;  // every group of a thread has the same columns
    static_assert(CPR == 24 || (CPR >= 8 && (CPR & (CPR - 1)) == 0), "row chunks");
    static_assert(RP * ROWB <= LDS_BYTES, "a pass must fit in LDS");
    static_assert(IT * NT == RP * GPR, "the row copy covers a pass in whole rounds of NT threads");
    const int mlim = M - m0, nlim = N - n0;
    const int lane = tid & 63;
    // the mode, taken anew wherever it is tested (see EpiArgs)
    auto mode = [&]() __attribute__((always_inline)) {
        int m = e.mode;
        asm volatile("" : "+s"(m));
        return m;
    };
    float cs[8], cb[8];
    auto columns = [&](int g) __attribute__((always_inline)) {
        const int n = min(8, nlim - 8 * g), md = mode();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            cs[x] = 1.0f;
            cb[x] = 0.0f;
        }
        if (n <= 0) return;
        if (md & EPI_COL_SCALE) decode8(load_raw8(e.col_scale, GEMM_BT_F32, (size_t)n0 + 8 * g, n), GEMM_BT_F32, cs);
        if (md & EPI_BIAS) {
            const int t = epi_type(md, EPI_BIAS_TYPE);
            decode8(load_raw8(e.bias, t, (size_t)n0 + 8 * g, n), t, cb);
        }
    };
    if constexpr (FIXED) columns(tid % GPR);
    constexpr int U = IT % 4 == 0 ? 4 : (IT % 3 == 0 ? 3 : IT);  // groups whose residuals are in flight
#pragma unroll 1
    for (int p = 0; p < P; ++p) {
        Raw8 res[U];
        float rs[U];
        // the residual and the row's scale of round it
        auto fetch = [&](int it, Raw8& rv, float& sv) __attribute__((always_inline)) {
            const int q = it * NT + renew(tid);
            const int g = q % GPR, row = p * RP + q / GPR;
            const int md = mode();
            sv = 1.0f;
            if (it < IT && row < mlim && 8 * g < nlim) {
                if (md & EPI_ROW_SCALE) sv = e.row_scale[(size_t)m0 + row];
                if (md & EPI_RESIDUAL)
                    rv = load_raw8(e.residual, epi_type(md, EPI_RESIDUAL_TYPE), (size_t)(m0 + row) * N + n0 + 8 * g,
                                   min(8, nlim - 8 * g));
            }
        };
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            fetch(u, res[u], rs[u]);
        });
        if (P == 1 || wm == p) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const int r = (mw + MF * j + AB::row(lane)) % RP;  // tile row within the pass
#pragma unroll
                    for (int g = 0; g < AB::regs / 4; ++g) {
                        const int c = (nw + MF * i + AB::col(lane, g)) / 4;
                        float v[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float s = acc[i][j][4 * g + x];
                            v[x] = INT ? (float)(int)as_u32(s) : s;
                        }
                        *(u32x4*)(lds + r * ROWB + epi_chunk(c, r, CPR) * 16) =
                            u32x4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])};
                    }
                }
        }
        __syncthreads();
#pragma unroll 1
        for (int it0 = 0; it0 < IT; it0 += U)
            static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int q = (it0 + u) * NT + renew(tid);
                const int g = q % GPR, r = q / GPR, row = p * RP + r;
                if (row < mlim && 8 * g < nlim) {
                    if constexpr (!FIXED) columns(g);
                    const int n = min(8, nlim - 8 * g), md = mode();
                    const size_t at = (size_t)(m0 + row) * N + n0 + 8 * g;
                    const u32x4 lo = *(const u32x4*)(lds + r * ROWB + epi_chunk(2 * g, r, CPR) * 16);
                    const u32x4 hi = *(const u32x4*)(lds + r * ROWB + epi_chunk(2 * g + 1, r, CPR) * 16);
                    float z[8];
                    decode8(Raw8{lo, hi}, GEMM_BT_F32, z);
#pragma unroll
                    for (int x = 0; x < 8; ++x) z[x] = __builtin_fmaf(z[x] * rs[u], cs[x], cb[x]);
                    if (md & EPI_PREACT) store8(e.preact, epi_type(md, EPI_PREACT_TYPE), at, n, z);
                    with_act(md >> EPI_ACT, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
                        for (int x = 0; x < 8; ++x) z[x] = act_value<decltype(act)::value>(z[x]);
                    });
                    if (md & EPI_RESIDUAL) {
                        float v[8];
                        decode8(res[u], epi_type(md, EPI_RESIDUAL_TYPE), v);
#pragma unroll
                        for (int x = 0; x < 8; ++x) z[x] += v[x];
                    }
                    store8(C, epi_type(md, EPI_OUT_TYPE), at, n, z);
                }
                fetch(it0 + U + u, res[u], rs[u]);
            });
        __syncthreads();
    }
}

// What an epilogue adds to outputs j .. j+n-1 (n in 0..4) of row i: fetched
// ahead of the sums, so that its latency passes behind them.
struct Epi4 {
    float rs, cs[4], cb[4], res[4];
};
__device__ __forceinline__ Epi4 load_epi4(int N, size_t i, int j, int n, const EpiArgs& e) {
    Epi4 v = {1.0f, {1.0f, 1.0f, 1.0f, 1.0f}, {0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    const int md = e.mode;
    if (n > 0 && (md & EPI_ROW_SCALE)) v.rs = e.row_scale[i];
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (x < n) {
            if (md & EPI_COL_SCALE) v.cs[x] = e.col_scale[j + x];
            if (md & EPI_BIAS) v.cb[x] = load1(e.bias, epi_type(md, EPI_BIAS_TYPE), j + x);
            if (md & EPI_RESIDUAL) v.res[x] = load1(e.residual, epi_type(md, EPI_RESIDUAL_TYPE), i * N + j + x);
        }
    return v;
}
__device__ __forceinline__ void store4(void* p, int t, size_t i, int n, const float (&v)[4]) {
    if (n == 4) {
        if (t == GEMM_BT_F32)
            *(u32x4_any*)((u32*)p + i) = u32x4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])};
        else if (t == GEMM_BT_BF16)
            *(u32x2_any*)((u16*)p + i) = u32x2{pack2<GEMM_BT_BF16>(v[0], v[1]), pack2<GEMM_BT_BF16>(v[2], v[3])};
        else
            *(u32x2_any*)((u16*)p + i) = u32x2{pack2<GEMM_BT_F16>(v[0], v[1]), pack2<GEMM_BT_F16>(v[2], v[3])};
    } else {
#pragma unroll
        for (int x = 0; x < 3; ++x)
            if (x < n) store1(p, t, i + x, v[x]);
    }
}
__device__ __forceinline__ void store_epi4(const float (&s)[4], const Epi4& v, void* C, int N, size_t i, int j, int n,
                                           const EpiArgs& e) {
    const size_t at = i * N + j;
    const int md = e.mode;
    float z[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) z[x] = __builtin_fmaf(s[x] * v.rs, v.cs[x], v.cb[x]);
    if (md & EPI_PREACT) store4(e.preact, epi_type(md, EPI_PREACT_TYPE), at, n, z);
    with_act(md >> EPI_ACT, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int x = 0; x < 4; ++x) z[x] = act_value<decltype(act)::value>(z[x]);
    });
    if (md & EPI_RESIDUAL)
#pragma unroll
        for (int x = 0; x < 4; ++x) z[x] += v.res[x];
    store4(C, epi_type(md, EPI_OUT_TYPE), at, n, z);
}

}  // namespace gbt
