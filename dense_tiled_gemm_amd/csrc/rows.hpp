// rows.hpp -- what norm.hip and linear_back.hip share: the fold of partial
// column sums, and the backward pass of an activation.
#pragma once

#include "epilogue.hpp"

namespace gbt {

// out[j] = sum over `parts` rows of d fp32 partial sums.
struct FoldArgs {
    const float* partials;
    void* out;
    long long d;
    int parts, out_type;
};

inline unsigned fold_blocks(int64_t d) { return (unsigned)((d + 15) / 16); }

// Block `blk` of the fold: 16 columns, in an order that depends on `parts`
// only.  NT / 16 threads per column take every (NT / 16)-th row, 8 of them in
// flight at a time, then a tree.
template <int NT>
__device__ __forceinline__ void fold_columns(const FoldArgs& a, long long blk, float (*sums)[17]) {
    constexpr int G = NT / 16;
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const long long j = blk * 16 + c;
    float s = 0.0f;
    if (j < a.d) {
        for (int r = k; r < a.parts; r += 8 * G) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r + e * G < a.parts ? a.partials[(size_t)(r + e * G) * a.d + j] : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];
        }
    }
    sums[k][c] = s;
    __syncthreads();
    if (k == 0 && j < a.d) {
        float v[G];
#pragma unroll
        for (int i = 0; i < G; ++i) v[i] = sums[i][c];
#pragma unroll
        for (int w = G / 2; w > 0; w >>= 1)
#pragma unroll
            for (int i = 0; i < w; ++i) v[i] += v[i + w];
        store1(a.out, a.out_type, (size_t)j, v[0]);
    }
}

// dz = dy act'(preact) and, in partials, its sums over blocks of rows.
struct ActBackArgs {
    const void* dy;
    const void* preact;  // nullptr: no activation
    void* dz;            // nullptr: not wanted
    float* partials;     // nullptr: no column sums; else act_back_parts rows of n sums of dz
    long long rows;
    int n;
    int ldz;             // row pitch of dz, n or that rounded up to whole groups of 8 (the rest is zeros)
    int rows_per_block;  // set by launch_act_back
    int type, preact_type, act;
    int nt;              // set by launch_act_back: read past the caches
};
int64_t act_back_parts(int64_t rows, int64_t n, int num_cu);
int launch_act_back(ActBackArgs a, int num_cu, void* stream);

// The same for a gated pair: z has rows of 2 n elements, the gate's and then the
// other factor's, and so has dz (pitch ldz >= 2 n):
//   dz[:n] = dy z[n:] act'(z[:n]),  dz[n:] = dy act(z[:n]);
// partials hold rows of 2 n sums.
int64_t gated_back_parts(int64_t rows, int64_t n, int num_cu);
int launch_gated_back(ActBackArgs a, int num_cu, void* stream);

// ---- host helpers ----------------------------------------------------------------

inline int launch(const void* fn, dim3 grid, int threads, void** args, void* stream) {
    if (hipLaunchKernel(fn, grid, dim3(threads), args, 0, (hipStream_t)stream) != hipSuccess) {
        (void)hipGetLastError();
        return GEMM_BT_ERR_LAUNCH;
    }
    return GEMM_BT_OK;
}
inline bool float_type(int t) { return t == GEMM_BT_F32 || t == GEMM_BT_F16 || t == GEMM_BT_BF16; }
inline bool aligned(const void* p, int t) { return (uintptr_t)p % elem_size(t) == 0; }

}  // namespace gbt
