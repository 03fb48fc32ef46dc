// skinny_dma.hpp -- streaming MFMA kernel for C = A * B^T with M <= 16
// (gfx950).
//
// With at most 16 rows in A the product is bound by reading B once from HBM
// (2 bytes per multiply-add pair): a 16-row tile has an arithmetic intensity
// of about 16 FLOP per byte ("Chapter 7: Writing custom kernels with Pallas",
// section 6.3, intensity bm*bn/(bm+bn) per tile), far below the MI355X
// MFMA/HBM ridge.  So this kernel is organised around keeping enough bytes of
// B in flight, not around data reuse:
//   * each workgroup owns BN rows of B and the whole K range; B and the 16
//     rows of A stream through an STAGES-deep LDS ring, KB elements of K per
//     stage, with buffer_load_dwordx4 ... lds (no register staging), so about
//     (STAGES-1) * (16 + BN) * KB * 2 bytes per workgroup are in flight.  HBM
//     streams B fastest when each workgroup walks few rows at a time, so BN
//     may be 8: the MFMA's first operand then repeats those 8 rows and the
//     repeated outputs are never stored (the matrix cores have ample slack
//     here), and LDS holds only the 8 real rows, so more workgroups fit;
//   * rows are 2*KB bytes long in LDS; the 16-byte chunk index is XORed with
//     the low 4 row bits so the 16 rows read by one MFMA operand load fall
//     in 16 different bank groups of the 64-bank LDS (the same swizzle idea as
//     the tiled kernel, "Optimizing Blackwell matrix multiplication in Mojo
//     (part 2)", section "Kernel 3: Swizzling");
//   * the W waves split each stage's 32-element k-blocks; each runs
//     v_mfma_f32_16x16x32_{bf16,f16} with B as first operand (rows = columns
//     of C) and A as second, fp32 accumulators; at the end the W partial sums
//     are added through LDS in a fixed order, rounded once and stored masked
//     to i < M, j < N;
//   * rows of A past M and of B past N, and chunks at k >= K, read as zero
//     through the buffer range check ("Chapter 7", section 4.3: zero the K
//     overhang of both operands);
//   * rows need only 2-byte alignment: the LDS DMA moves the whole 16-byte
//     chunks below Kf = K & ~7 from any even address, and the last K - Kf
//     (1 to 7) elements of each row, fetched with 16-bit loads before the
//     loop, form one more zero-padded k-block multiplied after it, so each
//     sum still runs over k in increasing order.
#pragma once

#include "common.hpp"
#include "dma_kernel.hpp"
#include "epilogue.hpp"

namespace gbt {

// acc += the products of one 64-byte k-block: 16 bytes of one row per lane and
// operand.  16-bit inputs: one 16x16x32 instruction; int8: one 16x16x64 (int32
// sums in the accumulator's bits); 8-bit floats: two 16x16x32, one per 8-byte
// half (the same half of A and of B, so the sum over both is the full one).
template <int IN>
__device__ __forceinline__ f32x4 skinny_mma(u32x4 b, u32x4 a, f32x4 c) {
    if constexpr (IN == GEMM_BT_INT8) {
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a),
                                                                               __builtin_bit_cast(i32x4, c), 0, 0, 0));
    } else if constexpr (in_size(IN) == 1) {
        const long b0 = (long)b[0] | (long)b[1] << 32, b1 = (long)b[2] | (long)b[3] << 32;
        const long a0 = (long)a[0] | (long)a[1] << 32, a1 = (long)a[2] | (long)a[3] << 32;
        if constexpr (IN == GEMM_BT_FP8_E4M3)
            return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(b1, a1, __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(b0, a0, c, 0, 0, 0), 0,
                                                              0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf8_bf8(b1, a1, __builtin_amdgcn_mfma_f32_16x16x32_bf8_bf8(b0, a0, c, 0, 0, 0), 0,
                                                              0, 0);
    } else {
        return Mfma<IN>::m16x16x32(b, a, c);
    }
}

// The kernel's body.  `epi` is the epilogue's arguments (EpiArgs, or SkinnyGated
// for the gated one), or nothing (SkinnyPlain): then the sums are rounded into C
// as they are.  Gated: the BN rows of B are BN / 2 of its first N rows and the same
// of its second N rows, so a lane finds the other product of its outputs 2 BN lanes
// on.
struct SkinnyPlain {};
struct SkinnyGated {
    EpiArgs e;
};
// One scale per block of 128 (see BLK in dma_kernel.hpp): a stage holds whole
// blocks, and the scales of its rows come with it, 4 bytes per lane.  A block's
// sums start from zero and are added to the others times both scales.
template <bool TALL, bool WIDE>
struct SkinnyBlocks {
    EpiArgs e;
    BlkArgs b;
};
template <class T>
struct is_blocks : std::false_type {
    static constexpr bool wide = false;
};
template <bool TALL, bool WIDE>
struct is_blocks<SkinnyBlocks<TALL, WIDE>> : std::true_type {
    static constexpr bool tall = TALL, wide = WIDE;  // wide: fp32 results (see kBlkWide)
};
template <int IN, int OUT, int BN, int KB, int STAGES, int W, int ROT, class Epi>
__device__ __forceinline__ void skinny_body(const u16* __restrict__ A, const u16* __restrict__ B, void* __restrict__ C,
                                            int M, int N, int K, int vec_store, const Epi& epi) {
    constexpr int AR = 16;                 // rows of A held (M <= 16)
    constexpr int ESZ = in_size(IN);       // bytes per input element
    constexpr int EPC = 16 / ESZ;          // elements per 16-byte chunk
    constexpr int CPR = KB / EPC;          // 16-byte chunks per row per stage
    constexpr int ROWB = KB * ESZ;         // bytes per row per stage
    constexpr int RPI = 1024 / ROWB;       // rows per wave load instruction
    constexpr int BR = BN < 16 ? BN : 16;   // distinct B rows under one 16-row MFMA operand
    constexpr int BNP = BN;                 // B rows held in LDS
    constexpr int A_LOADS = AR / RPI, B_LOADS = BN / RPI;
    constexpr int LOADS = (A_LOADS + B_LOADS) / W;  // per wave per stage
    constexpr int STAGE_BYTES = (AR + BNP) * ROWB;
    constexpr int KBLK = ROWB / 64;        // k-blocks of 64 bytes per stage, 16 bytes per lane
    constexpr int KPW = KBLK / W;          // k-blocks per wave per stage
    constexpr int NBLK = BN < 16 ? 1 : BN / 16;
    constexpr int PEND = (STAGES - 2) * LOADS;
    constexpr int OSZ = OUT == GEMM_BT_F32 ? 4 : 2;
    static_assert(RPI >= 1 && ROWB * RPI == 1024, "stage rows must tile 1 KiB loads");
    static_assert(STAGES >= 2 && BN % RPI == 0 && (BN % 16 == 0 || BN < 16), "B rows per workgroup");
    static_assert((A_LOADS + B_LOADS) % W == 0, "loads split evenly over waves");
    static_assert(KBLK % W == 0, "k-blocks split evenly over waves");
    static_assert(CPR >= 16, "swizzle needs 16 chunks per row");
    static_assert(PEND < 64, "vmcnt range");
    static_assert(STAGES * STAGE_BYTES + W * NBLK * 64 * 16 <= 160 * 1024, "LDS budget");
    static_assert(16 % BR == 0, "B rows repeat evenly under a 16-row operand");
    static_assert(LOADS * W == A_LOADS + B_LOADS, "loads split evenly");

    __shared__ __attribute__((aligned(1024))) unsigned char lds[STAGES * STAGE_BYTES];
    __shared__ f32x4 red[W][NBLK][64];
    constexpr bool BLOCKS = is_blocks<Epi>::value;
    constexpr int BPS = KB / 128;  // blocks of 128 per stage
    static_assert(!BLOCKS || (W == 1 && ESZ == 1 && NBLK == 1 && ROT == 0 && BPS * AR <= 64 && BPS * BN <= 64), "a lane per scale");
    // a stage's scales: those of A, block by block, in the first 64 places, those of B in the others
    __shared__ float scales[BLOCKS ? STAGES : 1][BLOCKS ? 128 : 1];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr bool GATE = std::is_same_v<Epi, SkinnyGated>;
    constexpr int BNR = GATE ? BN / 2 : BN;  // columns of C per workgroup
    static_assert(!GATE || (NBLK == 1 && BNR % 4 == 0 && BNR % RPI == 0), "whole lanes, and a load lies in one half of B");
    const int n0 = blockIdx.x * BNR;
    const int rows_a = min(AR, M), rows_b = min(BNR, N - n0);
    const i32x4 ra = rsrc_words(A, (u32)rows_a * (u32)K * (u32)ESZ);
    const i32x4 rb = rsrc_words((const unsigned char*)B + (size_t)n0 * K * ESZ, (u32)rows_b * (u32)K * (u32)ESZ);
    const i32x4 rb2 = GATE ? rsrc_words((const unsigned char*)B + (size_t)(N + (int64_t)n0) * K * ESZ, (u32)rows_b * (u32)K * (u32)ESZ) : rb;
    const u32 row_bytes = (u32)K * (u32)ESZ;

    // Loads: stage rows 0..15 hold A, rows 16..16+BN-1 hold B.  Load
    // instruction j (j = wave + i*W) fills stage rows j*RPI .. j*RPI+RPI-1;
    // lane L writes row j*RPI + L/CPR at physical chunk L%CPR, fetching the
    // logical chunk (L%CPR) ^ (row & 15) of that row.
    const int lrow = lane / CPR, lphys = lane % CPR;
    u32 off[LOADS];
    int kc[LOADS];
    bool is_a[LOADS], is_up[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int j = wave + i * W;
        const int srow = j * RPI + lrow;  // stage row
        const int c = lphys ^ (srow & 15);
        const bool a = srow < AR;
        const bool up = GATE && srow >= AR + BNR;
        const int grow = a ? srow : srow - AR - (up ? BNR : 0);  // row within A or within this block of B
        off[i] = (u32)grow * row_bytes + (u32)c * 16u;
        kc[i] = c * EPC;
        is_a[i] = a;
        is_up[i] = up;
    }
    const int Kf = K & ~(EPC - 1);  // whole 16-byte chunks: through the LDS DMA (8-bit inputs: all of K)
    const int nk = (Kf + KB - 1) / KB;
    // ROT > 0: workgroup g walks the K steps starting at (g * ROT) mod nk and
    // wraps around, so that concurrent workgroups read different K offsets
    const int k0 = ROT > 0 && nk > 0 ? (int)(((long long)blockIdx.x * ROT) % nk) : 0;
    // the lane's scales of A and of B: row lane % 16 (B: % BN) of block lane / 16 (/ BN) of the stage
    [[maybe_unused]] u32 so[2] = {kOutOfRange, kOutOfRange};
    [[maybe_unused]] int sk_block[2] = {0, 0};
    [[maybe_unused]] long long s_first = 0;
    if constexpr (BLOCKS) {
        constexpr bool tall = is_blocks<Epi>::tall;
        sk_block[0] = lane / AR;
        sk_block[1] = lane / BN;
        s_first = tall ? n0 >> 7 : n0;
        const int ra_ = lane % AR, rb_ = lane % BN;
        if (ra_ < rows_a && sk_block[0] < BPS) so[0] = ((u32)ra_ * (u32)epi.b.a.row + (u32)sk_block[0] * (u32)epi.b.a.block) * 4u;
        if (rb_ < rows_b && sk_block[1] < BPS)
            so[1] = ((u32)(tall ? ((n0 + rb_) >> 7) - (int)s_first : rb_) * (u32)epi.b.b.row + (u32)sk_block[1] * (u32)epi.b.b.block) * 4u;
    }
    auto issue_scales = [&](int stage, int kt) {
        if constexpr (BLOCKS) {
            const int left = (K + 127) / 128 - kt * BPS;  // blocks from this stage on
            const long long at = (long long)kt * BPS;
            dma4(rsrc_words(epi.b.a.s + at * epi.b.a.block, 0x7FFFFFFFu), (unsigned char*)scales[stage],
                 sk_block[0] < left ? so[0] : kOutOfRange, 0u);
            dma4(rsrc_words(epi.b.b.s + s_first * epi.b.b.row + at * epi.b.b.block, 0x7FFFFFFFu), (unsigned char*)(scales[stage] + 64),
                 sk_block[1] < left ? so[1] : kOutOfRange, 0u);
        }
    };
    auto issue = [&](int stage, int kstep) {
        const int kt = ROT > 0 ? (kstep + k0 >= nk ? kstep + k0 - nk : kstep + k0) : kstep;
        unsigned char* sbase = lds + stage * STAGE_BYTES;
        const u32 kbytes = (u32)kt * (u32)ROWB;
        const int kleft = Kf - kt * KB;
        issue_scales(stage, kt);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int j = wave + i * W;
            const u32 o = kc[i] < kleft ? off[i] : kOutOfRange;
            // whether load i reads A or B is fixed per (wave, i) and uniform
            // B is read exactly once: non-temporal; A is re-read by every
            // workgroup and should stay in L2
            if (is_a[i]) dma16<false>(ra, sbase + j * 1024, o, kbytes);
            else if (GATE && is_up[i]) dma16<true>(rb2, sbase + j * 1024, o, kbytes);
            else dma16<true>(rb, sbase + j * 1024, o, kbytes);
        }
    };

    // Operand reads: lane (r = l%16, q = l/16) reads row r of a 16-row block,
    // logical chunk 4*kb + q.
    const int r16 = lane & 15, q = lane >> 4;
    // K tail: in the extra k-block, lanes with q = 0 hold elements Kf ..
    // Kf + 7 of their row (zeros past K and for rows past M or N); the other
    // lanes' chunks are zero.  Fetched now so the loads hide behind the loop.
    const int tail = ESZ == 2 ? K - Kf : 0;
    u32x4 ta = {0u, 0u, 0u, 0u}, tb[NBLK];
#pragma unroll
    for (int b = 0; b < NBLK; ++b) tb[b] = u32x4{0u, 0u, 0u, 0u};
    if (tail > 0 && wave == 0 && q == 0) {
        auto fetch = [&](const u16* src) {
            u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < tail) v[e >> 1] |= (u32)__builtin_nontemporal_load(src + e) << (16 * (e & 1));
            return v;
        };
        if (r16 < rows_a) ta = fetch(A + (size_t)r16 * K + Kf);
#pragma unroll
        for (int b = 0; b < NBLK; ++b) {
            const int br = 16 * b + (r16 % BR);  // B row of the operand's row r16 within this block
            const bool up = GATE && br >= BNR;
            if (br - (up ? BNR : 0) < rows_b) tb[b] = fetch(B + (size_t)(n0 + (int64_t)br + (up ? (int64_t)N - BNR : 0)) * K + Kf);
        }
    }
    // with an epilogue: what it adds to this lane's outputs, columns n0 + 4 q ..
    // of row lane % 16 (the first block of B rows is the only one there is)
    constexpr bool EPI = !std::is_same_v<Epi, SkinnyPlain>;
    static_assert(!EPI || (NBLK == 1 && W == 1), "one wave stores 4 outputs per lane");
    // (gated: the second half of the lanes that hold results have the second products, with terms of their own)
    const int up_q = GATE && 4 * q >= BNR ? 1 : 0, col = GATE ? n0 + 4 * q - up_q * BNR : n0 + 4 * q;
    const int epi_n = !EPI || r16 >= M || 4 * q >= BN ? 0 : min(4, N - col);
    Epi4 terms;
    if constexpr (GATE) terms = load_epi4(N, r16, col + up_q * N, epi_n, epi.e);
    else if constexpr (BLOCKS) terms = load_epi4(N, r16, n0 + 4 * q, epi_n, epi.e);
    else if constexpr (EPI) terms = load_epi4(N, r16, n0 + 4 * q, epi_n, epi);

    f32x4 acc[NBLK];
#pragma unroll
    for (int b = 0; b < NBLK; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto compute = [&](int stage) {
        const unsigned char* s = lds + stage * STAGE_BYTES;
        f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < KPW; ++t) {
            const int kb = wave * KPW + t;
            const int ch = ((4 * kb + q) ^ r16) * 16;  // A rows 0..15: swizzle term r16
            const u32x4 fa = *(const u32x4*)(s + r16 * ROWB + ch);
#pragma unroll
            for (int b = 0; b < NBLK; ++b) {
                // with BN < 16 the operand's rows r16 and r16 + BN repeat B row r16 % BN;
                // the repeated output columns are never stored
                const int brow = AR + 16 * b + (r16 % BR);
                const int chb = ((4 * kb + q) ^ (brow & 15)) * 16;
                const u32x4 fb = *(const u32x4*)(s + brow * ROWB + chb);
                if constexpr (BLOCKS) {
                    if constexpr (is_blocks<Epi>::wide) {
                        part = Mfma<GEMM_BT_F16>::m16x16x32(widen_e4m3(fb[0], fb[1]), widen_e4m3(fa[0], fa[1]), part);
                        part = Mfma<GEMM_BT_F16>::m16x16x32(widen_e4m3(fb[2], fb[3]), widen_e4m3(fa[2], fa[3]), part);
                    } else {
                        part = skinny_mma<IN>(fb, fa, part);
                    }
                    if (t % 2 == 1) {  // a block is two k-blocks of 64 bytes
                        const float sa = scales[stage][t / 2 * AR + r16];
                        const f32x4 sb = *(const f32x4*)&scales[stage][64 + t / 2 * BN + 4 * q % BN];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = part[e], w = sb[e], c = acc[b][e];
                            acc[b][e] = __builtin_fmaf(p * sa, w, c);
                        }
                        part = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                } else {
                    acc[b] = skinny_mma<IN>(fb, fa, acc[b]);
                }
            }
        }
    };

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(s, s);
    int cs = 0, ls = STAGES - 1;
    for (int kt = 0; kt < nk; ++kt) {
        wait_vmcnt<PEND + (BLOCKS ? 2 * (STAGES - 2) : 0)>();
        // the stage refilled next is the one that the step before this one read, whatever their number: its reads have
        // returned (each is used in its own step, so this waits for nothing, but no order of instructions is relied on)
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        barrier_no_fence();
        issue(ls, kt + STAGES - 1);
        compute(cs);
        cs = cs + 1 == STAGES ? 0 : cs + 1;
        ls = ls + 1 == STAGES ? 0 : ls + 1;
    }
    wait_vmcnt<0>();
    if (tail > 0 && wave == 0)
#pragma unroll
        for (int b = 0; b < NBLK; ++b) acc[b] = skinny_mma<IN>(tb[b], ta, acc[b]);

    if constexpr (EPI) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = acc[0][e];
            v[e] = IN == GEMM_BT_INT8 ? (float)(int)as_u32(x) : x;
        }
        if constexpr (GATE) {
            const int md = epi.e.mode;
            float up[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(v[e] * terms.rs, terms.cs[e], terms.cb[e]);
            if (epi_n > 0 && (md & EPI_PREACT))
                store4(epi.e.preact, epi_type(md, EPI_PREACT_TYPE), (size_t)(2 * r16 + up_q) * N + col, epi_n, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) up[e] = __shfl(v[e], (lane + 4 * BNR) & 63);
            with_act(md >> EPI_ACT, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = act_value<decltype(act)::value>(v[e]) * up[e];
            });
            if (epi_n > 0 && up_q == 0) store4(C, epi_type(md, EPI_OUT_TYPE), (size_t)r16 * N + col, epi_n, v);
        } else if constexpr (BLOCKS) {
            if (epi_n > 0) store_epi4(v, terms, C, N, r16, n0 + 4 * q, epi_n, epi.e);
        } else {
            if (epi_n > 0) store_epi4(v, terms, C, N, r16, n0 + 4 * q, epi_n, epi);
        }
        return;
    }
#pragma unroll
    for (int b = 0; b < NBLK; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    if (wave != 0) return;
    const int m = lane & 15;  // accumulator lane l holds D[4*(l/16) + e][l % 16]: column m of C^T
    if (m >= M) return;
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(C, (u32)min((size_t)M * N * OSZ, (size_t)0x7FFFFFFF));
#pragma unroll
    for (int b = 0; b < NBLK; ++b) {
        f32x4 sum = red[0][b][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += red[w][b][lane];
        const int nl = 16 * b + 4 * q;  // padding rows (nl >= BN) are not stored
        const int n = n0 + nl;
        const u32 o = ((u32)m * (u32)N + (u32)n) * OSZ;
        const float v0 = sum[0], v1 = sum[1], v2 = sum[2], v3 = sum[3];
        if (nl >= BN) continue;
        if (vec_store) {
            if (n < N) {
                if constexpr (OUT == GEMM_BT_F32) {
                    u32x4 w4 = {as_u32(v0), as_u32(v1), as_u32(v2), as_u32(v3)};
                    __builtin_amdgcn_raw_buffer_store_b128(w4, rc, o, 0, 0);
                } else {
                    u32x2 w2 = {pack2<OUT>(v0, v1), pack2<OUT>(v2, v3)};
                    __builtin_amdgcn_raw_buffer_store_b64(w2, rc, o, 0, 0);
                }
            }
        } else {
            const float vv[4] = {v0, v1, v2, v3};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e < N) {
                    if constexpr (OUT == GEMM_BT_F32) {
                        __builtin_amdgcn_raw_buffer_store_b32(as_u32(vv[e]), rc, o + 4u * e, 0, 0);
                    } else {
                        const u32 p = pack2<OUT>(vv[e], 0.0f);
                        __builtin_amdgcn_raw_buffer_store_b16((u16)(p & 0xFFFFu), rc, o + 2u * e, 0, 0);
                    }
                }
            }
        }
    }
}

template <int IN, int OUT, int BN, int KB, int STAGES, int W, int ROT = 0>
__global__ __launch_bounds__(64 * W) void skinny_dma_kernel(const u16* __restrict__ A, const u16* __restrict__ B,
                                                           void* __restrict__ C, int M, int N, int K,
                                                           int vec_store, long long sa, long long sb, long long sc) {
    batch_item(blockIdx.y, A, B, C, sa, sb, sc);  // one grid row per batch item
    skinny_body<IN, OUT, BN, KB, STAGES, W, ROT>(A, B, C, M, N, K, vec_store, SkinnyPlain{});
}

// With an epilogue, in any input type: bound by one read of B (16 x 8192 x 8192
// bf16 with bias and silu 26.1 us, 5.2 TB/s, as without; int8 15.8 us, 4.2).
template <int IN, int BN, int KB, int STAGES, int W>
__global__ __launch_bounds__(64 * W) void skinny_epi_kernel(const u16* __restrict__ A, const u16* __restrict__ B,
                                                           void* __restrict__ C, int M, int N, int K,
                                                           const EpiArgs epi) {
    skinny_body<IN, GEMM_BT_F32, BN, KB, STAGES, W, 0>(A, B, C, M, N, K, 0, epi);  // (OUT is not used)
}

// The gated epilogue.
template <int IN, int BN, int KB, int STAGES, int W>
__global__ __launch_bounds__(64 * W) void skinny_gated_kernel(const u16* __restrict__ A, const u16* __restrict__ B,
                                                             void* __restrict__ C, int M, int N, int K,
                                                             const EpiArgs epi) {
    skinny_body<IN, GEMM_BT_F32, BN, KB, STAGES, W, 0>(A, B, C, M, N, K, 0, SkinnyGated{epi});  // (OUT is not used)
}

// E4M3 with scales per block, B's per 128 rows (TALL) or per row; WIDE: fp32 results.
template <bool TALL, bool WIDE, int BN, int KB, int STAGES>
__global__ __launch_bounds__(64) void skinny_block_kernel(const u16* __restrict__ A, const u16* __restrict__ B, void* __restrict__ C,
                                                         int M, int N, int K, const EpiArgs epi, const BlkArgs blk) {
    skinny_body<GEMM_BT_FP8_E4M3, GEMM_BT_F32, BN, KB, STAGES, 1, 0>(A, B, C, M, N, K, 0, SkinnyBlocks<TALL, WIDE>{epi, blk});
}

}  // namespace gbt
