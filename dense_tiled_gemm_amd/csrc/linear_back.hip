// linear_back.hip -- the backward pass of the product with bias and
// activation: with dz = dy act'(z),
//   dX = dz W        (M x K, summed over N)
//   dW = dz^T X      (N x K, summed over M)
//   db = sum over rows of dz.
// dz is made once by one pass over dy and z that also leaves partial sums of db
// (act_back_kernel).  It is rounded into the inputs' 16-bit type, since the
// matrix instructions take 16-bit operands at the rate counted on here: in
// bf16 the relative error of dX and dW is 0.0024 with it, 0.0017 without (their
// own rounding).  db is summed before that rounding.  Both products then run in
// ONE launch on the transpose-read tiles of trans_kernel.hpp, operands as they
// lie in memory: the tiles of one fill the compute units that the other leaves
// idle, the last block of each column of db is folded by a few more
// workgroups, and a backward pass costs two launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "rows.hpp"
#include "trans_kernel.hpp"

namespace gbt {

// One of the two products, in tiles of BM x BN, each tile's K steps of 64 in
// `pieces` runs of `per` steps.  A single piece is rounded into `out`; of
// several, piece j leaves fp32 sums in `parts` + j * rows * cols.
struct BackProduct {
    const u16* a;
    const u16* b;
    void* out;
    float* parts;
    int rows, cols, depth;  // of the result, and of the sum
    int lda, ldb;
    int tiles_m, tiles_n, pieces, per;
    int blocks;   // workgroups: tiles_m * tiles_n * pieces, padded to whole rounds of the 8 dies
    int shifted;  // rows of `out` are not whole 16-byte chunks (of `parts`: shifted_parts)
    int shifted_parts;

    int steps() const { return blocks ? std::min(per, (depth + 63) / 64) : 0; }  // of its longest run
};
struct BackArgs {
    BackProduct dw, dx;
    int dx_first;   // the product whose runs are longer goes first, so that the shorter ones fill what it leaves
    FoldArgs fold;  // out == nullptr: none
};

template <int IN, bool TA, int BM, int BN, int WN, int S>
__device__ __forceinline__ void back_tile(const BackProduct& p, int pid, unsigned char* lds) {
    const int total = p.tiles_m * p.tiles_n * p.pieces;
    if (pid >= total) return;
    // die by die, the pieces of a tile next to each other
    const int v = (int)xcd_seq(pid, total);
    const int tile = v / p.pieces, j = v - tile * p.pieces;
    int64_t tm, tn;
    band_coord(tile, p.tiles_m, p.tiles_n, 4, &tm, &tn);
    const int k0 = j * p.per * 64;
    const int depth = min(p.depth - k0, p.per * 64);
    const u16* a = TA ? p.a + (size_t)k0 * p.lda : p.a + k0;
    const u16* b = p.b + (size_t)k0 * p.ldb;
    if (p.pieces == 1)
        trans_body<IN, IN, TA, true, BM, BN, 2, WN, S>(a, b, p.out, p.rows, p.cols, depth, p.lda, p.ldb, (int)tm * BM,
                                                       (int)tn * BN, p.shifted, lds);
    else
        trans_body<IN, GEMM_BT_F32, TA, true, BM, BN, 2, WN, S>(a, b, p.parts + (size_t)j * p.rows * p.cols, p.rows, p.cols,
                                                                depth, p.lda, p.ldb, (int)tm * BM, (int)tn * BN,
                                                                p.shifted_parts, lds);
}

// Bound by the tiles' operand reads (see trans_kernel.hpp): 4096^3 bf16, both
// products, 220 us (1250 TFLOP/s); 2048^3 38 us; 1000x512x2048 12 us.
template <int IN, int BM, int BN, int WN, int S>
__global__ __launch_bounds__(128 * WN) void linear_back_kernel(const BackArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S * (BM + BN) * 64 * 2];
    int blk = blockIdx.x;
    const int w0 = a.dx_first ? a.dx.blocks : 0, x0 = a.dx_first ? 0 : a.dw.blocks;
    if (blk >= w0 && blk < w0 + a.dw.blocks) return back_tile<IN, true, BM, BN, WN, S>(a.dw, blk - w0, lds);
    if (blk >= x0 && blk < x0 + a.dx.blocks) return back_tile<IN, false, BM, BN, WN, S>(a.dx, blk - x0, lds);
    blk -= a.dw.blocks + a.dx.blocks;
    fold_columns<128 * WN>(a.fold, blk, (float(*)[17])lds);
}

// out = sum of `pieces` slices of n fp32 sums, in order, rounded once.
struct SliceArgs {
    const float* parts[2];
    void* out[2];
    long long n[2];
    int pieces[2];
    int type;
};
__global__ __launch_bounds__(256) void slices_kernel(const SliceArgs a) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const long long step = (long long)gridDim.x * 256 * 8;
        for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < a.n[s]; i += step) {
            const int n = (int)min(8LL, a.n[s] - i);
            float v[8];
            decode8(load_raw8(a.parts[s], GEMM_BT_F32, (size_t)i, n), GEMM_BT_F32, v);
            for (int j = 1; j < a.pieces[s]; ++j) {
                float w[8];
                decode8(load_raw8(a.parts[s], GEMM_BT_F32, (size_t)(j * a.n[s] + i), n), GEMM_BT_F32, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            }
            store8(a.out[s], a.type, (size_t)i, n, v);
        }
    }
}

// Rows of x and then of w, k elements each, into rows of `pitch` elements (the
// rest zeros): for k % 8 != 0, whose rows are not whole 16-byte chunks.
__global__ __launch_bounds__(256) void pad_rows_kernel(const u16* x, const u16* w, u16* out, long long m, long long n, int k,
                                                       int pitch) {
    const int groups = pitch / 8;
    const long long total = (m + n) * groups;
    for (long long q = (long long)blockIdx.x * 256 + threadIdx.x; q < total; q += (long long)gridDim.x * 256) {
        const long long row = q / groups;
        const int j = (int)(q - row * groups) * 8;
        const u16* src = row < m ? x + row * k : w + (row - m) * k;
        const Raw8 r = load_raw8(src, GEMM_BT_BF16, (size_t)j, min(8, k - j));
        *(u32x4*)(out + row * pitch + j) = r.a;
    }
}

__global__ void fill_zero16_kernel(u16* p, long long n) {
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) p[i] = 0;
}

// ---- host ------------------------------------------------------------------------

static int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
static int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Everything a backward pass of these sizes needs: its tiles, and where its
// parts lie in the workspace (byte offsets; the sizes do not depend on which
// gradients are asked for).
struct BackPlan {
    int bm, bn;
    bool make_dz, pad;
    int64_t ldz, ldk;  // row pitches of dz, and of X and W (elements)
    int pieces_w, per_w, pieces_x, per_x;
    int64_t sums_parts;
    int64_t off_dz, off_sums, off_parts_w, off_parts_x, off_pad, bytes;
};

// Runs of K steps for a product of `tiles` tiles of `steps` steps each, where
// all tiles of both products would take `fair` steps on every CU: a tile much
// longer than that is cut into runs of about that length, each of which leaves
// fp32 sums; the cut costs a launch that adds them, so only a gain of `least`
// steps is taken (128 x 128 tiles, us, at 24, 12 and 6: 131x1536x192 21.1, 15.9,
// 15.9; 2048x1024x1024 30.3, 28.4, 28.1; 1024x1024x1024 20.4, 20.3, 25.9;
// 1000x512x2048 19.3, 19.2, 20.9).  `most` steps is what a run may hold (2 GiB of an operand).
static void cut(int64_t steps, int64_t fair, int64_t least, int64_t most, int* pieces, int* per) {
    int64_t run = steps;
    if (steps - fair >= least) run = std::max<int64_t>(fair, 8);
    run = std::max<int64_t>(1, std::min(run, most));
    *pieces = (int)std::max<int64_t>(1, (steps + run - 1) / run);
    *per = (int)((steps + *pieces - 1) / std::max(1, *pieces));
    *per = std::max(1, *per);
    *pieces = (int)std::max<int64_t>(1, (steps + *per - 1) / *per);
}

// Steps until the last of `cu` compute units is done, when t1 runs of s1 steps
// and then t2 of s2 <= s1 go to whichever is free first.
static int64_t makespan(int64_t t1, int64_t s1, int64_t t2, int64_t s2, int64_t cu) {
    const int64_t rounds = t1 / cu, rest = t1 % cu;
    int64_t T = std::max((rest ? rounds + 1 : rounds) * s1, (t1 * s1 + t2 * s2 + cu - 1) / cu);
    if (t2 == 0) return T;
    auto fits = [&](int64_t at) {  // runs of s2 done by then
        const int64_t late = std::max<int64_t>(0, at - (rounds + 1) * s1) / s2, early = std::max<int64_t>(0, at - rounds * s1) / s2;
        return rest * late + (cu - rest) * early >= t2;
    };
    while (!fits(T)) ++T;
    return T;
}

// The tile shapes, and what one of their K steps takes on a compute unit that
// is kept busy (us; 128 x 128: of two workgroups on a unit, per workgroup).
struct BackTile {
    int bm, bn;
    double step, ragged;  // ragged: where rows of dz, X or W do not start on 128-byte lines (narrow tiles then fetch
                          // more lines for the same columns)
};
constexpr BackTile kBackTiles[] = {{128, 128, 0.60, 0.69}, {128, 256, 1.05, 1.15}, {256, 256, 1.5, 1.57}};

// The plan with the shortest estimate: the longest unit's steps (each run three
// more, for its start and its stores), and the slices' way to memory and back.
// Whole calls on 128 x 128, 128 x 256 and 256 x 256 tiles (M x N x K, us, bf16):
// 2048^3 49.1, 46.4, 61.6; 4096x4096x1024 99.4, 91.4, 107.0; 528x1728x7040 50.8,
// 55.8, 62.0; 8192x1024x4096 167.7, 159.8, 152.9; 4096^3 302.6, 284.1, 236.8.
// The longer runs first, instead of dW always: 2048x4096x4096 147.8 -> 129.5,
// 1024x4096x4096 92.4 -> 79.8, 528x1728x7040 50.8 -> 45.8.
static BackPlan back_plan(int64_t M, int64_t N, int64_t K, bool act, int num_cu) {
    BackPlan p = {};
    p.make_dz = act || N % 8 != 0;
    p.pad = K % 8 != 0;
    p.ldz = up8(N);
    p.ldk = up8(K);
    const int64_t steps_w = (M + 63) / 64, steps_x = (N + 63) / 64;
    // steps of 64 rows that one run may take of its K-outer operands: 2 GiB of
    // each (dW: dz and X; dX: W alone, dz is read row by row; with dz's limit on
    // dX too, ms: 4096x128256x4096 8.5, without 7.2; 8192x128256x4096 18.3, 14.4)
    auto steps_of = [](int64_t ld) { return std::max<int64_t>(1, 0x7FFFFFFFLL / (128 * std::max<int64_t>(1, ld))); };
    const int64_t most_w = steps_of(std::max(p.ldz, p.ldk)), most_x = steps_of(p.ldk);
    double best = 0.0;
    for (const BackTile& t : kBackTiles) {
        auto tiles = [&](int64_t r, int64_t c) { return ((r + t.bm - 1) / t.bm) * ((c + t.bn - 1) / t.bn); };
        const int64_t tiles_w = tiles(N, K), tiles_x = tiles(M, K);
        const int64_t fair = (tiles_w * steps_w + tiles_x * steps_x + num_cu - 1) / num_cu;
        int pieces_w, per_w, pieces_x, per_x;
        cut(steps_w, fair, 12, most_w, &pieces_w, &per_w);
        cut(steps_x, fair, 12, most_x, &pieces_x, &per_x);
        const int64_t runs_w = tiles_w * pieces_w, runs_x = tiles_x * pieces_x;
        const int64_t span = per_w >= per_x ? makespan(runs_w, per_w + 3, runs_x, per_x + 3, num_cu)
                                            : makespan(runs_x, per_x + 3, runs_w, per_w + 3, num_cu);
        const double slices = (pieces_w > 1 ? (double)pieces_w * N * K : 0.0) + (pieces_x > 1 ? (double)pieces_x * M * K : 0.0);
        const bool lines = p.ldz % 64 == 0 && p.ldk % 64 == 0;
        const double time = (lines ? t.step : t.ragged) * span + slices * 8.0 / 4e6 + (slices > 0.0 ? 3.0 : 0.0);
        if (best > 0.0 && time >= best) continue;
        best = time;
        p.bm = t.bm;
        p.bn = t.bn;
        p.pieces_w = pieces_w;
        p.per_w = per_w;
        p.pieces_x = pieces_x;
        p.per_x = per_x;
    }
    p.sums_parts = M > 0 && N > 0 ? act_back_parts(M, N, num_cu) : 0;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up256(bytes);
        return here;
    };
    p.off_dz = take(p.make_dz ? M * p.ldz * 2 : 0);
    p.off_sums = take(p.sums_parts * N * 4);
    p.off_parts_w = take(p.pieces_w > 1 ? p.pieces_w * N * K * 4 : 0);
    p.off_parts_x = take(p.pieces_x > 1 ? p.pieces_x * M * K * 4 : 0);
    p.off_pad = take(p.pad ? (M + N) * p.ldk * 2 : 0);
    p.bytes = at;
    return p;
}

static bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    // 32-bit buffer offsets inside one panel of 256 rows, and of 64 steps of K
    const int64_t most = 0x7FFFFFFFLL / 1024;
    if (M > 0x7FFFFFFF - 256 || N > most || K > most) return false;
    // and a grid of at most 2^32 threads, 512 or fewer to a tile: 2^21 tiles of 128 x 128 of each product
    const int64_t tiles = ((M + 127) / 128) * ((K + 127) / 128), tiles_w = ((N + 127) / 128) * ((K + 127) / 128);
    return tiles <= 1 << 21 && tiles_w <= 1 << 21;
}

static int fill_zero(void* out, int64_t n, void* stream) {
    if (n == 0) return GEMM_BT_OK;
    u16* p = (u16*)out;
    long long nn = n;
    void* args[] = {&p, &nn};
    return launch((const void*)&fill_zero16_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), 256, args, stream);
}

static int linear_backward(const void* dy, const void* x, const void* w, const void* preact, void* dx, void* dw, void* dbias,
                           int64_t M, int64_t N, int64_t K, int act, int type, int preact_type, char* ws, const BackPlan& p,
                           int num_cu, void* stream) {
    int st;
    // dz, and the partial sums of its columns
    const void* dz = dy;
    if (p.make_dz || dbias) {
        if (p.make_dz) dz = ws + p.off_dz;
        st = launch_act_back({dy, act != GEMM_BT_ACT_NONE ? preact : nullptr, p.make_dz && (dx || dw) ? (void*)dz : nullptr,
                              dbias ? (float*)(ws + p.off_sums) : nullptr, M, (int)N, (int)p.ldz, 0, type, preact_type, act},
                             num_cu, stream);
        if (st != GEMM_BT_OK) return st;
    }
    if (p.pad && (dx || dw)) {
        // X for dW, W for dX: only what is read
        const u16 *sx = (const u16*)x, *sw = (const u16*)w;
        long long m = dw ? M : 0, n = dx ? N : 0;
        u16 *at = (u16*)(ws + p.off_pad), *out = dw ? at : at + M * p.ldk;
        int k = (int)K, pitch = (int)p.ldk;
        void* args[] = {&sx, &sw, &out, &m, &n, &k, &pitch};
        st = launch((const void*)&pad_rows_kernel, dim3((unsigned)std::min<int64_t>(((m + n) * p.ldk / 8 + 255) / 256, 1 << 16)),
                    256, args, stream);
        if (st != GEMM_BT_OK) return st;
        x = at;
        w = at + M * p.ldk;
    }
    auto product = [&](const void* a, const void* b, void* out, float* parts, int64_t rows, int64_t cols, int64_t depth,
                       int64_t lda, int64_t ldb, int pieces, int per) {
        BackProduct q = {};
        if (!out || rows == 0 || cols == 0) return q;
        q.a = (const u16*)a;
        q.b = (const u16*)b;
        q.out = out;
        q.parts = parts;
        q.rows = (int)rows;
        q.cols = (int)cols;
        q.depth = (int)depth;
        q.lda = (int)lda;
        q.ldb = (int)ldb;
        q.tiles_m = (int)((rows + p.bm - 1) / p.bm);
        q.tiles_n = (int)((cols + p.bn - 1) / p.bn);
        q.pieces = pieces;
        q.per = per;
        q.blocks = (q.tiles_m * q.tiles_n * pieces + 7) / 8 * 8;
        q.shifted = cols % 8 != 0 || (uintptr_t)out % 16 != 0;
        q.shifted_parts = cols % 4 != 0;
        return q;
    };
    BackArgs a = {};
    a.dw = product(dz, x, dw, (float*)(ws + p.off_parts_w), N, K, M, p.ldz, p.ldk, p.pieces_w, p.per_w);
    a.dx = product(dz, w, dx, (float*)(ws + p.off_parts_x), M, K, N, p.ldz, p.ldk, p.pieces_x, p.per_x);
    a.dx_first = a.dx.steps() > a.dw.steps();
    unsigned grid = (unsigned)(a.dw.blocks + a.dx.blocks);
    if (dbias) {
        a.fold = {(const float*)(ws + p.off_sums), dbias, N, (int)p.sums_parts, type};
        grid += fold_blocks(N);
    }
    if (grid == 0) return GEMM_BT_OK;
    // 128 x 128 tiles that leave every CU at most one workgroup, and 16 or more
    // steps: a ring of four stages in place of two workgroups' worth of two (us:
    // 1024x1024x1024 22.6 vs 20.4, 2048x1024x1024 35.0 vs 30.3; with 8 steps
    // the longer start loses, 4096x512x512 25.1 vs 28.5)
    const bool deep = p.bn == 128 && a.dw.blocks + a.dx.blocks <= num_cu && std::max(a.dw.steps(), a.dx.steps()) >= 16;
    auto pick = [&](auto in) -> const void* {
        constexpr int IN = decltype(in)::value;
        if (p.bm == 256) return (const void*)&linear_back_kernel<IN, 256, 256, 4, 2>;
        if (p.bn == 256) return (const void*)&linear_back_kernel<IN, 128, 256, 4, 3>;
        return deep ? (const void*)&linear_back_kernel<IN, 128, 128, 2, 4> : (const void*)&linear_back_kernel<IN, 128, 128, 2, 2>;
    };
    const void* fn = type == GEMM_BT_BF16 ? pick(std::integral_constant<int, GEMM_BT_BF16>{})
                                          : pick(std::integral_constant<int, GEMM_BT_F16>{});
    void* args[] = {&a};
    st = launch(fn, dim3(grid), p.bn == 256 ? 512 : 256, args, stream);
    if (st != GEMM_BT_OK) return st;
    SliceArgs s = {};
    s.type = type;
    int64_t most = 0;
    const BackProduct* q[2] = {&a.dw, &a.dx};
    for (int i = 0; i < 2; ++i)
        if (q[i]->pieces > 1) {
            s.parts[i] = q[i]->parts;
            s.out[i] = q[i]->out;
            s.n[i] = (long long)q[i]->rows * q[i]->cols;
            s.pieces[i] = q[i]->pieces;
            most = std::max<int64_t>(most, s.n[i]);
        }
    if (most == 0) return GEMM_BT_OK;
    void* sargs[] = {&s};
    return launch((const void*)&slices_kernel, dim3((unsigned)std::min<int64_t>((most + 2047) / 2048, 8 * num_cu)), 256, sargs,
                  stream);
}

}  // namespace gbt

using namespace gbt;

extern "C" {

int gemm_bt_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int activation, size_t* bytes) {
    if (!bytes) return GEMM_BT_ERR_INVALID_VALUE;
    *bytes = 0;
    if (M < 0 || N < 0 || K < 0 || activation < GEMM_BT_ACT_NONE || activation > GEMM_BT_ACT_SILU)
        return GEMM_BT_ERR_INVALID_VALUE;
    if (!sizes_ok(M, N, K)) return GEMM_BT_ERR_UNSUPPORTED;
    if (M > 0 && N > 0) *bytes = (size_t)back_plan(M, N, K, activation != GEMM_BT_ACT_NONE, plan_cus()).bytes;
    return GEMM_BT_OK;
}

int gemm_bt_linear_backward(const void* dy, const void* x, const void* w, const void* preact, void* dx, void* dw, void* dbias,
                            int64_t M, int64_t N, int64_t K, int activation, int dtype, int preact_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 0 || activation < GEMM_BT_ACT_NONE || activation > GEMM_BT_ACT_SILU)
        return GEMM_BT_ERR_INVALID_VALUE;
    const bool act = activation != GEMM_BT_ACT_NONE;
    if ((dtype != GEMM_BT_F16 && dtype != GEMM_BT_BF16) || (act && !float_type(preact_dtype))) return GEMM_BT_ERR_UNSUPPORTED;
    if (!sizes_ok(M, N, K)) return GEMM_BT_ERR_UNSUPPORTED;
    if (K == 0) dx = dw = nullptr;  // nothing to write
    if (M == 0) dx = nullptr;
    if (N == 0) dw = dbias = nullptr;
    if (!dx && !dw && !dbias) return GEMM_BT_OK;
    if (!aligned(dx, dtype) || !aligned(dw, dtype) || !aligned(dbias, dtype)) return GEMM_BT_ERR_INVALID_VALUE;
    const bool empty = M == 0 || N == 0;  // the sums have no terms
    if (!empty) {
        if (!dy || (dx && !w) || (dw && !x) || (act && !preact)) return GEMM_BT_ERR_INVALID_VALUE;
        if (!aligned(dy, dtype) || (act && !aligned(preact, preact_dtype)) || !aligned(x, dtype) || !aligned(w, dtype))
            return GEMM_BT_ERR_INVALID_VALUE;
    }
    int num_cu = 0;
    int st = check_device(&num_cu);
    if (st != GEMM_BT_OK) return st;
    if (empty) {
        if (dx) st = fill_zero(dx, M * K, stream);
        if (st == GEMM_BT_OK && dw) st = fill_zero(dw, N * K, stream);
        if (st == GEMM_BT_OK && dbias) st = fill_zero(dbias, N, stream);
        return st;
    }
    const BackPlan p = back_plan(M, N, K, act, num_cu);
    if (p.bytes > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < (size_t)p.bytes))
        return GEMM_BT_ERR_INVALID_VALUE;
    // the products read whole 16-byte chunks of their operands where they lie
    auto chunks = [](const void* q) { return (uintptr_t)q % 16 == 0; };
    if ((dx || dw) && ((!p.make_dz && !chunks(dy)) || (!p.pad && ((dw && !chunks(x)) || (dx && !chunks(w))))))
        return GEMM_BT_ERR_UNSUPPORTED;
    return linear_backward(dy, x, w, preact, dx, dw, dbias, M, N, K, activation, dtype, preact_dtype,
                           (char*)workspace, p, num_cu, stream);
}

}  // extern "C"
