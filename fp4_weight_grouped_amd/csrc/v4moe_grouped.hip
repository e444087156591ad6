// v4moe_grouped.hip -- products grouped by expert with ragged sizes, bf16 weights.
//
//   rows m of expert e: offsets[e] <= m < offsets[e + 1]
//   forward           y[m]  = W[e] x[m]                      W [E][N][K]
//   data gradient     dx[m] = W[e]^T dy[m]
//   weight gradient   dW[e] = sum over e's rows of dy[m] x[m]^T
//
// Nothing but the offsets says how many tiles an expert has, and they stay on the
// device: the grid is the most that any split of the rows needs, each block
// derives its tile from the offsets, and blocks without one end.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"
#include "v4moe_mm.h"

#include <hip/hip_runtime.h>

namespace v4moe {

namespace {

struct GroupedArgs {
    int M, N, K, E;                  // rows, and a group's product: C columns N, contraction K (data gradients: the weight's K and N)
    const int32_t* offsets;
    const uint16_t* a; int64_t lda;  // rows x or dy
    const uint16_t* b; int64_t ldb;  // weights, `group` elements apart; weight gradients: rows x
    int64_t group;
    MmOut c;
};

// Rows [first, first + count) of expert e, within [0, M] whatever the offsets hold.
__device__ __forceinline__ int rows_of(const int32_t* offsets, int e, int M, int& first)
{
    first = min(max(offsets[e], 0), M);
    return max(min(max(offsets[e + 1], 0), M) - first, 0);     // (both ends clamped first: their difference cannot overflow)
}

// Finds the expert of a block's tile, per row tile tn column tiles: experts in order, an
// expert's tiles column by column in bands of eight row tiles.  `found` is LDS.
struct Found { int e, first, count, tile, total, wave[16]; };
template <int BM, int THREADS>
__device__ __forceinline__ bool find_tile(const GroupedArgs& g, int tn, int block, int blocks, Found* found, int& e, int& first,
                                          int& count, int& im, int& in)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int each = (g.E + THREADS - 1) / THREADS, e0 = t * each, e1 = min(e0 + each, g.E);
    int mine = 0;
    for (int i = e0; i < e1; i++) {
        int f;
        mine += (rows_of(g.offsets, i, g.M, f) + BM - 1) / BM;
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 63) found->wave[wave] = scan;
    __syncthreads();
    int before = scan - mine, total = 0;
    for (int w = 0; w < THREADS / 64; w++) {
        if (w < wave) before += found->wave[w];
        total += found->wave[w];
    }
    if ((int64_t)total * tn > blocks) return false;        // (offsets that do not ascend: nothing is done)
    const int turn = mm_turn(block, total * tn);
    if (turn < 0) return false;
    if (turn >= before * tn && turn < (before + mine) * tn) {
        for (int i = e0; i < e1; i++) {
            int f;
            const int n = rows_of(g.offsets, i, g.M, f), tiles = (n + BM - 1) / BM;
            if (turn < (before + tiles) * tn) {
                found->e = i;
                found->first = f;
                found->count = n;
                found->tile = turn - before * tn;
                break;
            }
            before += tiles;
        }
    }
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(found->e);
    first = __builtin_amdgcn_readfirstlane(found->first);
    count = __builtin_amdgcn_readfirstlane(found->count);
    mm_band(__builtin_amdgcn_readfirstlane(found->tile), (count + BM - 1) / BM, tn, im, in);
    __syncthreads();
    return true;
}

// Forward and data gradient: row tiles of each expert by column tiles of C.  Few rows: the weights' bytes (1024 rows of
// 256 experts, 2048 x 4096: 677 us, 6.2 TB/s; 8 rows of 8 experts 25, 5.3).  Many: the matrix units (65536 uneven rows
// of those experts 1305 us, 0.84 PFLOP/s, with 4.3 GB of weights on the way; 2048 rows each of 32 experts 886, 1.24;
// data gradient of 32768 rows, 4096 x 2048, 32 experts 518; the first launches after a pause, as under a profiler, take up
// to a tenth longer).
template <class L>
__device__ __forceinline__ void rows_tile(const GroupedArgs& g, int tn, int block, int blocks, uint8_t* smem)
{
    int e, first, count, im, in;
    if (!find_tile<L::BM, L::THREADS>(g, tn, block, blocks, reinterpret_cast<Found*>(smem), e, first, count, im, in)) return;
    const MmOperand a{g.a + first * g.lda, g.lda, count}, b{g.b + e * g.group, g.ldb, L::BCOL ? (g.N + 7) / 8 * 8 : g.N};
    v4f acc[L::MI][L::NI];
    mm_tile<L>(a, b, im * L::BM, in * L::BN, g.K, smem, acc);
    MmOut c = g.c;
    c.M = count;
    c.c = static_cast<uint8_t*>(c.c) + first * c.ldc * (c.bf16 ? 2 : 4);
    mm_store_tile<L>(acc, smem, c, im * L::BM, in * L::BN);
}
template <class L>
__global__ __launch_bounds__(L::THREADS) void k_grouped_rows(GroupedArgs g, int tn)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    rows_tile<L>(g, tn, blockIdx.x, gridDim.x, smem);
}

// Weight gradient: the tiles of each expert's dW, its rows the contraction (32768 rows, 4096 x 2048, 32 experts 609 us,
// under a profiler up to 670: 16 chunks a tile, so that its begin and its end, with 0.5 GB of dW to store, weigh more).
template <class L>
__device__ __forceinline__ void weights_tile(const GroupedArgs& g, int tm, int tn, int block, uint8_t* smem)
{
    const int turn = mm_turn(block, g.E * tm * tn), e = turn / (tm * tn), tile = turn % (tm * tn);
    int first;
    const int count = rows_of(g.offsets, e, g.M, first);
    MmOut c = g.c;
    if (count == 0 && c.accumulate) return;          // (adding a sum of nothing would turn -0 into 0)
    int im, in;
    mm_band(tile, tm, tn, im, in);
    const int m0 = im * L::BM, n0 = in * L::BN;
    const MmOperand a{g.a + first * g.lda, g.lda, (c.M + 7) / 8 * 8}, b{g.b + first * g.ldb, g.ldb, (g.N + 7) / 8 * 8};
    v4f acc[L::MI][L::NI];
    mm_tile<L>(a, b, m0, n0, count, smem, acc);
    c.c = static_cast<uint8_t*>(c.c) + (int64_t)e * c.M * c.ldc * (c.bf16 ? 2 : 4);
    mm_store_tile<L>(acc, smem, c, m0, n0);
}
template <class L>
__global__ __launch_bounds__(L::THREADS) void k_grouped_weights(GroupedArgs g, int tm, int tn)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    weights_tile<L>(g, tm, tn, blockIdx.x, smem);
}

// Both gradients in a launch, the data gradient's blocks first.
template <class R, class W>
__global__ __launch_bounds__(R::THREADS) void k_grouped_both(GroupedArgs r, int rtn, int rblocks, GroupedArgs w, int wtm, int wtn)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((int)blockIdx.x < rblocks) rows_tile<R>(r, rtn, blockIdx.x, rblocks, smem);
    else weights_tile<W>(w, wtm, wtn, (int)blockIdx.x - rblocks, smem);
}

// Rows of 2-byte elements, src [R][C] -> dst [R][C8] (C8 = C rounded up to 8), zeros past C: what the
// copies of mm_tile need of operands whose rows do not begin or end at 16 bytes.
// Up to three matrices in a launch, their blocks one after the other (a launch each: 6 us more apiece).  At the copy's
// rate where they are large (50021 x 1001 33 us), latency where not (three of some thousand rows 12).
struct PadJobs {
    PadRows job[3];
    int blocks[3];
};
__global__ __launch_bounds__(256) void k_pad_rows(PadJobs p)
{
    int block = blockIdx.x, j = 0;
    while (j < 2 && block >= p.blocks[j]) block -= p.blocks[j++];
    const PadRows& g = p.job[j];
    const int C8 = (g.C + 7) / 8 * 8, segs = C8 / 8;
    for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < g.R * segs; i += (int64_t)p.blocks[j] * 256) {
        const int64_t r = i / segs;
        const int c = (int)(i - r * segs) * 8;
        *reinterpret_cast<v4u32*>(g.dst + r * C8 + c) = load8(g.src + r * g.ld, c, g.C);
    }
}

// the most row tiles: every expert's last one may hold a single row
int64_t most_row_tiles(const GroupedArgs& g, int64_t bm) { return g.M / bm + (g.M < g.E ? g.M : g.E); }
template <class L>
hipError_t launch_rows(const GroupedArgs& g, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_grouped_rows<L>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int64_t tn = over(g.N, L::BN), tm = most_row_tiles(g, L::BM);
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(L::THREADS), L::BYTES, s, g, (int)tn);
    return hipGetLastError();
}
template <class L>
hipError_t launch_weights(const GroupedArgs& g, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_grouped_weights<L>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int64_t tn = over(g.N, L::BN), tm = over(g.c.M, L::BM);
    if (g.E * tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(g.E * tm * tn)), dim3(L::THREADS), L::BYTES, s, g, (int)tm, (int)tn);
    return hipGetLastError();
}
template <class R, class W>
hipError_t launch_both(const GroupedArgs& r, const GroupedArgs& w, hipStream_t s)
{
    static_assert(R::THREADS == W::THREADS, "one launch");
    static LdsAllowed allowed;
    const auto kernel = k_grouped_both<R, W>;
    constexpr int BYTES = R::BYTES > W::BYTES ? R::BYTES : W::BYTES;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), BYTES, allowed); e != hipSuccess) return e;
    const int64_t rtn = over(r.N, R::BN), rblocks = most_row_tiles(r, R::BM) * rtn;
    const int64_t wtn = over(w.N, W::BN), wtm = over(w.c.M, W::BM), all = rblocks + w.E * wtm * wtn;
    if (all > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)all), dim3(R::THREADS), BYTES, s, r, (int)rtn, (int)rblocks, w, (int)wtm, (int)wtn);
    return hipGetLastError();
}

template <int V, bool BCOL>
struct RowTile;
template <bool BCOL> struct RowTile<0, BCOL> { using L = MmTile<1, 4, 1, 1, 4, false, BCOL>; };
template <bool BCOL> struct RowTile<1, BCOL> { using L = MmTile<2, 2, 1, 2, 4, false, BCOL>; };
template <bool BCOL> struct RowTile<2, BCOL> { using L = MmTile<2, 2, 2, 2, 3, false, BCOL>; };
template <bool BCOL> struct RowTile<3, BCOL> { using L = MmTile<2, 2, 4, 4, 2, false, BCOL, true>; };
template <bool BCOL> struct RowTile<4, BCOL> { using L = MmTile<2, 4, 8, 4, 2, false, BCOL, true>; };
using Weights64 = MmTile<2, 2, 2, 2, 3, true, true>;
using Weights128 = MmTile<2, 2, 4, 4, 2, true, true>;
using Weights256 = MmTile<2, 4, 8, 4, 2, true, true>;

// Row tiles are estimated: the offsets are the device's.  Every expert's last one is half empty on average, and an
// expert with rows has one at least.
int64_t row_tiles(const GroupedArgs& g, int64_t bm, int64_t bn)
{
    const int64_t groups = g.M < g.E ? g.M : g.E, tm = g.M / bm + (groups + 1) / 2;
    return (tm > groups ? tm : groups) * over(g.N, bn);
}
int64_t weight_tiles(const GroupedArgs& g, int64_t bm, int64_t bn) { return g.E * over(g.c.M, bm) * over(g.N, bn); }
int row_variant(const GroupedArgs& g)
{
    return mm_choose(0, g.K, [&](int64_t bm, int64_t bn) { return row_tiles(g, bm, bn); });
}
int weight_variant(const GroupedArgs& g)
{
    return mm_choose(2, g.M / g.E, [&](int64_t bm, int64_t bn) { return weight_tiles(g, bm, bn); });
}
template <bool BCOL>
hipError_t run_rows(const GroupedArgs& g, hipStream_t s)
{
    switch (row_variant(g)) {
    case 0: return launch_rows<typename RowTile<0, BCOL>::L>(g, s);
    case 1: return launch_rows<typename RowTile<1, BCOL>::L>(g, s);
    case 2: return launch_rows<typename RowTile<2, BCOL>::L>(g, s);
    case 3: return launch_rows<typename RowTile<3, BCOL>::L>(g, s);
    default: return launch_rows<typename RowTile<4, BCOL>::L>(g, s);
    }
}
hipError_t run_weights(const GroupedArgs& g, hipStream_t s)
{
    switch (weight_variant(g)) {
    case 2: return launch_weights<Weights64>(g, s);
    case 3: return launch_weights<Weights128>(g, s);
    default: return launch_weights<Weights256>(g, s);
    }
}
// Both gradients.  Where neither fills the GPU for long they go out in one launch, the end of the one beside the begin of
// the other, with 128x128 tiles both (3001 rows of 12 experts, 1001 x 499: 30 us with the copies of its odd operands, 36
// in two launches with the tiles that are best alone, 33 with those in one).
bool one_launch(const GroupedArgs& r, const GroupedArgs& w)
{
    const int rv = row_variant(r), wv = weight_variant(w);
    return (rv == 2 || rv == 3) && wv < 4 && row_tiles(r, 128, 128) <= 1024 && weight_tiles(w, 128, 128) <= 1024;
}
hipError_t run_both(const GroupedArgs& r, const GroupedArgs& w, hipStream_t s)
{
    if (one_launch(r, w))
        return launch_both<RowTile<3, true>::L, Weights128>(r, w, s);
    if (const hipError_t e = run_rows<true>(r, s); e != hipSuccess) return e;
    return run_weights(w, s);
}

struct GroupedLayout {
    size_t x, dy, w, total;
    bool pad_x, pad_dy, pad_w;
};
// Room for padded copies of the operands that cannot be read in place.
GroupedLayout grouped_layout(int64_t M, int64_t E, int64_t N, int64_t K, const void* x, int64_t ldx, const void* dy,
                             int64_t lddy, const void* w, bool backward)
{
    GroupedLayout L{};
    L.pad_x = !in_place(x, K, ldx);
    L.pad_dy = backward && !in_place(dy, N, lddy);
    L.pad_w = !in_place(w, K, K);
    size_t o = 0;
    auto take = [&](int64_t rows, int64_t cols, bool need) {
        const size_t at = o;
        if (need) o += up256((size_t)(rows * up8(cols) * 2));
        return at;
    };
    L.x = take(M, K, L.pad_x);
    L.dy = take(M, N, L.pad_dy);
    L.w = take(E * N, K, L.pad_w);
    L.total = o;
    return L;
}

int check_grouped(int32_t M, int32_t E, int32_t N, int32_t K)
{
    return side_ok(M) && side_ok(N) && side_ok(K) && N >= 1 && K >= 1 && E >= 1 && E <= 1024 ? V4MOE_OK : V4MOE_EDIMS;
}
struct GroupedCall {
    const uint16_t *x, *dy, *w;
    int64_t ldx, lddy, ldw;
};
// The operands as the products read them: in place, or copied into the workspace.
int grouped_operands(GroupedCall& o, int32_t M, int32_t E, int32_t N, int32_t K, bool backward, bool need_x, bool need_w,
                     void* workspace, size_t ws_bytes, hipStream_t s)
{
    const GroupedLayout L = grouped_layout(M, E, N, K, o.x, o.ldx, o.dy, o.lddy, o.w, backward);
    if (L.total > 0 && !workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    if (ws_bytes < L.total) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PadRows jobs[3];
    int n = 0;
    auto pad = [&](const uint16_t*& p, int64_t& ld, int64_t rows, int cols, size_t at) {
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + at);
        jobs[n++] = PadRows{rows, cols, p, ld, to};
        p = to;
        ld = up8(cols);
    };
    if (L.pad_x && need_x) pad(o.x, o.ldx, M, K, L.x);
    if (L.pad_dy) pad(o.dy, o.lddy, M, N, L.dy);
    if (L.pad_w && need_w) pad(o.w, o.ldw, (int64_t)E * N, K, L.w);
    if (launch_pad_rows(jobs, n, s) != hipSuccess) return V4MOE_ELAUNCH;
    return V4MOE_OK;
}

}  // namespace

hipError_t launch_pad_rows(const PadRows* jobs, int n, hipStream_t s)
{
    PadJobs p{};
    int all = 0;
    for (int j = 0; j < n; j++) {
        p.job[j] = jobs[j];
        const int64_t blocks = over(jobs[j].R * (up8(jobs[j].C) / 8), 256);
        p.blocks[j] = (int)(blocks < 16384 ? blocks : 16384);
        all += p.blocks[j];
    }
    if (all == 0) return hipSuccess;
    hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)all), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) size_t moe_grouped_workspace_bytes(int32_t M, int32_t E, int32_t N, int32_t K,
                                                                          const uint16_t* x, int64_t ldx,
                                                                          const uint16_t* dy, int64_t lddy,
                                                                          const uint16_t* w, int32_t backward)
{
    if (check_grouped(M, E, N, K)) return 0;
    return grouped_layout(M, E, N, K, x, ldx, dy, lddy, w, backward != 0).total;
}

__attribute__((visibility("default"))) int32_t moe_grouped_tile(int32_t M, int32_t E, int32_t N, int32_t K, int32_t what,
                                                                int32_t both)
{
    if (check_grouped(M, E, N, K) || what < V4MOE_PRODUCT_FORWARD || what > V4MOE_PRODUCT_DW) return 0;
    // the sizes as the calls below give them to the launches
    GroupedArgs y{}, dx{}, dw{};
    y.M = M, y.N = N, y.K = K, y.E = E;
    dx.M = M, dx.N = K, dx.K = N, dx.E = E;
    dw.M = M, dw.N = K, dw.E = E, dw.c.M = N;
    if (what == V4MOE_PRODUCT_FORWARD) return tile_code(kMmVariants[row_variant(y)]);
    if (both && one_launch(dx, dw)) return 128 << 16 | 128 | V4MOE_TILE_SHARED;
    return tile_code(kMmVariants[what == V4MOE_PRODUCT_DX ? row_variant(dx) : weight_variant(dw)]);
}

__attribute__((visibility("default"))) int moe_grouped_linear(int32_t M, int32_t E, int32_t N, int32_t K,
                                                              const uint16_t* x, int64_t ldx, const uint16_t* w,
                                                              const int32_t* offsets, void* y, int32_t y_type,
                                                              int64_t ldy, void* workspace, size_t ws_bytes,
                                                              void* stream)
{
    if (const int rc = check_grouped(M, E, N, K)) return rc;
    if (const int rc = check_rows(x, M, K, ldx)) return rc;
    if (const int rc = check_out(y, y_type, M, N, ldy)) return rc;
    if (M == 0) return V4MOE_OK;
    if (!w || !offsets) return V4MOE_ENULL;
    if (!aligned_to(w, 2) || !aligned_to(offsets, 4)) return V4MOE_EALIGN;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    GroupedCall o{x, nullptr, w, ldx, 0, K};
    if (const int rc = grouped_operands(o, M, E, N, K, false, true, true, workspace, ws_bytes, s)) return rc;
    const GroupedArgs g{M, N, K, E, offsets, o.x, o.ldx, o.w, o.ldw, (int64_t)N * o.ldw,
                        MmOut{y, ldy, 0, N, y_type == V4MOE_TYPE_BF16, 0}};
    return run_rows<false>(g, s) == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_grouped_linear_backward(
    int32_t M, int32_t E, int32_t N, int32_t K, const uint16_t* x, int64_t ldx, const uint16_t* dy, int64_t lddy,
    const uint16_t* w, const int32_t* offsets, void* dx, int32_t dx_type, int64_t lddx, void* dw, int32_t dw_type,
    int32_t accumulate, void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_grouped(M, E, N, K)) return rc;
    if (!dx && !dw) return V4MOE_ENULL;
    if (dw)
        if (const int rc = check_rows(x, M, K, ldx)) return rc;
    if (const int rc = check_rows(dy, M, N, lddy)) return rc;
    if (dx)
        if (const int rc = check_out(dx, dx_type, M, K, lddx)) return rc;
    if (dw)
        if (const int rc = check_out(dw, dw_type, 1, K, K)) return rc;
    if (!offsets || (dx && M > 0 && !w)) return V4MOE_ENULL;
    if (!aligned_to(offsets, 4) || !aligned_to(w, 2)) return V4MOE_EALIGN;
    if (M == 0 && (!dw || accumulate)) return V4MOE_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    GroupedCall o{x, dy, w, ldx, lddy, K};
    if (const int rc = grouped_operands(o, M, E, N, K, true, dw != nullptr, dx != nullptr && M > 0, workspace, ws_bytes, s))
        return rc;
    // data gradient: the contraction is over N, which the weights have across their rows
    const GroupedArgs r{M, K, N, E, offsets, o.dy, o.lddy, o.w, o.ldw, (int64_t)N * o.ldw,
                        MmOut{dx, lddx, 0, K, dx_type == V4MOE_TYPE_BF16, 0}};
    const GroupedArgs g{M, K, 0, E, offsets, o.dy, o.lddy, o.x, o.ldx, 0,
                        MmOut{dw, K, N, K, dw_type == V4MOE_TYPE_BF16, accumulate != 0}};
    const bool rows = dx && M > 0;
    if ((rows && dw ? run_both(r, g, s) : rows ? run_rows<true>(r, s) : dw ? run_weights(g, s) : hipSuccess) != hipSuccess)
        return V4MOE_ELAUNCH;
    return V4MOE_OK;
}

}  // extern "C"
