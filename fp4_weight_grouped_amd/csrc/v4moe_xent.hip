// v4moe_xent.hip -- softmax cross entropy over a large vocabulary from the hidden
// states and the head's weight: loss, and the gradients of both, without the logits
// [T][V] in memory.
//
//   z[t][v] = sum_h x[t][h] W[v][h]
//   lse[t]  = log sum_v exp(z[t][v]),   loss[t] = lse[t] - z[t][y_t]
//   d[t][v] = g_t (exp(z[t][v] - lse[t]) - [v = y_t]),   dx = d W,   dW = d^T x
//
// Tokens without a target (y_t not in [0, V)) have loss 0 and no gradient, and what
// their rows hold reaches nothing: the others' rows are packed first, so that they cost
// nothing either.
//
// Forward: the logits of a tile end in registers, where each row's maximum and sum of
// exponentials over 64 columns are taken; the parts are joined in a fixed order.
// Backward: pieces of the vocabulary, of which d is held in bf16 (at most about 256 MiB);
// the logits are computed again from the same operands, in the same order.  Most of a
// gradient is its target's term, -g W[y_t] and -g x_t, so that d there is not left at
// 8 bits: what its rounding left, one number a token, is added to both products (dx: in
// fp32 where its slices meet; dW: as 16 bits in all, by one more product of the few tokens
// whose target a tile has).  A caller who wants fp32 results as fp32 products give them has
// all of d as two bf16 numbers, and twice the products for it.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"
#include "v4moe_mm.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace v4moe {

namespace {

// What k_xent_rows leaves for the later kernels: how many rows were packed, and the
// largest finite |g| among them (1 where that is 0).
struct XentCtrl { int n; float largest; };

__device__ __forceinline__ float exp_(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// Numbers the tokens with a target: pos[t] their place among them (-1 for the others),
// idx the tokens in order.  More than kFewTokens of them; one block, 4096 tokens a step: 10 us at
// 8192, beside products that take milliseconds by then.
// loss, lse (or null): zeros for the tokens without one.  g (or null): the incoming gradients.
__global__ __launch_bounds__(1024) void k_xent_rows(int T, int V, const int64_t* __restrict__ targets,
                                                    const float* __restrict__ g, int64_t gs, int* __restrict__ pos,
                                                    int* __restrict__ idx, XentCtrl* __restrict__ ctrl,
                                                    float* __restrict__ loss, float* __restrict__ lse)
{
    __shared__ int totals[16];
    __shared__ float largest[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int done = 0;
    float big = 0.0f;
    for (int base = 0; base < T; base += 4096) {
        const int t0 = base + 4 * tid;
        bool has[4];
        int mine = 0;
#pragma unroll
        for (int u = 0; u < 4; u++) {
            has[u] = false;
            if (t0 + u < T) {
                const int64_t y = targets[t0 + u];
                has[u] = y >= 0 && y < V;
                if (has[u] && g) {
                    const float f = fabsf(g[(t0 + u) * gs]);
                    if (f < INFINITY) big = fmaxf(big, f);
                }
                if (!has[u] && loss) loss[t0 + u] = lse[t0 + u] = 0.0f;
            }
            mine += has[u];
        }
        int scan = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 63) totals[wave] = scan;
        __syncthreads();
        int at = done + scan - mine;
        for (int w = 0; w < 16; w++) {
            if (w < wave) at += totals[w];
            done += totals[w];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (t0 + u < T) {
                pos[t0 + u] = has[u] ? at : -1;
                if (has[u]) idx[at++] = t0 + u;
            }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) big = fmaxf(big, __shfl_xor(big, o));
    if (lane == 0) largest[wave] = big;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 16; w++) big = fmaxf(big, largest[w]);
        *ctrl = XentCtrl{done, big > 0.0f ? big : 1.0f};
    }
}

// The packed rows: x [n][H8] (zeros past H), targets, and in the backward lse and g / largest
// (a mean's gradients are equal: theirs is exactly 1, and d is not rounded twice).
struct PackArgs {
    int H, H8;
    const uint16_t* x; int64_t ldx;
    const int64_t* targets;
    const float *lse, *g; int64_t gs;           // (or null)
    uint16_t* xp; int* yp; float *lsep, *gp;
};
// row(r): the r-th token with a target
template <typename F>
__device__ __forceinline__ void pack_rows(const PackArgs& p, int n, float largest, F&& row)
{
    const int segs = p.H8 / 8;
    const int64_t all = (int64_t)n * segs;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
        const int r = (int)(i / segs), c = (int)(i - (int64_t)r * segs) * 8, t = row(r);
        *reinterpret_cast<v4u32*>(p.xp + (int64_t)r * p.H8 + c) = load8(p.x + t * p.ldx, c, p.H);
        if (c == 0) {
            p.yp[r] = (int)p.targets[t];
            if (p.g) {
                p.lsep[r] = p.lse[t];
                p.gp[r] = p.g[t * p.gs] / largest;
            }
        }
    }
}
__global__ __launch_bounds__(256) void k_xent_pack(PackArgs p, const int* __restrict__ idx, const XentCtrl* __restrict__ ctrl)
{
    pack_rows(p, ctrl->n, ctrl->largest, [&](int r) { return idx[r]; });
}

// Both at once, where one step numbers every token: each block does so for itself, the first one for the later kernels
// too (1.4 to 2 us less than two launches: 23 tokens, V = 704, H = 64 12.7 -> 11.2 us as a whole, 512 tokens, V = 2048,
// H = 512 19.9 -> 18.3).
constexpr int kFewTokens = 4096;
__global__ __launch_bounds__(1024) void k_xent_rows_pack(int T, int V, PackArgs p, int* __restrict__ pos, int* __restrict__ idx,
                                                         XentCtrl* __restrict__ ctrl, float* __restrict__ loss,
                                                         float* __restrict__ lse)
{
    __shared__ uint16_t token[kFewTokens];
    __shared__ int totals[16];
    __shared__ float largest[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t0 = 4 * tid;
    const bool first = blockIdx.x == 0;
    bool has[4];
    int mine = 0;
    float big = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; u++) {
        has[u] = false;
        if (t0 + u < T) {
            const int64_t y = p.targets[t0 + u];
            has[u] = y >= 0 && y < V;
            if (has[u] && p.g) {
                const float f = fabsf(p.g[(t0 + u) * p.gs]);
                if (f < INFINITY) big = fmaxf(big, f);
            }
            if (first && !has[u] && loss) loss[t0 + u] = lse[t0 + u] = 0.0f;
        }
        mine += has[u];
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(scan, o);
        if (lane >= o) scan += v;
        big = fmaxf(big, __shfl_xor(big, o));
    }
    if (lane == 63) totals[wave] = scan, largest[wave] = big;
    __syncthreads();
    int at = scan - mine, n = 0;
    big = 0.0f;
    for (int w = 0; w < 16; w++) {
        if (w < wave) at += totals[w];
        n += totals[w];
        big = fmaxf(big, largest[w]);
    }
    big = big > 0.0f ? big : 1.0f;
#pragma unroll
    for (int u = 0; u < 4; u++)
        if (t0 + u < T) {
            if (first) pos[t0 + u] = has[u] ? at : -1;
            if (has[u]) {
                if (first) idx[at] = t0 + u;
                token[at++] = (uint16_t)(t0 + u);
            }
        }
    if (first && tid == 0) *ctrl = XentCtrl{n, big};
    __syncthreads();
    pack_rows(p, n, big, [&](int r) { return (int)token[r]; });
}

// What rounding to bf16 leaves of v (0 of what is no number, which stands alone).
__device__ __forceinline__ float rounding_of(float v)
{
    const float hi = bf16_to_f32(bf16x2(v, 0.0f) & 0xFFFFu);
    return fabsf(hi) < INFINITY ? v - hi : 0.0f;
}

struct LogitsArgs {
    int T, H, V;                       // V: columns of this piece
    int v0;                            // its first
    const XentCtrl* ctrl;
    const uint16_t* x; int64_t ldx;    // packed rows
    const uint16_t* w; int64_t ldw;    // the piece's rows of the weight
    const int* y;
    // forward: (maximum, sum of exponentials) of 64 columns each, [V/64][T], and the target's logit
    float2* parts; float* zy;
    // backward
    const float* lse; const float* g;
    uint16_t* d; int64_t ldd;
    int64_t plane;                     // to d's second numbers, what the first ones' rounding left; 0: none
    float* rest;                       // what d's rounding left at each token's target
    uint16_t* hits; int hits_ld;       // [columns / 64][tokens / 16]: which of 16 tokens have their target in 64 columns
};

// Logits of a piece, a tile per block, and what becomes of them.  16 tokens, H = 4096, V = 131072: 172 us, W's bytes at
// 6.2 TB/s.  8192 tokens: 6.1 ms, 1.30 PFLOP/s, the matrix units 65% busy at the board's power limit; its epilogue looks
// for targets and for the vocabulary's end once per row tile (per element: 4% more).
template <class L, bool GRAD>
__global__ __launch_bounds__(L::THREADS) void k_xent_logits(LogitsArgs p)
{
    static_assert(L::NI % 4 == 0, "parts are of 64 columns in every variant, so that a row's result is the same in all");
    extern __shared__ __align__(1024) uint8_t smem[];
    const int n = p.ctrl->n, tm = (n + L::BM - 1) / L::BM, tn = (p.V + L::BN - 1) / L::BN;
    const int turn = mm_turn(blockIdx.x, tm * tn);
    if (turn < 0) return;
    int im, in;
    mm_band(turn, tm, tn, im, in);
    const MmOperand a{p.x, p.ldx, n}, b{p.w, p.ldw, p.V};
    v4f acc[L::MI][L::NI];
    mm_tile<L>(a, b, im * L::BM, in * L::BN, p.H, smem, acc);
    const int lane = threadIdx.x & 63, r16 = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int mw = im * L::BM + L::first_row(wave / L::WN), nw = in * L::BN + wave % L::WN * L::NI * 16;
    if constexpr (!GRAD) {
#pragma unroll
        for (int i = 0; i < L::MI; i++) {
            const int m = mw + 16 * L::STEP * i + r16;
            if (mw + 16 * L::STEP * i >= n) break;
            const int target = m < n ? p.y[m] - p.v0 - nw : -1;
#pragma unroll
            for (int j0 = 0; j0 < L::NI; j0 += 4) {
                const int n0 = nw + 16 * j0, y = target - 16 * j0;
                if (n0 >= p.V) continue;
                if (n0 + 64 > p.V) {                                   // the last group's end
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (n0 + 16 * j + 4 * kq + e >= p.V) acc[i][j0 + j][e] = -INFINITY;
                }
                if (__ballot((uint32_t)y < 64u)) {                     // a target of the 16 rows lies here
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (y == 16 * j + 4 * kq + e) p.zy[m] = acc[i][j0 + j][e];
                }
                float big = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++) big = fmaxf(big, acc[i][j0 + j][e]);
                big = fmaxf(big, __shfl_xor(big, 16));
                big = fmaxf(big, __shfl_xor(big, 32));
                const float off = big == -INFINITY ? 0.0f : big;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++) sum += exp_(acc[i][j0 + j][e] - off);
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                if (kq == 0 && m < n) p.parts[(int64_t)((p.v0 + n0) >> 6) * p.T + m] = make_float2(big, sum);
            }
        }
    } else {
        static_assert(L::NI == 4, "a wave has one group of 64 columns");
        uint32_t hits = 0;                                             // lane i: of row tile i
#pragma unroll
        for (int i = 0; i < L::MI; i++) {
            if (mw + 16 * L::STEP * i >= n) break;
            const int m = min(mw + 16 * L::STEP * i + r16, n - 1);
            const int y = p.y[m] - p.v0 - nw;
            const float lse = p.lse[m], g = p.g[m];
            // d without the target's 1, which is taken off where a target of the 16 rows lies here
            const uint64_t here = __ballot((uint32_t)y < 16u * L::NI && mw + 16 * L::STEP * i + r16 < n);
            const bool end = nw + 16 * L::NI > p.V, target = here != 0;
            if (lane == i) hits = (uint32_t)here & 0xFFFFu;
#pragma unroll
            for (int j = 0; j < L::NI; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = exp_(acc[i][j][e] - lse);
            if (target) {
#pragma unroll
                for (int j = 0; j < L::NI; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (y == 16 * j + 4 * kq + e) acc[i][j][e] -= 1.0f;
            }
#pragma unroll
            for (int j = 0; j < L::NI; j++) acc[i][j] *= g;
            if (target) {
#pragma unroll
                for (int j = 0; j < L::NI; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (y == 16 * j + 4 * kq + e) p.rest[m] = rounding_of(acc[i][j][e]);
            }
            if (end) {
#pragma unroll
                for (int j = 0; j < L::NI; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (nw + 16 * j + 4 * kq + e >= p.V) acc[i][j][e] = 0.0f;
            }
        }
        if (lane < L::MI && mw + 16 * L::STEP * lane < n && nw < p.V)
            p.hits[(int64_t)(nw >> 6) * p.hits_ld + (mw >> 4) + L::STEP * lane] = (uint16_t)hits;
        // (columns up to a multiple of 8: the products read whole segments)
        const MmOut o{p.d, p.ldd, n, (p.V + 7) / 8 * 8, 1, 0};
        mm_store_tile<L, false>(acc, smem, o, im * L::BM, in * L::BN);
        if (p.plane) {
#pragma unroll
            for (int i = 0; i < L::MI; i++)
#pragma unroll
                for (int j = 0; j < L::NI; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[i][j][e] = rounding_of(acc[i][j][e]);
            mm_store_tile<L, false>(acc, smem, MmOut{p.d + p.plane, p.ldd, n, o.N, 1, 0}, im * L::BM, in * L::BN);
        }
    }
}

// lse and loss of the packed rows from P parts each (8192 tokens, P = 2048: 29 us, 4.2 TB/s): 16 rows by 64 groups of parts per
// block; a group takes every 64th part in order, then the groups are joined in a tree.
__global__ __launch_bounds__(1024) void k_xent_join(int T, int P, const XentCtrl* __restrict__ ctrl,
                                                    const int* __restrict__ idx, const float2* __restrict__ parts,
                                                    const float* __restrict__ zy, float* __restrict__ loss,
                                                    float* __restrict__ lse)
{
    __shared__ float2 joined[64][17];
    const int n = ctrl->n, r = threadIdx.x & 15, grp = threadIdx.x >> 4, m = blockIdx.x * 16 + r;
    if (blockIdx.x * 16 >= n) return;
    auto join = [](float2 a, float2 b) {
        const float big = fmaxf(a.x, b.x);
        if (big == -INFINITY) return make_float2(big, a.y + b.y);
        return make_float2(big, a.y * exp_(a.x - big) + b.y * exp_(b.x - big));
    };
    float2 acc = make_float2(-INFINITY, 0.0f);
    for (int p0 = grp; p0 < P; p0 += 64 * 8) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; u++)
            v[u] = p0 + 64 * u < P && m < n ? parts[(int64_t)(p0 + 64 * u) * T + m] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int u = 0; u < 8; u++) acc = join(acc, v[u]);
    }
    joined[grp][r] = acc;
    __syncthreads();
    for (int o = 32; o > 0; o >>= 1) {
        if (grp < o) joined[grp][r] = join(joined[grp][r], joined[grp + o][r]);
        __syncthreads();
    }
    if (grp == 0 && m < n) {
        const float2 v = joined[0][r];
        const float l = v.x + logf(v.y);
        const int t = idx[m];
        lse[t] = l;
        loss[t] = l - zy[m];
    }
}

struct XentGradArgs {
    int T, H, H8, V;                    // V: columns of this piece
    int piece;                          // columns of a whole piece
    const XentCtrl* ctrl;
    const uint16_t* x; const uint16_t* w; int64_t ldw;
    const uint16_t* d; int64_t ldd;
    int parts; int64_t plane;           // numbers of d, from one to the next
    int v0; const int* y; const float* rest;
    const uint16_t* hits; int hits_ld;
    float* dx;                          // [slices][n][H8] of the n packed rows
    int first;                          // the first piece writes dx, the others add to it
    MmOut dw;                           // the piece's rows
};

// Slices of a piece's contraction for dx: where the packed rows make few tiles, until there is a block for each CU
// at 256 rows a tile and two at fewer.  A slice's columns are a multiple of 64.
__host__ __device__ inline int dx_blocks(int bm) { return bm >= 256 ? 256 : 512; }
struct DxSlices { int count, columns; };
__host__ __device__ inline DxSlices dx_slices(int64_t tiles, int bm, int piece)
{
    int64_t n = tiles > 0 ? dx_blocks(bm) / tiles : 1;
    const int64_t most = (piece + 255) / 256;
    n = n < 1 ? 1 : n > most ? most : n;
    return DxSlices{(int)n, (int)(((piece + 63) / 64 + n - 1) / n * 64)};
}

// dx of the packed rows over a slice of a piece's columns.  4096 tokens by 32768 columns, H = 4096: 800 us, 1.37 PFLOP/s.
template <class L>
__device__ __forceinline__ void dx_block(const XentGradArgs& p, int block, uint8_t* smem)
{
    const int n = p.ctrl->n, tm = (n + L::BM - 1) / L::BM, tn = (p.H8 + L::BN - 1) / L::BN;
    const DxSlices sl = dx_slices((int64_t)tm * tn, L::BM, p.piece);
    const int turn = mm_turn(block, tm * tn * sl.count);
    if (turn < 0) return;
    const int slice = turn / (tm * tn), k0 = slice * sl.columns;
    int im, in;
    mm_band(turn % (tm * tn), tm, tn, im, in);
    const MmOperand b{p.w + k0 * p.ldw, p.ldw, p.H8};
    v4f acc[L::MI][L::NI];
    mm_zero<L>(acc);
    for (int part = 0; part < p.parts; part++) {
        const MmOperand a{p.d + part * p.plane + k0, p.ldd, n};
        mm_tile<L, true>(a, b, im * L::BM, in * L::BN, max(min(p.V - k0, sl.columns), 0), smem, acc);
    }
    const MmOut o{p.dx + (int64_t)slice * n * p.H8, p.H8, n, p.H8, 0, !p.first};
    mm_store_tile<L>(acc, smem, o, im * L::BM, in * L::BN);
}

// The tokens, of 4096 from base on, whose target is one of a wave's rows of dW: 64 for each lane.
template <class L>
__device__ __forceinline__ uint64_t targets_of(const XentGradArgs& p, int n, int first, int base)
{
    const int t = base + 64 * ((int)threadIdx.x & 63);
    uint64_t in = 0;
#pragma unroll
    for (int c = 0; c < L::MI * 16; c += 64)
        if (t < n && first + c < p.V)
            in |= *reinterpret_cast<const uint64_t*>(p.hits + (int64_t)((first + c) >> 6) * p.hits_ld + (t >> 4));
    return n - t < 64 ? in & ((1ull << max(n - t, 0)) - 1) : in;
}

// Adds what d's rounding left at the targets to a wave's tile of dW: rest[t] x[t] to row y[t], 32 tokens at a time, in
// order.  `in`: targets_of the first 4096, fetched ahead of the tile.  A wave without any is done; one with a few waits
// for a list and two loads in a row: 1237 tokens, 495 of them with a target, 50021 x 1001, the call 229 -> 238 us (249 where
// a block looked through the tokens here); 4096 tokens, V = 131072, H = 4096, 1.2% more (1.6).  One target for all of 4096
// tokens, so that one tile has them all: both gradients of 131072 columns 10000 -> 11400 us.
template <class L>
__device__ __forceinline__ void add_targets(const XentGradArgs& p, uint64_t in, int n, int first, int column, uint8_t* smem,
                                            v4f (&acc)[L::MI][L::NI])
{
    static_assert(!L::RAGGED && L::MI % 4 == 0, "a wave's rows follow each other, in groups of 64");
    static_assert(L::C_BYTES >= 4096 * 2, "the list has the room that the wave's sums have later");
    typedef short v8s __attribute__((ext_vector_type(8)));
    const int lane = threadIdx.x & 63, r16 = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + wave * L::C_BYTES);
    for (int base = 0; base < n; base += 4096) {
        if (base > 0) in = targets_of<L>(p, n, first, base);
        if (!__ballot(in != 0)) continue;
        int at = __popcll(in), all = at;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(all, o);
            if (lane >= o) all += v;
        }
        at = all - at;
        all = __builtin_amdgcn_readlane(all, 63);
        __builtin_amdgcn_wave_barrier();
        for (; in; in &= in - 1) list[at++] = (uint16_t)(64 * lane + __builtin_ctzll(in));
        __builtin_amdgcn_wave_barrier();
        for (int k0 = 0; k0 < all; k0 += 32) {
            v8s rest, x[L::NI];
            int row[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int k = k0 + 8 * kq + e, t = base + list[min(k, all - 1)];
                row[e] = p.y[t] - p.v0 - first;
                rest[e] = k < all ? (short)bf16x2(p.rest[t], 0.0f) : (short)0;
#pragma unroll
                for (int j = 0; j < L::NI; j++) x[j][e] = (short)p.x[(int64_t)t * p.H8 + min(column + 16 * j, p.H8 - 1)];
            }
#pragma unroll
            for (int i = 0; i < L::MI; i++) {
                v8s a;
                bool any = false;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const bool here = row[e] == 16 * i + r16;
                    any |= here;
                    a[e] = here ? rest[e] : (short)0;
                }
                if (!__ballot(any)) continue;
#pragma unroll
                for (int j = 0; j < L::NI; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x[j]),
                                                                        __builtin_bit_cast(v8bf, a), acc[i][j], 0, 0, 0);
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
}

// The piece's rows of dW: the packed tokens are the contraction (the same sizes 830 us, 30 of them the targets').
template <class L>
__device__ __forceinline__ void dw_block(const XentGradArgs& p, int tm, int tn, int block, uint8_t* smem)
{
    const int n = p.ctrl->n;
    if (n == 0 && p.dw.accumulate) return;          // (adding a sum of nothing would turn -0 into 0)
    int im, in;
    mm_band(mm_turn(block, tm * tn), tm, tn, im, in);
    const MmOperand b{p.x, p.H8, p.H8};
    v4f acc[L::MI][L::NI];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int first = im * L::BM + L::first_row(wave / L::WN);
    const int column = in * L::BN + wave % L::WN * L::NI * 16 + ((int)threadIdx.x & 15);
    const uint64_t targets = p.parts == 1 ? targets_of<L>(p, n, first, 0) : 0;
    mm_zero<L>(acc);
    for (int part = 0; part < p.parts; part++) {
        const MmOperand a{p.d + part * p.plane, p.ldd, (p.V + 7) / 8 * 8};
        mm_tile<L, true>(a, b, im * L::BM, in * L::BN, n, smem, acc);
    }
    if (p.parts == 1) add_targets<L>(p, targets, n, first, column, smem, acc);
    const float s = p.ctrl->largest;
#pragma unroll
    for (int i = 0; i < L::MI; i++)
#pragma unroll
        for (int j = 0; j < L::NI; j++) acc[i][j] *= s;
    mm_store_tile<L>(acc, smem, p.dw, im * L::BM, in * L::BN);
}

template <class L>
__global__ __launch_bounds__(L::THREADS) void k_xent_dx(XentGradArgs p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    dx_block<L>(p, blockIdx.x, smem);
}
template <class L>
__global__ __launch_bounds__(L::THREADS) void k_xent_dw(XentGradArgs p, int tm, int tn)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    dw_block<L>(p, tm, tn, blockIdx.x, smem);
}
// Both, dx's blocks, whose contraction is the longer one, first (1237 tokens, 495 of them with a target, 50021 x 1001:
// 138 us, 9 of them the targets'; one after the other, with the tiles best for each, 19 more).
template <class X, class W>
__global__ __launch_bounds__(X::THREADS) void k_xent_gradients(XentGradArgs p, int xblocks, int tm, int tn)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((int)blockIdx.x < xblocks) dx_block<X>(p, blockIdx.x, smem);
    else dw_block<W>(p, tm, tn, (int)blockIdx.x - xblocks, smem);
}

// dx of every token: the slices' sums in order and what d's rounding left at the target, times the largest |g|; zeros
// without a target.  4096 tokens, H = 4096: 29 us, 7 of them the targets' rows of W.
template <typename T_>
__global__ __launch_bounds__(256) void k_xent_finish(int T, int H, int H8, int bm, int bn, int piece,
                                                     const XentCtrl* __restrict__ ctrl,
                                                     const int* __restrict__ pos, const float* __restrict__ acc,
                                                     const int* __restrict__ y, const float* __restrict__ rest,
                                                     const uint16_t* __restrict__ w, int64_t ldw, T_* __restrict__ dx,
                                                     int64_t ld)
{
    const int quads = H8 / 4;
    const int64_t all = (int64_t)T * quads;
    const float s = ctrl->largest;
    const int n = ctrl->n, slices = dx_slices((int64_t)((n + bm - 1) / bm) * ((H8 + bn - 1) / bn), bm, piece).count;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int t = (int)(i / quads), c = (int)(i - (int64_t)t * quads) * 4, m = pos[t];
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (m >= 0) {
            const v2u32 wy = *reinterpret_cast<const v2u32*>(w + y[m] * ldw + c);
            const float left = rest ? rest[m] : 0.0f;          // (null: d has two numbers)
            for (int k = 0; k < slices; k += 4) {
                float4 f[4];
#pragma unroll
                for (int u = 0; u < 4; u++)
                    f[u] = k + u < slices ? *reinterpret_cast<const float4*>(acc + ((int64_t)(k + u) * n + m) * H8 + c)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    v[0] += f[u].x;
                    v[1] += f[u].y;
                    v[2] += f[u].z;
                    v[3] += f[u].w;
                }
            }
            v[0] += left * bf16_to_f32(wy[0] & 0xFFFFu);
            v[1] += left * bf16_to_f32(wy[0] >> 16);
            v[2] += left * bf16_to_f32(wy[1] & 0xFFFFu);
            v[3] += left * bf16_to_f32(wy[1] >> 16);
        }
        T_* o = dx + t * ld + c;
        if constexpr (sizeof(T_) == 2) {
            const uint32_t lo = bf16x2(v[0] * s, v[1] * s), hi = bf16x2(v[2] * s, v[3] * s);
            if (c + 4 <= H) {
                *reinterpret_cast<v2u32_any*>(o) = v2u32{lo, hi};
            } else {
                for (int e = 0; e < 4 && c + e < H; e++) o[e] = (uint16_t)((e < 2 ? lo : hi) >> (16 * (e & 1)));
            }
        } else {
            for (int e = 0; e < 4 && c + e < H; e++) o[e] = v[e] * s;
        }
    }
}

// ---- host ----
template <class L, bool GRAD>
hipError_t launch_logits(const LogitsArgs& p, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_xent_logits<L, GRAD>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int64_t tiles = over(p.T, L::BM) * over(p.V, L::BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(L::THREADS), L::BYTES, s, p);
    return hipGetLastError();
}
// Rows of the logits' tiles: those of the few tokens', 256 columns wide, or of a square one.
int logits_rows(int64_t T, int64_t H, int64_t V)
{
    if (T <= 64) return T <= 16 ? 16 : T <= 32 ? 32 : 64;
    return kMmVariants[mm_choose(3, H, [&](int64_t bm, int64_t bn) { return over(T, bm) * over(V, bn); })].bm;
}
template <bool GRAD>
hipError_t run_logits(const LogitsArgs& p, hipStream_t s)
{
    switch (logits_rows(p.T, p.H, p.V)) {
    case 16: return launch_logits<MmTile<1, 4, 1, 4, 4, false, false>, GRAD>(p, s);
    case 32: return launch_logits<MmTile<1, 4, 2, 4, 3, false, false>, GRAD>(p, s);
    case 64: return launch_logits<MmTile<1, 4, 4, 4, 2, false, false>, GRAD>(p, s);
    case 128: return launch_logits<MmTile<2, 2, 4, 4, 2, false, false>, GRAD>(p, s);
    default: return launch_logits<MmTile<2, 4, 8, 4, 2, false, false>, GRAD>(p, s);
    }
}

// blocks of dx, whatever n is
template <class L>
int64_t dx_tiles(const XentGradArgs& p) { return std::max<int64_t>(over(p.T, L::BM) * over(p.H8, L::BN), dx_blocks(L::BM)); }
template <class L>
hipError_t launch_dx(const XentGradArgs& p, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_xent_dx<L>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int64_t tiles = dx_tiles<L>(p);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(L::THREADS), L::BYTES, s, p);
    return hipGetLastError();
}
using XentW128 = MmTile<2, 2, 4, 4, 2, true, true>;
using XentX128 = MmTile<2, 2, 4, 4, 2, false, true>;
constexpr int kX128 = 3;                // of kMmVariants
int dw_variant(int64_t T, int64_t H, int64_t V)
{
    return mm_choose(3, T, [&](int64_t bm, int64_t bn) { return over(V, bm) * over(H, bn); });
}
// Both gradients in one launch where dW has few tiles, with 128x128 ones both: the end of the one runs beside the
// begin of the other.
bool both_at_once(int64_t T, int64_t H, int64_t piece) { return dw_variant(T, H, piece) == kX128; }

// The tile of the least time with its slices, whose sums are written and read again at some 5 TB/s.  (The tokens
// with a target are the device's to know: all of them are counted.)
const MmVariant& dx_tile(int64_t T, int64_t H8, int64_t piece, bool both)
{
    if (both) return kMmVariants[kX128];
    int best = 1;
    float least = 0.0f;
    for (int v = 1; v < 5; v++) {
        const int64_t tiles = over(T, kMmVariants[v].bm) * over(H8, kMmVariants[v].bn);
        const DxSlices sl = dx_slices(tiles, kMmVariants[v].bm, (int)piece);
        const float us = mm_time(kMmVariants[v], tiles * sl.count, sl.columns) + (float)(T * H8) * sl.count * 8.0f / 5.0e6f;
        if (v == 1 || us < least) best = v, least = us;
    }
    return kMmVariants[best];
}
hipError_t run_dx(const XentGradArgs& p, hipStream_t s)
{
    switch (dx_tile(p.T, p.H8, p.piece, false).bm) {
    case 32: return launch_dx<MmTile<2, 2, 1, 2, 4, false, true>>(p, s);
    case 64: return launch_dx<MmTile<2, 2, 2, 2, 3, false, true>>(p, s);
    case 128: return launch_dx<XentX128>(p, s);
    default: return launch_dx<MmTile<2, 4, 8, 4, 2, false, true>>(p, s);
    }
}
template <class L>
hipError_t launch_dw(const XentGradArgs& p, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_xent_dw<L>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int64_t tm = over(p.V, L::BM), tn = over(p.H, L::BN);
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(L::THREADS), L::BYTES, s, p, (int)tm, (int)tn);
    return hipGetLastError();
}
hipError_t run_dw(const XentGradArgs& p, hipStream_t s)
{
    if (dw_variant(p.T, p.H, p.piece) == kX128) return launch_dw<XentW128>(p, s);
    return launch_dw<MmTile<2, 4, 8, 4, 2, true, true>>(p, s);
}
hipError_t run_gradients(const XentGradArgs& p, hipStream_t s)
{
    if (!both_at_once(p.T, p.H, p.piece)) {
        if (const hipError_t e = run_dx(p, s); e != hipSuccess) return e;
        return run_dw(p, s);
    }
    using X = XentX128;
    using W = XentW128;
    static_assert(X::BYTES == W::BYTES && X::THREADS == W::THREADS, "one launch");
    static LdsAllowed allowed;
    const auto kernel = k_xent_gradients<X, W>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), X::BYTES, allowed); e != hipSuccess) return e;
    const int64_t blocks = dx_tiles<X>(p), tm = over(p.V, W::BM), tn = over(p.H, W::BN);
    if (blocks + tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks + tm * tn)), dim3(X::THREADS), X::BYTES, s, p, (int)blocks, (int)tm, (int)tn);
    return hipGetLastError();
}

// Masks of 16 tokens for a group of columns: whole 64-bit words.
int64_t hits_ld(int64_t T) { return over(T, 64) * 4; }

struct XentLayout {
    size_t ctrl, idx, pos, y, zy, x, parts, lse, g, rest, hits, d, dx, w, total;
    bool pad_w;
    int piece;                      // columns of a piece; half as many where d has two numbers
};
XentLayout xent_layout(int64_t T, int64_t H, int64_t V, const void* w, int64_t ldw, bool backward)
{
    XentLayout L{};
    if (T == 0) T = 1;
    L.pad_w = !in_place(w, H, ldw);
    size_t o = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += up256((size_t)bytes);
        return at;
    };
    const int64_t H8 = up8(H);
    L.ctrl = take(sizeof(XentCtrl));
    L.idx = take(T * 4);
    L.pos = take(T * 4);
    L.y = take(T * 4);
    L.x = take(T * H8 * 2);
    if (L.pad_w) L.w = take(V * H8 * 2);
    if (!backward) {
        L.zy = take(T * 4);
        L.parts = take(over(V, 64) * T * 8);
    } else {
        // d of a piece in at most 256 MiB, but for 256 columns at least
        const int64_t most = std::max<int64_t>((int64_t(128) << 20) / T / 256 * 256, 256);
        L.piece = (int)std::min(most, (V + 255) / 256 * 256);
        L.lse = take(T * 4);
        L.g = take(T * 4);
        L.rest = take(T * 4);
        L.hits = take(over(L.piece, 64) * hits_ld(T) * 2);
        L.d = take(T * (int64_t)L.piece * 2);
        // dx of every row, or of fewer rows in slices: dx_blocks tiles then (of either tile, with dW or alone)
        int64_t most_dx = T * H8;
        for (int both = 0; both < 2; both++)
            for (const int piece : {L.piece, L.piece / 2}) {
                const MmVariant& t = dx_tile(T, H8, piece, both && both_at_once(T, H, piece));
                most_dx = std::max(most_dx, std::min<int64_t>((int64_t)dx_blocks(t.bm) * t.bm * t.bn, T * H8 * over(piece, 256)));
            }
        L.dx = take(most_dx * 4);
    }
    L.total = o;
    return L;
}

int check_xent(int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
               const int64_t* targets)
{
    if (!side_ok(T) || !side_ok(H) || !side_ok(V) || H < 1 || V < 1) return V4MOE_EDIMS;
    if (const int rc = check_rows(x, T, H, ldx)) return rc;
    if (const int rc = check_rows(w, V, H, ldw)) return rc;
    if (T > 0 && !targets) return V4MOE_ENULL;
    return aligned_to(targets, 8) ? V4MOE_OK : V4MOE_EALIGN;
}

// The weight as the products read it, and the packed rows.
struct XentCall {
    XentLayout L;
    uint8_t* ws;
    const uint16_t* w;
    int64_t ldw;
    int H8;
    template <typename T> T* at(size_t o) const { return reinterpret_cast<T*>(ws + o); }
};
int xent_begin(XentCall& c, int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
               const int64_t* targets, const float* lse_in, const float* g, int64_t gs, float* loss, float* lse, void* workspace,
               size_t ws_bytes, bool backward, hipStream_t s)
{
    if (!workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    c.L = xent_layout(T, H, V, w, ldw, backward);
    if (ws_bytes < c.L.total) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    c.ws = static_cast<uint8_t*>(workspace);
    c.w = w;
    c.ldw = ldw;
    c.H8 = (int)up8(H);
    if (c.L.pad_w) {
        const PadRows job{V, H, w, ldw, c.at<uint16_t>(c.L.w)};
        if (launch_pad_rows(&job, 1, s) != hipSuccess) return V4MOE_ELAUNCH;
        c.w = job.dst;
        c.ldw = c.H8;
    }
    const PackArgs p{H, c.H8, x, ldx, targets, lse_in, g, gs, c.at<uint16_t>(c.L.x), c.at<int>(c.L.y), c.at<float>(c.L.lse),
                     c.at<float>(c.L.g)};
    const int64_t segs = (int64_t)T * (c.H8 / 8);
    if (T <= kFewTokens) {
        const unsigned blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>(over(segs, 1024), 512));
        hipLaunchKernelGGL(k_xent_rows_pack, dim3(blocks), dim3(1024), 0, s, T, V, p, c.at<int>(c.L.pos), c.at<int>(c.L.idx),
                           c.at<XentCtrl>(c.L.ctrl), loss, lse);
    } else {
        hipLaunchKernelGGL(k_xent_rows, dim3(1), dim3(1024), 0, s, T, V, targets, g, gs, c.at<int>(c.L.pos), c.at<int>(c.L.idx),
                           c.at<XentCtrl>(c.L.ctrl), loss, lse);
        hipLaunchKernelGGL(k_xent_pack, dim3((unsigned)std::min<int64_t>(over(segs, 256), 8192)), dim3(256), 0, s, p,
                           c.at<int>(c.L.idx), c.at<XentCtrl>(c.L.ctrl));
    }
    return hipGetLastError() == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) size_t moe_linear_xent_workspace_bytes(int32_t T, int32_t H, int32_t V,
                                                                              const uint16_t* w, int64_t ldw,
                                                                              int32_t backward)
{
    if (!side_ok(T) || !side_ok(H) || !side_ok(V) || H < 1 || V < 1) return 0;
    return xent_layout(T, H, V, w, ldw, backward != 0).total;
}

__attribute__((visibility("default"))) int32_t moe_linear_xent_tile(int32_t T, int32_t H, int32_t V, int32_t what, int32_t both)
{
    if (!side_ok(T) || !side_ok(H) || !side_ok(V) || T < 1 || H < 1 || V < 1) return 0;
    if (what < V4MOE_PRODUCT_FORWARD || what > V4MOE_PRODUCT_AGAIN) return 0;
    const int piece = xent_layout(T, H, V, nullptr, up8(H), true).piece, columns = std::min(piece, V);
    if (what == V4MOE_PRODUCT_FORWARD || what == V4MOE_PRODUCT_AGAIN) {
        const int bm = logits_rows(T, H, what == V4MOE_PRODUCT_FORWARD ? V : columns);
        return bm << 16 | (bm == 128 ? 128 : 256);
    }
    const bool shared = both && both_at_once(T, H, piece);
    const MmVariant& t = what == V4MOE_PRODUCT_DX ? dx_tile(T, up8(H), piece, shared) : kMmVariants[dw_variant(T, H, piece)];
    return tile_code(t) | (shared ? V4MOE_TILE_SHARED : 0);
}

__attribute__((visibility("default"))) int moe_linear_xent(int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx,
                                                           const uint16_t* w, int64_t ldw, const int64_t* targets,
                                                           float* loss, float* lse, void* workspace, size_t ws_bytes,
                                                           void* stream)
{
    if (const int rc = check_xent(T, H, V, x, ldx, w, ldw, targets)) return rc;
    if (T == 0) return V4MOE_OK;
    if (!loss || !lse) return V4MOE_ENULL;
    if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return V4MOE_EALIGN;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    XentCall c;
    if (const int rc = xent_begin(c, T, H, V, x, ldx, w, ldw, targets, nullptr, nullptr, 0, loss, lse, workspace, ws_bytes,
                                  false, s))
        return rc;
    LogitsArgs p{};
    p.T = T, p.H = H, p.V = V;
    p.ctrl = c.at<XentCtrl>(c.L.ctrl);
    p.x = c.at<uint16_t>(c.L.x), p.ldx = c.H8;
    p.w = c.w, p.ldw = c.ldw;
    p.y = c.at<int>(c.L.y);
    p.parts = c.at<float2>(c.L.parts), p.zy = c.at<float>(c.L.zy);
    if (run_logits<false>(p, s) != hipSuccess) return V4MOE_ELAUNCH;
    hipLaunchKernelGGL(k_xent_join, dim3((unsigned)over(T, 16)), dim3(1024), 0, s, T, (int)over(V, 64), p.ctrl,
                       c.at<int>(c.L.idx), p.parts, p.zy, loss, lse);
    return hipGetLastError() == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_linear_xent_backward(
    int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, const int64_t* targets,
    const float* lse, const float* dloss, int64_t dloss_stride, void* dx, int32_t dx_type, int64_t lddx, void* dw,
    int32_t dw_type, int64_t lddw, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_xent(T, H, V, x, ldx, w, ldw, targets)) return rc;
    if (!dx && !dw) return V4MOE_ENULL;
    if (dx)
        if (const int rc = check_out(dx, dx_type, T, H, lddx)) return rc;
    if (dw)
        if (const int rc = check_out(dw, dw_type, V, H, lddw)) return rc;
    if (dloss_stride < 0 || dloss_stride > (1ll << 40)) return V4MOE_EDIMS;
    if (T > 0 && (!lse || !dloss)) return V4MOE_ENULL;
    if (!aligned_to(lse, 4) || !aligned_to(dloss, 4)) return V4MOE_EALIGN;
    if (T == 0 && (!dw || (accumulate & ~V4MOE_GRAD_FULL))) return V4MOE_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    XentCall c;
    if (const int rc = xent_begin(c, T, H, V, x, ldx, w, ldw, targets, lse, dloss, dloss_stride, nullptr, nullptr, workspace,
                                  ws_bytes, true, s))
        return rc;
    const auto* ctrl = c.at<XentCtrl>(c.L.ctrl);
    const bool full = accumulate & V4MOE_GRAD_FULL, add = accumulate & ~V4MOE_GRAD_FULL;
    const int piece = full ? c.L.piece / 2 : c.L.piece;
    for (int v0 = 0; v0 < V; v0 += piece) {
        const int n = std::min(piece, V - v0);
        LogitsArgs p{};
        p.T = T, p.H = H, p.V = n, p.v0 = v0;
        p.ctrl = ctrl;
        p.x = c.at<uint16_t>(c.L.x), p.ldx = c.H8;
        p.w = c.w + v0 * c.ldw, p.ldw = c.ldw;
        p.y = c.at<int>(c.L.y);
        p.lse = c.at<float>(c.L.lse), p.g = c.at<float>(c.L.g);
        p.d = c.at<uint16_t>(c.L.d), p.ldd = piece;
        p.plane = full ? (int64_t)T * piece : 0;
        p.rest = c.at<float>(c.L.rest);
        p.hits = c.at<uint16_t>(c.L.hits), p.hits_ld = (int)hits_ld(T);
        if (T > 0 && run_logits<true>(p, s) != hipSuccess) return V4MOE_ELAUNCH;
        XentGradArgs q{};
        q.T = T, q.H = H, q.H8 = c.H8, q.V = n;
        q.piece = piece;
        q.parts = full ? 2 : 1, q.plane = p.plane;
        q.ctrl = ctrl;
        q.x = p.x, q.w = p.w, q.ldw = p.ldw, q.d = p.d, q.ldd = p.ldd;
        q.v0 = v0, q.y = p.y, q.rest = p.rest;
        q.hits = p.hits, q.hits_ld = p.hits_ld;
        q.dx = c.at<float>(c.L.dx), q.first = v0 == 0;
        if (dw) {
            const bool bf16 = dw_type == V4MOE_TYPE_BF16;
            q.dw = MmOut{static_cast<uint8_t*>(dw) + (int64_t)v0 * lddw * (bf16 ? 2 : 4), lddw, n, H, bf16, add};
        }
        const bool rows = dx && T > 0;
        if ((rows && dw ? run_gradients(q, s) : rows ? run_dx(q, s) : dw ? run_dw(q, s) : hipSuccess) != hipSuccess)
            return V4MOE_ELAUNCH;
    }
    if (dx && T > 0) {
        const dim3 grid((unsigned)std::min<int64_t>(over((int64_t)T * (c.H8 / 4), 256), 8192));
        const MmVariant& t = dx_tile(T, c.H8, piece, dw && both_at_once(T, H, piece));
        const float* rest = full ? nullptr : c.at<float>(c.L.rest);
        if (dx_type == V4MOE_TYPE_BF16)
            hipLaunchKernelGGL(k_xent_finish<uint16_t>, grid, dim3(256), 0, s, T, H, c.H8, t.bm, t.bn, piece, ctrl,
                               c.at<int>(c.L.pos), c.at<float>(c.L.dx), c.at<int>(c.L.y), rest, c.w, c.ldw,
                               static_cast<uint16_t*>(dx), lddx);
        else
            hipLaunchKernelGGL(k_xent_finish<float>, grid, dim3(256), 0, s, T, H, c.H8, t.bm, t.bn, piece, ctrl, c.at<int>(c.L.pos),
                               c.at<float>(c.L.dx), c.at<int>(c.L.y), rest, c.w, c.ldw, static_cast<float*>(dx), lddx);
    }
    return hipGetLastError() == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

}  // extern "C"
