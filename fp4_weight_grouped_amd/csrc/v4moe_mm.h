// v4moe_mm.h -- a block's tile of a bf16 matrix product on gfx950, for the kernels
// that differ in where a tile's operands lie and in what becomes of its sums.
//
//   C[m][n] = sum_k A(m, k) B(n, k),  fp32 sums
//
// Either operand may be contiguous along k ("rows": [m][k]) or along its own
// index ("columns": [k][m]), which the gradients need: dx = dy W reads W along
// the contraction, dW = dy^T x both operands.  Nothing is transposed in memory:
// columns are staged as they lie and gfx950's transposing LDS read turns them
// into the matrix instruction's operand.
//
// Every element of C is one chain of matrix instructions over k in steps of 32,
// ascending, whatever the tile: a result does not depend on the variant, nor on
// the other rows of a call, in any bit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

namespace v4moe {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u32 __attribute__((ext_vector_type(4)));
typedef v4u32 v4u32_any __attribute__((aligned(2)));
typedef uint32_t v2u32 __attribute__((ext_vector_type(2)));
typedef v2u32 v2u32_any __attribute__((aligned(2)));

// Sixteen bytes of a row from element k on; zeros past K.
__device__ __forceinline__ v4u32 load8(const uint16_t* row, int k, int K)
{
    if (k + 8 <= K) return *reinterpret_cast<const v4u32_any*>(row + k);
    v4u32 v;
#pragma unroll
    for (int u = 0; u < 4; u++)
        v[u] = (k + 2 * u < K ? (uint32_t)row[k + 2 * u] : 0u) | (k + 2 * u + 1 < K ? (uint32_t)row[k + 2 * u + 1] << 16 : 0u);
    return v;
}

// What a 16-byte segment past the end of the contraction is copied from.
static __device__ const uint4 g_mm_zeros[64] = {};

// An operand: element (i, k) at p[i * ld + k], or with columns at p[k * ld + i];
// i < n, n >= 1.  p 16-byte aligned, ld a multiple of 8, the contiguous length too.
struct MmOperand {
    const uint16_t* p;
    int64_t ld;
    int n;
};

// WM x WN waves, each MI x NI tiles of 16x16; NS stages of 64 k in LDS.  RAGGED: many tiles end before BM rows (the
// last one of each group).  The row tiles are then dealt to the wave rows in turn, and those past A's end cost no
// products, so that such a tile's waves end together and early (65536 uneven rows of 256 experts, 2048 x 4096: 1408 -> 1305
// us); whole tiles pay for it (8192x8192x8192 740 -> 779 us, 256 rows for each of those experts 1049 -> 1057).
template <int WM_, int WN_, int MI_, int NI_, int NS_, bool ACOL_, bool BCOL_, bool RAGGED_ = false>
struct MmTile {
    static constexpr bool RAGGED = RAGGED_;
    static constexpr int STEP = RAGGED_ ? WM_ : 1;                          // of a wave's row tiles
    static __host__ __device__ constexpr int first_row(int wm) { return wm * (RAGGED_ ? 1 : MI_) * 16; }
    static constexpr int WM = WM_, WN = WN_, MI = MI_, NI = NI_, NS = NS_;
    static constexpr bool ACOL = ACOL_, BCOL = BCOL_;
    static constexpr int NW = WM * WN, THREADS = 64 * NW, BM = WM * MI * 16, BN = WN * NI * 16;
    static constexpr int AP = BM / 8, BP = BN / 8;                          // 1 KiB pieces of a stage
    static constexpr int AJ = (AP + NW - 1) / NW, BJ = (BP + NW - 1) / NW;  // per wave
    static constexpr int OPS = AJ + BJ;
    static constexpr int B_OFF = BM * 128, STAGE = (BM + BN) * 128, RING = NS * STAGE;
    static constexpr int C_BYTES = 2 * 16 * NI * 16 * 4;                    // of staging per wave (mm_store)
    static constexpr int BYTES = RING > NW * C_BYTES ? RING : NW * C_BYTES;
    static_assert(NW > 1 && NS >= 2 && OPS * (NS - 1) < 64, "the barrier frees a slot; vmcnt range");
    static_assert(BYTES <= 163840, "LDS of a CU");
    static_assert(!ACOL || BM >= 64, "columns are staged in rows of 128 bytes or more");
    static_assert(!BCOL || BN >= 64, "columns are staged in rows of 128 bytes or more");
};

// Where the 16-byte segments of a stage go.  Rows [i][64 k]: segment s of row i at
// s ^ (i / 2 % 8), so that the 16 rows of an operand read hit distinct banks.
// Columns [k][W]: pairs of segments (the 32 bytes a transposing read takes of a row)
// XORed by column_swizzle(k), so that the eight rows read together do.
template <int W>
__device__ __forceinline__ int column_swizzle(int k)
{
    if constexpr (W >= 128) return (k & 3) | ((k >> 1) & 4);
    else if constexpr (W == 64) return ((k >> 1) & 1) | ((k >> 2) & 2);
    else return (k >> 3) & 1;
}

// The same pointer, in scalar registers.
__device__ __forceinline__ const uint8_t* mm_uniform(const uint8_t* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

// One operand of a tile, its first index i0: copies into LDS and reads of fragments.
// W: indices of the tile, COL: columns, PJ: pieces per wave, NW: waves.
template <int W, bool COL, int PJ, int NW>
struct MmSide {
    static constexpr int SEGS = W / 8;              // 16-byte segments of a row of k, columns
    const uint8_t* base;                            // of chunk 0
    int64_t step;                                   // bytes to the next chunk
    uint32_t off[PJ];                               // this lane's segments
    int wave, lane;

    __device__ __forceinline__ void begin(const MmOperand& o, int i0, int wave_, int lane_)
    {
        wave = wave_;
        lane = lane_;
        base = reinterpret_cast<const uint8_t*>(o.p + (COL ? (int64_t)i0 : (int64_t)i0 * o.ld));
        step = COL ? o.ld * 128 : 128;
#pragma unroll
        for (int j = 0; j < PJ; j++) {
            const int p = piece(j);
            if constexpr (COL) {
                const int k = row_of(p);
                off[j] = (uint32_t)(k * (int)o.ld * 2 + min(seg_of(p), (o.n - i0) / 8 - 1) * 16);
            } else {
                const int r = row_of(p);
                off[j] = (uint32_t)(min(r, o.n - 1 - i0) * (int)o.ld * 2 + seg_of(p) * 16);
            }
        }
    }
    __device__ __forceinline__ int piece(int j) const { return min(wave + j * NW, W / 8 - 1); }
    // the row (i, or k with columns) and the segment in it that this lane copies of a piece
    __device__ __forceinline__ int row_of(int p) const { return COL ? (p * 64 + lane) / SEGS : p * 8 + (lane >> 3); }
    __device__ __forceinline__ int seg_of(int p) const
    {
        if constexpr (COL) return ((p * 64 + lane) % SEGS) ^ (2 * column_swizzle<W>(row_of(p)));
        else return (lane & 7) ^ ((row_of(p) >> 1) & 7);
    }
    // this wave's copy j of a chunk into a stage (UNIFORM: c is in vector registers)
    template <bool UNIFORM>
    __device__ __forceinline__ void copy(int j, int c, uint32_t to) const
    {
        const uint8_t* from = base + (int64_t)c * step;
        if constexpr (UNIFORM) from = mm_uniform(from);
        dma16s(from, off[j], __builtin_amdgcn_readfirstlane(to + piece(j) * 1024));
    }
    // ... of the last chunk, of which `left` k are the contraction's: zeros past them
    __device__ __forceinline__ void copy_tail(int j, int c, uint32_t to, int left) const
    {
        const int p = piece(j);
        const bool in = COL ? row_of(p) < left : seg_of(p) * 8 < left;
        dma16(in ? (const void*)(base + (int64_t)c * step + off[j]) : (const void*)&g_mm_zeros[lane],
              __builtin_amdgcn_readfirstlane(to + p * 1024));
    }
};

// A lane's reads of the fragments of T tiles, `first` and every STEP-th further: fragment s (0, 1) of tile t
// holds index 16 (first + STEP t) + lane % 16 and k = 32 s + 8 (lane / 16) .. + 7.
template <int W, bool COL, int T, int STEP = 1>
struct MmReader {
    int at[COL ? T : 2];
    // columns, from k0 of the lane's own on (rows of k that its swizzle depends on: k0 + 0 .. 3, and 4 further)
    __device__ __forceinline__ void begin_at(int first, int lane, int k0)
    {
        const int i = lane & 15, k = k0 + (i >> 2), f = column_swizzle<W>(k);
#pragma unroll
        for (int t = 0; t < T; t++) at[t] = k * W * 2 + ((first + STEP * t) ^ f) * 32 + (i & 3) * 8;
    }
    __device__ __forceinline__ void begin(int first, int lane)
    {
        const int i = lane & 15, kq = lane >> 4;
        if constexpr (COL) {
            begin_at(first, lane, 8 * kq);
        } else {
            const int sw = (lane >> 1) & 7, row = (16 * first + i) * 128;
            at[0] = row + ((kq ^ sw) * 16);
            at[1] = row + (((4 + kq) ^ sw) * 16);
        }
    }
    __device__ __forceinline__ v8bf read(const uint8_t* stage, int t, int s) const
    {
        if constexpr (COL) return read_at(stage, t, 32 * s);
        else return *reinterpret_cast<const v8bf*>(stage + at[s] + t * STEP * 2048);
    }
    // columns: of eight k from k1 further on, a multiple of 16 (where the swizzle is the same, as it is 4 further on)
    __device__ __forceinline__ v8bf read_at(const uint8_t* stage, int t, int k1) const
    {
        typedef __attribute__((address_space(3))) v4s* lds4;
        const lds4 p = (lds4)(stage + at[t] + k1 * W * 2), q = (lds4)(stage + at[t] + (k1 + 4) * W * 2);
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p), hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(q);
        typedef short v8s __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(v8bf, v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
};

template <class L>
__device__ __forceinline__ void mm_zero(v4f (&acc)[L::MI][L::NI])
{
#pragma unroll
    for (int i = 0; i < L::MI; i++)
#pragma unroll
        for (int j = 0; j < L::NI; j++) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
}

// The sums of a block's tile from (m0, n0): acc[i][j] of a wave (wm, wn) holds, in lane l,
// row m0 + first_row(wm) + 16 STEP i + l % 16 and columns n0 + 16 (wn NI + j) + 4 (l / 16) .. + 3.
// B is the instruction's first operand, so that a lane has consecutive columns.  The
// block's LDS (L::BYTES) is free when it returns.  ADD: to what acc holds, the chain going on.
template <class L, bool ADD = false>
__device__ __forceinline__ void mm_tile(const MmOperand& a, const MmOperand& b, int m0, int n0, int K, uint8_t* smem,
                                        v4f (&acc)[L::MI][L::NI])
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / L::WN, wn = wave % L::WN;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
    MmSide<L::BM, L::ACOL, L::AJ, L::NW> sa;
    MmSide<L::BN, L::BCOL, L::BJ, L::NW> sb;
    sa.begin(a, m0, wave, lane);
    sb.begin(b, n0, wave, lane);
    const int nch = (K + 63) / 64;
    const int full = K / 64;
    // copies q0 .. of this wave's of chunk c, which is whole
    auto copy = [&](int c, int q0, int n) {
        const uint32_t slot = lds0 + (uint32_t)(c % L::NS) * L::STAGE;
#pragma unroll
        for (int q = q0; q < min(q0 + n, L::OPS); q++) {
            if (q < L::AJ) sa.template copy<L::RAGGED>(q, c, slot);
            else sb.template copy<L::RAGGED>(q - L::AJ, c, slot + L::B_OFF);
        }
    };
    // all of them of any chunk
    auto copy_all = [&](int c) {
        if (c < full) return copy(c, 0, L::OPS);
        const uint32_t slot = lds0 + (uint32_t)(c % L::NS) * L::STAGE;
#pragma unroll
        for (int q = 0; q < L::OPS; q++) {
            if (q < L::AJ) sa.copy_tail(q, c, slot, K - c * 64);
            else sb.copy_tail(q - L::AJ, c, slot + L::B_OFF, K - c * 64);
        }
    };
    MmReader<L::BM, L::ACOL, L::MI, L::STEP> ra;
    MmReader<L::BN, L::BCOL, L::NI> rb;
    ra.begin(L::first_row(wm) / 16, lane);
    rb.begin(wn * L::NI, lane);
    if constexpr (!ADD) mm_zero<L>(acc);
    if (nch > 0) {
#pragma unroll
        for (int c = 0; c < L::NS; c++)
            if (c < nch) copy_all(c);
        if (nch >= L::NS) wait_vm<L::OPS * (L::NS - 1)>();
        else wait_vm<0>();
        __syncthreads();
    }
    // Row tiles of A in registers: all of a small wave tile's, three of a large one's.
    constexpr int MI = L::MI, NI = L::NI, D = MI < 3 ? MI : 3;
    v8bf af[D][2], bf[NI][2];
    auto read_a = [&](const uint8_t* st, int i) {
#pragma unroll
        for (int s = 0; s < 2; s++) af[i % D][s] = ra.read(st, i, s);
    };
    auto open = [&](int c) {
        const uint8_t* st = smem + (c % L::NS) * L::STAGE;
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int s = 0; s < 2; s++) bf[j][s] = rb.read(st + L::B_OFF, j, s);
#pragma unroll
        for (int i = 0; i < (D < MI ? D - 1 : D); i++) read_a(st, i);
    };
    auto row = [&](int i) {
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int j = 0; j < NI; j++)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j][s], af[i % D][s], acc[i][j], 0, 0, 0);
    };
    // The copies of a large tile's next stage go out in groups, a row tile's products after each: all at once they
    // would hold up every wave's products until the memory path has taken them (8192x8192x8192, not RAGGED, 792 -> 752 us).
    constexpr int GROUPS = MI >= 4 ? MI / 2 : 1, PER = (L::OPS + GROUPS - 1) / GROUPS;
    // row tiles of this wave with rows in them
    const int live = __builtin_amdgcn_readfirstlane((min(a.n - m0, L::BM) - 16 * wm + 16 * L::WM - 1) / (16 * L::WM));
    if (nch > 0) open(0);
    for (int c = 0; c < nch; c++) {
        const uint8_t* st = smem + (c % L::NS) * L::STAGE;
        const bool rest = c > 0 && c - 1 + L::NS < full;          // of the stage that the last barrier freed
#pragma unroll
        for (int i = 0; i < MI - 1; i++) {
            if (i + 1 < GROUPS && rest) copy(c - 1 + L::NS, PER * (i + 1), PER);
            if (D < MI && i + D - 1 < MI && (!L::RAGGED || i + D - 1 < live)) read_a(st, i + D - 1);
            if (!L::RAGGED || i < live) row(i);
        }
        // Every operand of the chunk is in registers: the barrier frees its slot and makes the
        // next chunk whole (only later ones' copies are then out).
        if (c + 1 < nch) {
            if (c + L::NS <= nch) wait_vm<L::OPS * (L::NS - 2)>();
            else wait_vm<0>();
            __syncthreads();
            if (c + L::NS < full) copy(c + L::NS, 0, PER);
            else if (c + L::NS < nch) copy_all(c + L::NS);
        }
        if (!L::RAGGED || MI - 1 < live) row(MI - 1);
        if (c + 1 < nch) open(c + 1);
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// A matrix that takes a tile's sums
// ---------------------------------------------------------------------------
struct MmOut {
    void* c;                 // element (m, n) at c[m * ldc + n], m < M, n < N
    int64_t ldc;
    int M, N;
    int bf16, accumulate;    // accumulate: what c holds + the sum, in fp32, rounded once
};

// A wave's sums to C from (m0, n0), its row tiles STEP apart, 16 rows at a time through LDS
// (two buffers of 16 rows): a lane's four columns become 16-byte stores along the rows.
// Segments are XOR-swizzled by the row.  S: the type staged, fp32 where C is added to.
template <bool STREAM, int STEP, int MI, int NI, typename S, typename T>
__device__ __forceinline__ void mm_store(const v4f (&acc)[MI][NI], uint8_t* stage, const MmOut& o, int m0, int n0)
{
    constexpr int ES = sizeof(S), RB = NI * 16 * ES, LR = RB / 16, PER = 16 / ES;
    constexpr int RP = 64 / LR;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kq = lane >> 4;
#pragma unroll
    for (int i = 0; i < MI; i++) {
        if (m0 + 16 * STEP * i >= o.M) break;
        uint8_t* buf = stage + (i & 1) * (16 * NI * 16 * 4);
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int at = (16 * j + 4 * kq) * ES;
            uint8_t* d = buf + r16 * RB + (((at >> 4) ^ (r16 & (LR - 1))) << 4) + (at & 15);
            if constexpr (ES == 2)
                *reinterpret_cast<uint2*>(d) =
                    make_uint2(bf16x2(acc[i][j][0], acc[i][j][1]), bf16x2(acc[i][j][2], acc[i][j][3]));
            else
                *reinterpret_cast<float4*>(d) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 16; q += RP) {
            const int r = q + lane / LR, sg = lane % LR;
            if (r >= 16) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * RB + ((sg ^ (r & (LR - 1))) << 4));
            const int m = m0 + 16 * STEP * i + r, n = n0 + sg * PER;
            if (m >= o.M || n >= o.N) continue;
            T* c = static_cast<T*>(o.c) + (int64_t)m * o.ldc + n;
            if constexpr (sizeof(S) == sizeof(T)) {
                if (n + PER <= o.N && !o.accumulate) {
                    const v4u32 w4 = {v.x, v.y, v.z, v.w};
                    if (STREAM) __builtin_nontemporal_store(w4, reinterpret_cast<v4u32_any*>(c));
                    else *reinterpret_cast<v4u32_any*>(c) = w4;
                    continue;
                }
            }
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if constexpr (ES == 4) {
                if (n + PER <= o.N) {                  // added to, four at a time
                    const float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
                    if constexpr (sizeof(T) == 4) {
                        v4u32 b = *reinterpret_cast<const v4u32_any*>(c);
#pragma unroll
                        for (int e = 0; e < 4; e++) b[e] = __float_as_uint(__uint_as_float(b[e]) + f[e]);
                        *reinterpret_cast<v4u32_any*>(c) = b;
                    } else {
                        const v2u32 b = *reinterpret_cast<const v2u32_any*>(c);
                        *reinterpret_cast<v2u32_any*>(c) =
                            v2u32{bf16x2(bf16_to_f32(b[0] & 0xFFFFu) + f[0], bf16_to_f32(b[0] >> 16) + f[1]),
                                  bf16x2(bf16_to_f32(b[1] & 0xFFFFu) + f[2], bf16_to_f32(b[1] >> 16) + f[3])};
                    }
                    continue;
                }
            }
#pragma unroll
            for (int e = 0; e < PER; e++) {
                if (n + e >= o.N) break;
                if constexpr (ES == 2) c[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                else if constexpr (sizeof(T) == 2) c[e] = (uint16_t)bf16x2(bf16_to_f32(c[e]) + __uint_as_float(w[e]), 0.0f);
                else c[e] = o.accumulate ? c[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ... of a block's tile.  STREAM: past the caches, for what nothing reads soon.
template <class L, bool STREAM = (L::BM * L::BN >= 128 * 128)>
__device__ __forceinline__ void mm_store_tile(const v4f (&acc)[L::MI][L::NI], uint8_t* smem, const MmOut& o, int m0, int n0)
{
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    uint8_t* stage = smem + wave * L::C_BYTES;
    const int mw = m0 + L::first_row(wave / L::WN), nw = n0 + wave % L::WN * L::NI * 16;
    if (!o.bf16) mm_store<STREAM, L::STEP, L::MI, L::NI, float, float>(acc, stage, o, mw, nw);
    else if (o.accumulate) mm_store<STREAM, L::STEP, L::MI, L::NI, float, uint16_t>(acc, stage, o, mw, nw);
    else mm_store<STREAM, L::STEP, L::MI, L::NI, uint16_t, uint16_t>(acc, stage, o, mw, nw);
}

// The tile of a block's turn.  Blocks go to the eight XCDs in turn: XCD x takes the x-th
// eighth of n tiles, so that tiles that follow each other share operands in its L2.
__device__ __forceinline__ int mm_turn(int block, int n)
{
    const int x = block & 7, i = block >> 3, each = n >> 3, rest = n & 7;
    return i < each + (x < rest) ? x * each + min(x, rest) + i : -1;
}

// Tile `tile` of tm x tn, column by column in bands of eight row tiles: those that run
// together share rows of both operands.
__device__ __forceinline__ void mm_band(int tile, int tm, int tn, int& im, int& in)
{
    const int band = tile / (8 * tn), rows = min(8, tm - band * 8), inside = tile - band * 8 * tn;
    im = band * 8 + inside % rows;
    in = inside / rows;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
inline int64_t over(int64_t n, int64_t b) { return (n + b - 1) / b; }

// Sizes and leading dimensions of operands: a tile's 256 rows of this many elements stay below 2^31 bytes.
constexpr int64_t kMaxSide = 1 << 22;
inline bool side_ok(int64_t n) { return n >= 0 && n <= kMaxSide; }

// An operand that mm_tile reads in place: rows that begin at 16 bytes and are whole segments.
inline bool in_place(const void* p, int64_t cols, int64_t ld) { return aligned_to(p, 16) && cols % 8 == 0 && ld % 8 == 0; }

// bf16 rows [R][ld] of an operand, C used
inline int check_rows(const void* p, int64_t R, int64_t C, int64_t ld)
{
    if (ld < C || ld > kMaxSide) return V4MOE_EDIMS;
    if (R > 0 && !p) return V4MOE_ENULL;
    return aligned_to(p, 2) ? V4MOE_OK : V4MOE_EALIGN;
}
// an output [R][ld] of a type, C used
inline int check_out(const void* p, int32_t type, int64_t R, int64_t C, int64_t ld)
{
    if ((type != V4MOE_TYPE_F32 && type != V4MOE_TYPE_BF16) || ld < C || ld > (1ll << 40)) return V4MOE_EDIMS;
    if (R > 0 && !p) return V4MOE_ENULL;
    return aligned_to(p, type == V4MOE_TYPE_F32 ? 4 : 2) ? V4MOE_OK : V4MOE_EALIGN;
}

// Rows of bf16, src [R][ld] -> dst [R][C8] (C8 = C rounded up to 8), zeros past C: for operands that cannot be read
// in place.  Up to three of them in one launch.
struct PadRows {
    int64_t R;
    int C;
    const uint16_t* src; int64_t ld;
    uint16_t* dst;
};
hipError_t launch_pad_rows(const PadRows* jobs, int n, hipStream_t s);

// The tiles of a product.  A call takes the one of the least time in this table, by the rounds its tiles make (a
// round is one tile per CU): microseconds for 1 to 4 rounds at contractions of 256 and of 4096, between and beyond
// which times are nearly linear, in a graph of many calls (rows by rows; columns are within a few percent).
//                        K = 256                       K = 4096
//   16x64      4.2    4.7    5.4    5.9      15.1   18.8   26.9   33.5
//   32x64      4.3    5.0    5.7    7.8      18.4   23.5   31.7   41.7
//   64x64      4.9    5.9    6.9    9.6      23.6   32.0   43.9   55.2
//   128x128    7.2    8.9   13.7   16.2      47.5   65.6  106.7  121.9
//   256x256   15.3   32.6   41.0   59.9     107.7  206.0  300.5  394.1
// (128x256 and 256x128 of eight waves, 9.8 to 32 and 66 to 237, lie between the last two and are never the least by more
// than a few percent; 64x256 of four waves takes 51 / 73 / 115 / 136.)
struct MmVariant {
    int bm, bn;
    float us256[4], us4096[4];
};
constexpr MmVariant kMmVariants[] = {{16, 64, {4.2f, 4.7f, 5.4f, 5.9f}, {15.1f, 18.8f, 26.9f, 33.5f}},
                                     {32, 64, {4.3f, 5.0f, 5.7f, 7.8f}, {18.4f, 23.5f, 31.7f, 41.7f}},
                                     {64, 64, {4.9f, 5.9f, 6.9f, 9.6f}, {23.6f, 32.0f, 43.9f, 55.2f}},
                                     {128, 128, {7.2f, 8.9f, 13.7f, 16.2f}, {47.5f, 65.6f, 106.7f, 121.9f}},
                                     {256, 256, {15.3f, 32.6f, 41.0f, 59.9f}, {107.7f, 206.0f, 300.5f, 394.1f}}};
inline int32_t tile_code(const MmVariant& v) { return v.bm << 16 | v.bn; }
inline float mm_time(const MmVariant& v, int64_t tiles, int64_t K)
{
    const int64_t rounds = tiles < 1 ? 1 : (tiles + 255) / 256;
    const int r = rounds < 4 ? (int)rounds - 1 : 3;
    const float us = v.us256[r] + (v.us4096[r] - v.us256[r]) * (float)(K - 256) / 3840.0f;
    return rounds <= 4 ? us : us * (float)rounds / 4.0f;
}
// first: the smallest variant that may be taken; tiles(bm, bn): of the product
template <typename F>
int mm_choose(int first, int64_t K, F&& tiles)
{
    int best = first;
    float least = 0.0f;
    for (int v = first; v < 5; v++) {
        const float us = mm_time(kMmVariants[v], tiles(kMmVariants[v].bm, kMmVariants[v].bn), K);
        if (v == first || us < least) best = v, least = us;
    }
    return best;
}

// Lets a kernel have more than 64 KiB of LDS, once per device (or again by host threads that come to it at once).
using LdsAllowed = std::atomic<bool>[kMaxDevices];
inline hipError_t allow_lds(const void* kernel, int bytes, LdsAllowed& done)
{
    if (bytes <= 65536) return hipSuccess;
    int dev = 0;
    if (const hipError_t e = hipGetDevice(&dev); e != hipSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace v4moe
