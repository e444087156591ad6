// v4moe_lora.hip -- low-rank adapters of many requests beside a shared projection.
//
//   a = ids[m];  u[m] = scale[a] A[a] x[m]   (A [L][r][K]);  out[m] = y[m] + B[a]^T u[m]   (B [L][r][N])
//   dU[m] = scale[a] B[a] dy[m];  dx[m] = base[m] + A[a]^T dU[m]
//   dA[a] = sum over a's rows of dU[m] x[m]^T;  dB[a] = sum of u[m] dy[m]^T
//
// Both factors have the rank first, so that forward and backward are made of the same
// three products: rows by a factor (shrink), the result by a factor (expand), and sums
// over an adapter's rows (outer).  Rows of one adapter need not follow each other: a
// tile of rows is computed once for each adapter among its rows, and a row takes its own.
//
// u and dU pass between the products as two bf16 numbers, u rounded and what that leaves:
// 16 bits of significand, so that the results are as good as with fp32 (one bf16 number
// would add an error of the size of the results' own rounding).
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"
#include "v4moe_mm.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace v4moe {

namespace {

constexpr int kSlice = 256;      // of a shrink's contraction: one chain of matrix instructions; slices are added in order

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

// The adapters among a tile's rows, one after the other, in the order of their first rows:
// f(a, mask of a's rows) for every `slots`-th of them from `slot` on.  id: lane l's is row
// l's, negative for none.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int slot, int slots, F&& f)
{
    uint64_t left = __ballot(id >= 0);
    for (int i = 0; left != 0; i++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t rows = __ballot(id == a);
        if (i % slots == slot) f(a, rows);
        left &= ~rows;
    }
}
__device__ __forceinline__ int adapter_of(const int32_t* ids, int m, int M, int L)
{
    const int id = m < M ? ids[m] : -1;
    return id >= 0 && id < L ? id : -1;
}

struct ShrinkJob {
    const uint16_t* x; int64_t ldx; int K;     // rows
    const uint16_t* f;                         // factor [L][r][K]
    uint16_t* u;                               // [M][2][rp]
};
struct ShrinkArgs {
    int M, L, r, rp;
    const int32_t* ids; const float* scale;
    ShrinkJob job[2];
};

// u of 16 MI rows and 16 NJ ranks per block: the waves take the slices of the contraction
// in turn, operands straight from memory into registers (each is used once per wave), and
// the slices meet in LDS.  grid: row tiles, slots of the tile's adapters, rank chunks x jobs.
template <int MI, int NJ, int NW>
__global__ __launch_bounds__(64 * NW) void k_lora_shrink(ShrinkArgs p, int chunks)
{
    constexpr int LD = 16 * NJ + 4, QUADS = 16 * MI * 4 * NJ, PER = (QUADS + 64 * NW - 1) / (64 * NW);
    extern __shared__ __align__(16) float part[];            // [NW][16 MI][LD]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const ShrinkJob& job = p.job[blockIdx.z / chunks];
    const int m0 = blockIdx.x * 16 * MI, j0 = (int)(blockIdx.z % chunks) * 16 * NJ, K = job.K;
    const uint16_t* xrow[MI];
#pragma unroll
    for (int i = 0; i < MI; i++) xrow[i] = job.x + (int64_t)min(m0 + 16 * i + r16, p.M - 1) * job.ldx + 8 * kq;
    const int id = lane < 16 * MI ? adapter_of(p.ids, m0 + lane, p.M, p.L) : -1;
    each_adapter(id, blockIdx.y, gridDim.y, [&](int a, uint64_t rows) {
        const uint16_t* frow[NJ];
#pragma unroll
        for (int j = 0; j < NJ; j++) frow[j] = job.f + ((int64_t)a * p.r + min(j0 + 16 * j + r16, p.r - 1)) * K + 8 * kq;
        float4 sum[PER];
#pragma unroll
        for (int q = 0; q < PER; q++) sum[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < K; k0 += NW * kSlice) {
            const int k1 = k0 + wave * kSlice;
            if (k1 < K) {
                v4f acc[MI][NJ];
#pragma unroll
                for (int i = 0; i < MI; i++)
#pragma unroll
                    for (int j = 0; j < NJ; j++) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                auto products = [&](const v4u32 (&x)[MI], const v4u32 (&f)[NJ]) {
#pragma unroll
                    for (int i = 0; i < MI; i++)
#pragma unroll
                        for (int j = 0; j < NJ; j++)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(v8bf, f[j]), __builtin_bit_cast(v8bf, x[i]), acc[i][j], 0, 0, 0);
                };
                if (k1 + kSlice <= K) {
                    constexpr int AHEAD = NJ * MI <= 2 ? 8 : 4;      // steps whose operands are loaded together
#pragma unroll
                    for (int s0 = 0; s0 < kSlice / 32; s0 += AHEAD) {
                        v4u32 x[AHEAD][MI], f[AHEAD][NJ];
#pragma unroll
                        for (int s = 0; s < AHEAD; s++) {
#pragma unroll
                            for (int i = 0; i < MI; i++)
                                x[s][i] = *reinterpret_cast<const v4u32_any*>(xrow[i] + k1 + 32 * (s0 + s));
#pragma unroll
                            for (int j = 0; j < NJ; j++)
                                f[s][j] = *reinterpret_cast<const v4u32_any*>(frow[j] + k1 + 32 * (s0 + s));
                        }
#pragma unroll
                        for (int s = 0; s < AHEAD; s++) products(x[s], f[s]);
                    }
                } else {
                    for (int k = k1; k < K; k += 32) {
                        v4u32 x[MI], f[NJ];
#pragma unroll
                        for (int i = 0; i < MI; i++) x[i] = load8(xrow[i], k, K - 8 * kq);
#pragma unroll
                        for (int j = 0; j < NJ; j++) f[j] = load8(frow[j], k, K - 8 * kq);
                        products(x, f);
                    }
                }
                float* to = part + wave * 16 * MI * LD;
#pragma unroll
                for (int i = 0; i < MI; i++)
#pragma unroll
                    for (int j = 0; j < NJ; j++)
                        *reinterpret_cast<float4*>(to + (16 * i + r16) * LD + 16 * j + 4 * kq) =
                            make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            }
            __syncthreads();
            const int slices = min(NW, (K - k0 + kSlice - 1) / kSlice);
#pragma unroll
            for (int q = 0; q < PER; q++) {
                const int at = tid + q * 64 * NW;
                if (at < QUADS) {
                    const float* from = part + at / (4 * NJ) * LD + at % (4 * NJ) * 4;
                    for (int w = 0; w < slices; w++) {
                        const float4 v = *reinterpret_cast<const float4*>(from + w * 16 * MI * LD);
                        sum[q].x += v.x;
                        sum[q].y += v.y;
                        sum[q].z += v.z;
                        sum[q].w += v.w;
                    }
                }
            }
            __syncthreads();
        }
        const float scale = p.scale[a];
#pragma unroll
        for (int q = 0; q < PER; q++) {
            const int at = tid + q * 64 * NW, row = at / (4 * NJ), j = j0 + at % (4 * NJ) * 4;
            if (at < QUADS && (rows >> row & 1) && j < p.rp) {
                const float s[4] = {sum[q].x, sum[q].y, sum[q].z, sum[q].w};
                float hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float v = j + e < p.r ? s[e] * scale : 0.0f;
                    hi[e] = bf16_to_f32(bf16x2(v, 0.0f) & 0xFFFFu);
                    lo[e] = fabsf(hi[e]) < INFINITY ? v - hi[e] : 0.0f;     // (infinities and NaN stand alone)
                }
                uint16_t* u = job.u + (int64_t)(m0 + row) * 2 * p.rp + j;
                *reinterpret_cast<uint2*>(u) = make_uint2(bf16x2(hi[0], hi[1]), bf16x2(hi[2], hi[3]));
                *reinterpret_cast<uint2*>(u + p.rp) = make_uint2(bf16x2(lo[0], lo[1]), bf16x2(lo[2], lo[3]));
            }
        }
    });
}

struct ExpandArgs {
    int M, N, L, r, rp;
    const int32_t* ids;
    const uint16_t* u;                          // [M][2][rp]
    const uint16_t* f;                          // factor [L][r][N]
    const void* y; int64_t ldy;                 // added to (null: zeros)
    void* out; int64_t ldo;
    int tiles;                                  // 16-row tiles per wave
    int in_place;                               // out is y: rows without an adapter are there already
};

// Sixteen values of a row from column n on, as fp32; past N zeros.
template <typename T>
__device__ __forceinline__ void load16f(const T* row, int n, int N, float (&v)[16])
{
    if constexpr (sizeof(T) == 4) {
        if (n + 16 <= N) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const v4u32 w = *reinterpret_cast<const v4u32_any*>(row + n + 4 * q);
#pragma unroll
                for (int e = 0; e < 4; e++) v[4 * q + e] = __uint_as_float(w[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; e++) v[e] = n + e < N ? row[n + e] : 0.0f;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const v4u32 w = load8(row, n + 8 * q, N);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v[8 * q + 2 * e] = bf16_to_f32(w[e] & 0xFFFFu);
                v[8 * q + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
    }
}
template <typename T>
__device__ __forceinline__ void store16f(T* row, int n, int N, const float (&v)[16])
{
    if constexpr (sizeof(T) == 4) {
        if (n + 16 <= N) {
#pragma unroll
            for (int q = 0; q < 4; q++)
                *reinterpret_cast<v4u32_any*>(row + n + 4 * q) =
                    v4u32{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                          __float_as_uint(v[4 * q + 3])};
        } else {
#pragma unroll
            for (int e = 0; e < 16; e++)
                if (n + e < N) row[n + e] = v[e];
        }
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = bf16x2(v[2 * e], v[2 * e + 1]);
        if (n + 16 <= N) {
            *reinterpret_cast<v4u32_any*>(row + n) = v4u32{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<v4u32_any*>(row + n + 8) = v4u32{w[4], w[5], w[6], w[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 16; e++)
                if (n + e < N) row[n + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// A wave: 64 columns of `tiles` 16-row tiles.  The factor's 16 RC ranks by 64 columns pass
// through LDS, where transposing reads make operands of them that stay in registers while
// the adapter lasts.  A step of the contraction is 16 ranks twice, by u and by what its
// rounding left.  Columns are dealt so that a lane ends with 16 consecutive ones: of the
// instruction's column i of tile t it is 16 (i / 4) + 4 t + i % 4.
template <int RC, typename T>
__global__ __launch_bounds__(256) void k_lora_expand(ExpandArgs p)
{
    __shared__ __align__(128) uint8_t lds[4][16 * RC * 128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int c0 = ((int)blockIdx.x * 4 + wave) * 64;
    if (c0 >= p.N) return;                                    // (no barrier below: waves are on their own)
    uint8_t* mine = lds[wave];
    v8bf bf[RC][4];
    int staged = -1, staged_j = -1;
    // ranks j0 .. of adapter a into the operands
    auto stage = [&](int a, int j0) {
        if (a == staged && j0 == staged_j) return;
        staged = a;
        staged_j = j0;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 2 * RC; q++) {
            const int j = 8 * q + (lane >> 3), s = lane & 7;
            v4u32 v = {0u, 0u, 0u, 0u};
            if (j0 + j < p.r && c0 + 8 * s < p.N) v = load8(p.f + ((int64_t)a * p.r + j0 + j) * p.N, c0 + 8 * s, p.N);
            // the segment's halves: columns 16 (s / 2) + 4 t + 0 .. 3 for t = 2 (s % 2), + 1
            const int f = column_swizzle<64>(j);
#pragma unroll
            for (int h = 0; h < 2; h++)
                *reinterpret_cast<uint2*>(mine + j * 128 + ((2 * (s & 1) + h) ^ f) * 32 + (s >> 1) * 8) =
                    make_uint2(v[2 * h], v[2 * h + 1]);
        }
        __builtin_amdgcn_wave_barrier();
        MmReader<64, true, 4> reader;
        reader.begin_at(0, lane, 8 * (kq & 1));
#pragma unroll
        for (int c = 0; c < RC; c++)
#pragma unroll
            for (int t = 0; t < 4; t++) bf[c][t] = reader.read_at(mine, t, 16 * c);
    };
    for (int i = 0; i < p.tiles; i++) {
        const int m0 = ((int)blockIdx.y * p.tiles + i) * 16, m = m0 + r16;
        if (m0 >= p.M) return;
        const int id = adapter_of(p.ids, m, p.M, p.L);
        const int n = c0 + 16 * kq;
        const bool real = m < p.M && n < p.N;
        const T* yrow = static_cast<const T*>(p.y) + (int64_t)min(m, p.M - 1) * p.ldy;
        T* orow = static_cast<T*>(p.out) + (int64_t)min(m, p.M - 1) * p.ldo;
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; e++) y[e] = 0.0f;
        if (p.y && real) load16f(yrow, n, p.N, y);
        if (blockIdx.z == 0 && real && id < 0 && !p.in_place) store16f(orow, n, p.N, y);
        const uint16_t* urow = p.u + (int64_t)min(m, p.M - 1) * 2 * p.rp + (kq >> 1) * p.rp + 8 * (kq & 1);
        each_adapter(lane < 16 ? id : -1, blockIdx.z, gridDim.z, [&](int a, uint64_t) {
            v4f acc[4];
#pragma unroll
            for (int t = 0; t < 4; t++) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            for (int j0 = 0; j0 < p.r; j0 += 16 * RC) {
                v4u32 u[RC];
#pragma unroll
                for (int c = 0; c < RC; c++) {
                    u[c] = v4u32{0u, 0u, 0u, 0u};
                    // (rows of other adapters, or none, give results that nobody takes)
                    if (id == a && j0 + 16 * c < p.rp) u[c] = *reinterpret_cast<const v4u32*>(urow + j0 + 16 * c);
                }
                stage(a, j0);
#pragma unroll
                for (int c = 0; c < RC; c++)
#pragma unroll
                    for (int t = 0; t < 4; t++)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[c][t], __builtin_bit_cast(v8bf, u[c]), acc[t], 0, 0, 0);
            }
            if (id == a && real) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; e++) v[e] = y[e] + acc[e >> 2][e & 3];
                store16f(orow, n, p.N, v);
            }
        });
    }
}

struct OuterJob {
    const uint16_t* u;                          // [M][2][rp]
    const uint16_t* x; int64_t ldx; int N;      // rows, columns
    void* d;                                    // [L][r][N]
    int bf16, blocks;                           // column blocks of 64
};
struct OuterArgs {
    int M, L, r, rp, accumulate;
    const int32_t* ids;
    OuterJob job[2];
};

// Sums over the rows of one adapter: 16 RC ranks by 64 columns per block.  The block lists
// the adapter's rows, 2048 rows at a time, in order; its waves take 32 of the list in turn,
// the next ones on their way while these are multiplied, and add up in the order of the waves.
constexpr int kOuterRows = 2048;
template <int RC>
__global__ __launch_bounds__(256) void k_lora_outer(OuterArgs p)
{
    constexpr int UW = 32 * RC, XB = 32 * 128, UB = 32 * UW * 2;          // ranks of a row (twice 16 RC), bytes of a step
    __shared__ __align__(128) uint8_t lds[4][XB + UB];
    __shared__ uint16_t list[kOuterRows];
    __shared__ int counts[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const bool second = (int)blockIdx.x >= p.job[0].blocks;
    const OuterJob& job = p.job[second];
    const int c0 = ((int)blockIdx.x - (second ? p.job[0].blocks : 0)) * 64, j0 = blockIdx.z * 16 * RC, a = blockIdx.y;
    uint8_t *xs = lds[wave], *us = lds[wave] + XB;
    v4f acc[RC][4];
#pragma unroll
    for (int c = 0; c < RC; c++)
#pragma unroll
        for (int t = 0; t < 4; t++) acc[c][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    MmReader<64, true, 4> rx;
    MmReader<UW, true, 2 * RC> ru;
    rx.begin(0, lane);
    ru.begin(0, lane);
    int any = 0;
    for (int seg = 0; seg < p.M; seg += kOuterRows) {
        // this segment's rows of the adapter: eight ids per thread
        uint32_t has = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int m = seg + 8 * tid + e;
            if (m < p.M && p.ids[m] == a) has |= 1u << e;
        }
        int scan = __popc(has);
        const int mine = scan;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(scan, o);
            if (lane >= o) scan += v;
        }
        __syncthreads();                     // (the list and the counts of the segment before are read)
        if (lane == 63) counts[wave] = scan;
        __syncthreads();
        int at = scan - mine, n = 0;
        for (int w = 0; w < 4; w++) {
            if (w < wave) at += counts[w];
            n += counts[w];
        }
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (has >> e & 1) list[at++] = (uint16_t)(8 * tid + e);
        __syncthreads();
        any |= n;
        // 32 rows of the list: columns and ranks into registers, zeros past its end
        v4u32 xv[4], uv[2 * RC];
        auto load = [&](int s) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int i = 32 * s + 8 * q + (lane >> 3), c = c0 + 8 * (lane & 7);
                xv[q] = v4u32{0u, 0u, 0u, 0u};
                if (i < n && c < job.N) xv[q] = load8(job.x + (int64_t)(seg + list[i]) * job.ldx, c, job.N);
            }
#pragma unroll
            for (int q = 0; q < 2 * RC; q++) {
                constexpr int SEGS = UW / 8;                       // of a row: half for u, half for what it left
                const int at = q * 64 + lane, i = 32 * s + at / SEGS, sg = at % SEGS;
                const int j = j0 + (sg % (SEGS / 2)) * 8;
                uv[q] = v4u32{0u, 0u, 0u, 0u};
                if (i < n && j < p.rp)
                    uv[q] = *reinterpret_cast<const v4u32*>(job.u + (int64_t)(seg + list[i]) * 2 * p.rp +
                                                            (sg / (SEGS / 2)) * p.rp + j);
            }
        };
        const int steps = (n + 31) / 32;
        if (wave < steps) load(wave);
        for (int s = wave; s < steps; s += 4) {
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int i = 8 * q + (lane >> 3);
                *reinterpret_cast<v4u32*>(xs + i * 128 + ((lane & 7) ^ (2 * column_swizzle<64>(i))) * 16) = xv[q];
            }
#pragma unroll
            for (int q = 0; q < 2 * RC; q++) {
                constexpr int SEGS = UW / 8;
                const int at = q * 64 + lane, i = at / SEGS;
                *reinterpret_cast<v4u32*>(us + i * UW * 2 + ((at % SEGS) ^ (2 * column_swizzle<UW>(i))) * 16) = uv[q];
            }
            if (s + 4 < steps) load(s + 4);
            __builtin_amdgcn_wave_barrier();
            v8bf xf[4];
#pragma unroll
            for (int t = 0; t < 4; t++) xf[t] = rx.read(xs, t, 0);
#pragma unroll
            for (int c = 0; c < 2 * RC; c++) {
                const v8bf uf = ru.read(us, c, 0);
#pragma unroll
                for (int t = 0; t < 4; t++)
                    acc[c % RC][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[t], uf, acc[c % RC][t], 0, 0, 0);
            }
        }
    }
    if (any == 0 && p.accumulate) return;          // (adding a sum of nothing would turn -0 into 0)
    // lane: rank 16 c + r16, columns 16 t + 4 kq .. + 3
    float* sums = reinterpret_cast<float*>(lds);
    static_assert(sizeof(lds) >= 16 * RC * 64 * 4, "the sums fit");
    for (int w = 0; w < 4; w++) {
        __syncthreads();
        if (wave == w) {
#pragma unroll
            for (int c = 0; c < RC; c++)
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    float4* to = reinterpret_cast<float4*>(sums + (16 * c + r16) * 64 + 16 * t + 4 * kq);
                    float4 v = make_float4(acc[c][t][0], acc[c][t][1], acc[c][t][2], acc[c][t][3]);
                    if (w > 0) {
                        const float4 b = *to;
                        v = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
                    }
                    *to = v;
                }
        }
    }
    __syncthreads();
    for (int i = tid; i < 16 * RC * 64; i += 256) {
        const int j = j0 + i / 64, c = c0 + i % 64;
        if (j >= p.r || c >= job.N) continue;
        const int64_t to = ((int64_t)a * p.r + j) * job.N + c;
        if (job.bf16) {
            uint16_t* d = static_cast<uint16_t*>(job.d) + to;
            *d = (uint16_t)bf16x2(p.accumulate ? bf16_to_f32(*d) + sums[i] : sums[i], 0.0f);
        } else {
            float* d = static_cast<float*>(job.d) + to;
            *d = p.accumulate ? *d + sums[i] : sums[i];
        }
    }
}

// ---- host ----
template <int MI, int NJ, int NW>
hipError_t launch_shrink(const ShrinkArgs& p, int jobs, int slots, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_lora_shrink<MI, NJ, NW>;
    constexpr int BYTES = NW * 16 * MI * (16 * NJ + 4) * 4;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), BYTES, allowed); e != hipSuccess) return e;
    const int chunks = (int)over(p.r, 16 * NJ);
    hipLaunchKernelGGL(kernel, dim3((unsigned)over(p.M, 16 * MI), (unsigned)slots, (unsigned)(chunks * jobs)), dim3(64 * NW),
                       BYTES, s, p, chunks);
    return hipGetLastError();
}
// Blocks for a tile's adapters: one where there are tiles enough, up to one each where there are few.
int slots_of(int64_t blocks, int rows) { return (int)std::max<int64_t>(1, std::min<int64_t>(rows, 1024 / blocks)); }
hipError_t run_shrink(const ShrinkArgs& p, int jobs, hipStream_t s)
{
    if (p.M <= 2048) {
        const int slots = slots_of(over(p.M, 16), 16);
        if (p.r <= 16) return launch_shrink<1, 1, 16>(p, jobs, slots, s);
        if (p.r <= 32) return launch_shrink<1, 2, 16>(p, jobs, slots, s);
        return launch_shrink<1, 4, 16>(p, jobs, slots, s);
    }
    const int slots = slots_of(over(p.M, 32), 32);
    if (p.r <= 16) return launch_shrink<2, 1, 8>(p, jobs, slots, s);
    if (p.r <= 32) return launch_shrink<2, 2, 8>(p, jobs, slots, s);
    return launch_shrink<2, 4, 8>(p, jobs, slots, s);
}

template <int RC>
hipError_t launch_expand(ExpandArgs p, int bf16, hipStream_t s)
{
    const int64_t columns = over(p.N, 256), rows = over(p.M, 16);
    const int64_t waves = columns * 4 * rows;
    // some 8192 waves at least: a few tiles each where there are more, several for a tile's adapters where there are fewer
    p.tiles = (int)std::max<int64_t>(over(rows, 65535), std::min<int64_t>(4, std::max<int64_t>(1, waves / 8192)));
    const int slots = (int)std::max<int64_t>(1, std::min<int64_t>(16, 8192 / waves));
    const dim3 grid((unsigned)columns, (unsigned)over(rows, p.tiles), (unsigned)slots);
    if (bf16) hipLaunchKernelGGL((k_lora_expand<RC, uint16_t>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_lora_expand<RC, float>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t run_expand(const ExpandArgs& p, int bf16, hipStream_t s)
{
    if (p.r <= 16) return launch_expand<1>(p, bf16, s);
    if (p.r <= 32) return launch_expand<2>(p, bf16, s);
    return launch_expand<4>(p, bf16, s);
}

template <int RC>
hipError_t launch_outer(const OuterArgs& p, hipStream_t s)
{
    hipLaunchKernelGGL(k_lora_outer<RC>, dim3((unsigned)(p.job[0].blocks + p.job[1].blocks), (unsigned)p.L,
                                              (unsigned)over(p.r, 16 * RC)), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t run_outer(const OuterArgs& p, hipStream_t s)
{
    if (p.r <= 16) return launch_outer<1>(p, s);
    if (p.r <= 32) return launch_outer<2>(p, s);
    return launch_outer<4>(p, s);
}

int ranks(int r) { return (r + 15) / 16 * 16; }
size_t lora_u(int64_t M, int r) { return up256((size_t)(M * 2 * ranks(r) * 2)); }

int check_lora(const v4moe_lora* p)
{
    if (!p) return V4MOE_ENULL;
    if (!side_ok(p->M) || !side_ok(p->N) || !side_ok(p->K) || p->N < 1 || p->K < 1) return V4MOE_EDIMS;
    if (p->r < 1 || p->r > 512 || p->L < 1 || p->L > 65535) return V4MOE_EDIMS;
    return V4MOE_OK;
}
int check_factors(const v4moe_lora* p, const uint16_t* a, const uint16_t* b, const int32_t* ids, const float* scale)
{
    if (!a || !b || !scale || (p->M > 0 && !ids)) return V4MOE_ENULL;
    if (!aligned_to(a, 2) || !aligned_to(b, 2) || !aligned_to(ids, 4) || !aligned_to(scale, 4)) return V4MOE_EALIGN;
    return V4MOE_OK;
}

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) size_t moe_lora_workspace_bytes(const v4moe_lora* p, int32_t backward)
{
    if (check_lora(p)) return 0;
    return lora_u(p->M, p->r) * (backward ? 2 : 1);
}

__attribute__((visibility("default"))) int moe_lora_add(const v4moe_lora* p, const void* y, int32_t type, int64_t ldy,
                                                        const uint16_t* x, int64_t ldx, const uint16_t* a,
                                                        const uint16_t* b, const int32_t* ids, const float* scale,
                                                        void* out, int64_t ldo, void* workspace, size_t ws_bytes,
                                                        void* stream)
{
    if (const int rc = check_lora(p)) return rc;
    if (const int rc = check_rows(x, p->M, p->K, ldx)) return rc;
    if (const int rc = check_out(y, type, p->M, p->N, ldy)) return rc;
    if (const int rc = check_out(out, type, p->M, p->N, ldo)) return rc;
    if (out == y && ldo != ldy) return V4MOE_EDIMS;
    if (const int rc = check_factors(p, a, b, ids, scale)) return rc;
    if (p->M == 0) return V4MOE_OK;
    if (!workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    if (ws_bytes < lora_u(p->M, p->r)) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t* u = static_cast<uint16_t*>(workspace);
    const int rp = ranks(p->r);
    const ShrinkArgs sh{p->M, p->L, p->r, rp, ids, scale, {{x, ldx, p->K, a, u}, {}}};
    if (run_shrink(sh, 1, s) != hipSuccess) return V4MOE_ELAUNCH;
    const ExpandArgs ex{p->M, p->N, p->L, p->r, rp, ids, u, b, y, ldy, out, ldo, 1, out == y};
    return run_expand(ex, type == V4MOE_TYPE_BF16, s) == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_lora_backward(
    const v4moe_lora* p, const uint16_t* x, int64_t ldx, const uint16_t* dy, int64_t lddy, const uint16_t* a,
    const uint16_t* b, const int32_t* ids, const float* scale, const void* base, int64_t ldbase, void* dx, int32_t dx_type,
    int64_t lddx, void* da, int32_t da_type, void* db, int32_t db_type, int32_t accumulate, void* workspace, size_t ws_bytes,
    void* stream)
{
    if (const int rc = check_lora(p)) return rc;
    if (!dx && !da && !db) return V4MOE_ENULL;
    if (da || db)
        if (const int rc = check_rows(x, p->M, p->K, ldx)) return rc;
    if (const int rc = check_rows(dy, p->M, p->N, lddy)) return rc;
    if (dx) {
        if (const int rc = check_out(dx, dx_type, p->M, p->K, lddx)) return rc;
        if (base)
            if (const int rc = check_out(base, dx_type, p->M, p->K, ldbase)) return rc;
        if (base == dx && ldbase != lddx) return V4MOE_EDIMS;
    }
    if (da)
        if (const int rc = check_out(da, da_type, 1, p->K, p->K)) return rc;
    if (db)
        if (const int rc = check_out(db, db_type, 1, p->N, p->N)) return rc;
    if (const int rc = check_factors(p, a, b, ids, scale)) return rc;
    if (p->M == 0 && ((!da && !db) || accumulate)) return V4MOE_OK;
    if (p->M > 0 && !workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    const size_t each = lora_u(p->M, p->r);
    if (ws_bytes < 2 * each) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t* du = static_cast<uint16_t*>(workspace);
    uint16_t* u = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + each);
    const int rp = ranks(p->r);
    if (p->M > 0) {
        ShrinkArgs sh{p->M, p->L, p->r, rp, ids, scale, {}};
        int jobs = 0;
        if (dx || da) sh.job[jobs++] = ShrinkJob{dy, lddy, p->N, b, du};
        if (db) sh.job[jobs++] = ShrinkJob{x, ldx, p->K, a, u};
        if (run_shrink(sh, jobs, s) != hipSuccess) return V4MOE_ELAUNCH;
    }
    if (dx && p->M > 0) {
        const ExpandArgs ex{p->M, p->K, p->L, p->r, rp, ids, du, a, base, ldbase, dx, lddx, 1, base == dx};
        if (run_expand(ex, dx_type == V4MOE_TYPE_BF16, s) != hipSuccess) return V4MOE_ELAUNCH;
    }
    if (da || db) {
        OuterArgs o{p->M, p->L, p->r, rp, accumulate != 0, ids, {}};
        int jobs = 0;
        if (da) o.job[jobs++] = OuterJob{du, x, ldx, p->K, da, da_type == V4MOE_TYPE_BF16, (int)over(p->K, 64)};
        if (db) o.job[jobs++] = OuterJob{u, dy, lddy, p->N, db, db_type == V4MOE_TYPE_BF16, (int)over(p->N, 64)};
        if (run_outer(o, s) != hipSuccess) return V4MOE_ELAUNCH;
    }
    return V4MOE_OK;
}

}  // extern "C"
