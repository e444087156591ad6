// v4moe_lora.hip -- low-rank adapters of many requests beside a shared projection.
//
//   a = ids[m];  u[m] = scale[a] A[a] x[m]   (A [L][r][K]);  out[m] = y[m] + B[a]^T u[m]   (B [L][r][N])
//   dU[m] = scale[a] B[a] dy[m];  dx[m] = base[m] + A[a]^T dU[m]
//   dA[a] = sum over a's rows of dU[m] x[m]^T;  dB[a] = sum of u[m] dy[m]^T
//
// Both factors have the rank first, so that forward and backward are made of the same
// three products: rows by a factor (shrink), the result by a factor (expand), and sums
// over an adapter's rows (outer).  Rows of one adapter need not follow each other.  Many
// rows are listed by adapter first, and tiles are made of the list.  Where there are few
// (a launch would cost more than it saves), tiles are of rows as they come, computed once
// for each adapter among them, and a row takes its own.
//
// u and dU pass between the products as two bf16 numbers, u rounded and what that leaves:
// 16 bits of significand, so that the results are as good as with fp32 (one bf16 number
// would add an error of the size of the results' own rounding).  (What an infinite element of the other operand makes of
// the two may be NaN where one product would be infinite.)
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"
#include "v4moe_mm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

namespace v4moe {

namespace {

// A shrink's contraction in slices, each one chain of matrix instructions; every fourth slice is added to the same of
// four sums, in order, and these are added in order.
constexpr int kSlice = 256, kSums = 4;

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

// Rows listed by adapter, those of one in ascending order, those without one last (as
// adapter L): order[p] is the row at place p, begin[a] .. begin[a + 1] adapter a's places,
// tiles the list in pieces of 64 places of one adapter.
constexpr int kTile = 64;
struct Tile { int a, first, count, unused; };
struct Listing {
    int* order;
    int* begin;                      // [L + 2]
    int* tiles_n;
    Tile* tiles;
};
constexpr int kListAdapters = 2048;  // of a pass: counters of sixteen waves fit LDS up to here
// One block.  Each wave counts its share of the rows, the counts become places (adapter by
// adapter, wave by wave), and the waves go through their rows again; rows of one adapter
// among a wave's 64 find each other by a ballot for each bit of the id.  More adapters than
// the counters hold take a pass over the rows for each 2048 of them.
// 8192 rows 9 us, 512 rows 7 (10 and 8 where one pass of at most 1024 were written as any number of them).
// MANY: passes of up to 2048 adapters, two a thread; otherwise one pass, an adapter a thread.
template <bool MANY>
__global__ __launch_bounds__(1024) void k_lora_list(int M, int L, const int32_t* __restrict__ ids, Listing out, int most)
{
    extern __shared__ int counts[];               // [16][n], then [n] first place, [n] first tile
    __shared__ int wave_rows[16], wave_tiles[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int share = (M + 1023) / 1024 * 64, m0 = wave * share, m1 = min(m0 + share, M);
    const bool once = share <= 512;                                 // then the places below the wave's first stay here
    int rows_done = 0, tiles_done = 0;
    for (int a0 = 0; MANY ? a0 <= L : a0 == 0; a0 += kListAdapters) {
        const int n = MANY ? min(L + 1 - a0, kListAdapters) : L + 1;            // adapters of this pass, "none" among the last
        int* begin = counts + 16 * n;
        int* first_tile = begin + n;
        for (int i = tid; i < 16 * n; i += 1024) counts[i] = 0;
        __syncthreads();
        int* mine = counts + wave * n;
        // 512 rows of the wave's share at a time, eight loads on their way together; of those past the share and of
        // other passes' adapters -1
        int id[8];
        auto load = [&](int base) {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int m = base + 64 * q + lane;
                id[q] = m < m1 ? ids[m] : -1;
            }
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int a = (id[q] >= 0 && id[q] < L ? id[q] : L) - a0;
                id[q] = base + 64 * q + lane < m1 && (!MANY || (a >= 0 && a < n)) ? a : -1;
            }
        };
        int bits = 0;
        while ((n - 1) >> bits) bits++;
        // id[q]'s place among those of its adapter that the wave has counted, which it then joins
        auto join = [&](int q) {
            const int a = max(id[q], 0);
            const bool in = id[q] >= 0;
            uint64_t same = __ballot(in);
            for (int b = 0; b < bits; b++) {
                const uint64_t ones = __ballot(a >> b & 1);
                same &= a >> b & 1 ? ones : ~ones;
            }
            const int at = in ? mine[a] + __popcll(same & ((1ull << lane) - 1)) : 0;
            __builtin_amdgcn_wave_barrier();
            if (in && (same >> lane >> 1) == 0) mine[a] += __popcll(same);       // (the last of them)
            __builtin_amdgcn_wave_barrier();
            return at;
        };
        int at[8];
        for (int base = m0; base < m1; base += 512) {
            load(base);
#pragma unroll
            for (int q = 0; q < 8; q++) at[q] = join(q);
        }
        __syncthreads();
        // a thread's adapters: one, or two that follow each other
        constexpr int EACH = MANY ? 2 : 1;
        const int first = tid * EACH, last = min(first + EACH, n);
        int rows = 0, tiles = 0;
        for (int a = first; a < last; a++) {
            int r = 0;
            for (int w = 0; w < 16; w++) r += counts[w * n + a];
            rows += r, tiles += (r + kTile - 1) / kTile;
        }
        int r = rows, t = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(r, o), v = __shfl_up(t, o);
            if (lane >= o) r += u, t += v;
        }
        if (lane == 63) wave_rows[wave] = r, wave_tiles[wave] = t;
        __syncthreads();
        int place = rows_done + r - rows, tile = tiles_done + t - tiles;
        for (int w = 0; w < 16; w++) {
            if (w < wave) place += wave_rows[w], tile += wave_tiles[w];
            rows_done += wave_rows[w], tiles_done += wave_tiles[w];
        }
        for (int a = first; a < last; a++) {
            begin[a] = place;
            first_tile[a] = tile;
            out.begin[a0 + a] = place;
            const int before = place;
            for (int w = 0; w < 16; w++) {
                const int c = counts[w * n + a];
                counts[w * n + a] = place;
                place += c;
            }
            tile += (place - before + kTile - 1) / kTile;
        }
        __syncthreads();
        for (int base = m0; base < m1; base += 512) {
            if (!once) load(base);
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int a = max(id[q], 0), p = once ? mine[a] + at[q] : join(q), off = p - begin[a];
                if (id[q] < 0) continue;
                out.order[p] = base + 64 * q + lane;
                if (off % kTile == 0) {
                    const int end = a + 1 < n ? begin[a + 1] : rows_done;
                    out.tiles[first_tile[a] + off / kTile] = Tile{a0 + a, p, min(kTile, end - p), 0};
                }
            }
        }
        if (MANY) __syncthreads();                                  // (the counts are read)
    }
    if (tid == 0) {
        out.begin[L + 1] = M;
        *out.tiles_n = tiles_done;
    }
    // no tiles behind the last
    for (int i = tiles_done + tid; i < most; i += 1024) out.tiles[i] = Tile{-1, 0, 0, 0};
}

struct ShrinkJob {
    const uint16_t* x; int64_t ldx; int K;     // rows
    const uint16_t* f;                         // factor [L][r][K]
    uint16_t* u;                               // [M][2][rp], by row, or by place
};
struct ShrinkArgs {
    int M, L, r, rp;
    const int32_t* ids; const float* scale;
    ShrinkJob job[2];
    Listing list;
};

// Two numbers for each of four sums: rounded to bf16, and what that leaves.
__device__ __forceinline__ void store_u(uint16_t* u, int rp, const float (&v)[4])
{
    float hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        hi[e] = bf16_to_f32(bf16x2(v[e], 0.0f) & 0xFFFFu);
        lo[e] = fabsf(hi[e]) < INFINITY ? v[e] - hi[e] : 0.0f;     // (infinities and NaN stand alone)
    }
    *reinterpret_cast<uint2*>(u) = make_uint2(bf16x2(hi[0], hi[1]), bf16x2(hi[2], hi[3]));
    *reinterpret_cast<uint2*>(u + rp) = make_uint2(bf16x2(lo[0], lo[1]), bf16x2(lo[2], lo[3]));
}

// u of 16 rows and 16 NJ ranks per block, of any alignment.  The sixteen waves take the slices
// of the contraction in turn, rows straight from memory into registers, the factor through a
// wave's own LDS (as the instruction wants its lanes, neighbours would read rows far apart, and
// the L1 takes a lane at a time: 64 rows with adapters of their own 12.0 us, so 7.6); the slices meet in LDS.
// grid: 16-row tiles, slots of the tile's adapters (LISTED: quarters of a tile), rank chunks x jobs.
constexpr int kShrinkWaves = 16, kShrinkRow = kSlice * 2 + 16;       // bytes of a staged row: 16 rows hit distinct banks
template <int NJ>
constexpr int shrink_room()          // the waves' staged rows, then the slices' products
{
    const int staged = kShrinkWaves * 16 * kShrinkRow, part = kShrinkWaves * 16 * (16 * NJ + 4) * 4;
    return staged > part ? staged : part;
}
template <int NJ>
constexpr int shrink_bytes() { return shrink_room<NJ>() + 16 * 16 * NJ * kSums * 4; }
template <int NJ, bool LISTED>
__global__ __launch_bounds__(64 * kShrinkWaves) void k_lora_shrink(ShrinkArgs p, int chunks)
{
    constexpr int NW = kShrinkWaves, LD = 16 * NJ + 4, QUADS = 16 * 4 * NJ;
    static_assert(QUADS <= 64 * NW, "a thread per four sums");
    static_assert(shrink_bytes<NJ>() <= 163840, "LDS of a CU");
    extern __shared__ __align__(16) uint8_t lds[];           // [NW][16][kShrinkRow], then [NW][16][LD] fp32; the sums
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const ShrinkJob& job = p.job[blockIdx.z / chunks];
    const int j0 = (int)(blockIdx.z % chunks) * 16 * NJ, K = job.K;
    const uint16_t* xrow;
    int first;                                               // row or place of the tile's first
    uint8_t* mine = lds + wave * 16 * kShrinkRow;
    float* part = reinterpret_cast<float*>(lds);
    auto work = [&](int a, uint64_t rows) {
        const float scale = p.scale[a];
        const bool has = rows >> r16 & 1;
        const uint16_t* factor = job.f + (int64_t)a * p.r * K;
        float4* sums = reinterpret_cast<float4*>(lds + shrink_room<NJ>()) + (tid < QUADS ? tid : 0) * kSums;   // this thread's
        if (tid < QUADS) {
#pragma unroll
            for (int w = 0; w < kSums; w++) sums[w] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        for (int k0 = 0; k0 < K; k0 += NW * kSlice) {
            const int k1 = k0 + wave * kSlice;
            v4f acc[NJ];
#pragma unroll
            for (int j = 0; j < NJ; j++) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if (k1 < K) {
                constexpr int STEPS = kSlice / 32;
                v4u32 x[STEPS], f[STEPS];
                auto load = [&](int j) {                     // 16 ranks, two of them an instruction
                    int half = lane >> 5;
                    asm volatile("" : "+v"(half));           // (addresses are made here: kept over the loop they would not fit the registers)
#pragma unroll
                    for (int s = 0; s < STEPS; s++) {
                        const int rank = j0 + 16 * j + 2 * s + half, k = k1 + 8 * (lane & 31);
                        f[s] = v4u32{0u, 0u, 0u, 0u};
                        if (rank < p.r && k < K) f[s] = load8(factor + (int64_t)rank * K, k, K);
                    }
                };
#pragma unroll
                for (int s = 0; s < STEPS; s++) {
                    x[s] = v4u32{0u, 0u, 0u, 0u};
                    if (has && k1 + 32 * s + 8 * kq < K) x[s] = load8(xrow, k1 + 32 * s + 8 * kq, K);
                }
                if (NJ == 1) load(0);
#pragma unroll
                for (int j = 0; j < NJ; j++) {
                    asm volatile("" ::: "memory");           // (loads of later ranks stay behind: registers)
                    if (NJ > 1) load(j);
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int s = 0; s < STEPS; s++)
                        *reinterpret_cast<v4u32*>(mine + (2 * s + (lane >> 5)) * kShrinkRow + (lane & 31) * 16) = f[s];
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int s = 0; s < STEPS; s++) {
                        const v8bf fv = *reinterpret_cast<const v8bf*>(mine + r16 * kShrinkRow + s * 64 + kq * 16);
                        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, __builtin_bit_cast(v8bf, x[s]), acc[j], 0, 0, 0);
                    }
                }
            }
            __syncthreads();                                 // (the staged rows are read)
            if (k1 < K) {
#pragma unroll
                for (int j = 0; j < NJ; j++)
                    *reinterpret_cast<float4*>(part + (wave * 16 + r16) * LD + 16 * j + 4 * kq) =
                        make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
            }
            __syncthreads();
            const int slices = min(NW, (K - k0 + kSlice - 1) / kSlice);
            if (tid < QUADS) {
                const float* from = part + tid / (4 * NJ) * LD + tid % (4 * NJ) * 4;
                static_assert(NW % kSums == 0, "a round's slices go on where the last one's ended");
                float4 sum[kSums];
#pragma unroll
                for (int w = 0; w < kSums; w++) sum[w] = sums[w];
#pragma unroll
                for (int w0 = 0; w0 < NW; w0 += kSums) {
                    float4 v[kSums];
#pragma unroll
                    for (int w = 0; w < kSums; w++)
                        v[w] = w0 + w < slices ? *reinterpret_cast<const float4*>(from + (w0 + w) * 16 * LD)
                                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kSums; w++) {
                        sum[w].x += v[w].x;
                        sum[w].y += v[w].y;
                        sum[w].z += v[w].z;
                        sum[w].w += v[w].w;
                    }
                }
#pragma unroll
                for (int w = 0; w < kSums; w++) sums[w] = sum[w];
            }
            __syncthreads();
        }
        const int row = tid / (4 * NJ), j = j0 + tid % (4 * NJ) * 4;
        if (tid < QUADS && (rows >> row & 1) && j < p.rp) {
            float4 s = sums[0];
#pragma unroll
            for (int w = 1; w < kSums; w++) {
                s.x += sums[w].x;
                s.y += sums[w].y;
                s.z += sums[w].z;
                s.w += sums[w].w;
            }
            const float v[4] = {s.x * scale, j + 1 < p.r ? s.y * scale : 0.0f, j + 2 < p.r ? s.z * scale : 0.0f,
                                j + 3 < p.r ? s.w * scale : 0.0f};
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            store_u(job.u + (int64_t)(first + row) * 2 * p.rp + j, p.rp, j < p.r ? v : zero);
        }
    };
    if constexpr (LISTED) {
        const Tile t = p.list.tiles[blockIdx.x];
        const int at = 16 * blockIdx.y, count = min(16, t.count - at);
        if (t.a >= p.L || count <= 0) return;
        first = t.first + at;
        xrow = job.x + (int64_t)p.list.order[first + min(r16, count - 1)] * job.ldx;
        work(t.a, (1ull << count) - 1);
    } else {
        first = blockIdx.x * 16;
        xrow = job.x + (int64_t)min(first + r16, p.M - 1) * job.ldx;
        each_adapter(lane < 16 ? adapter_of(p.ids, first + lane, p.M, p.L) : -1, blockIdx.y, gridDim.y, work);
    }
}

// u of a tile of the list and 16 NI ranks per block, rows that begin at 16 bytes.  Each of the four
// waves has every fourth slice: rows and factor pass through a ring of its own in LDS, 64 k a stage
// (whole lines of 128 bytes: halves are requests of their own, and as many of those fit the L1), so
// that nothing waits for another wave until the four sums meet.  8192 rows, K = 4096, rank 64, 16 adapters: 27 us,
// 2.8 TB/s: 145 blocks with 64 KiB each on their way.  As two blocks of 32 ranks each 28; 32-row tiles would read the
// factor, larger than the rows here, twice as often.
template <int NI, int NS>
struct ShrinkRing {
    static constexpr int MI = kTile / 16, AP = 2 * MI, BP = 2 * NI, OPS = AP + BP;     // 1 KiB pieces of a stage: 8 rows each
    static constexpr int B_OFF = AP * 1024, STAGE = OPS * 1024, RING = NS * STAGE, LD = 16 * NI + 4;
    static constexpr int SUMS = kSums * kTile * LD * 4, BYTES = kSums * RING > SUMS ? kSums * RING : SUMS;
    static_assert(OPS * (NS - 1) < 64 && NS >= 2 && BYTES <= 163840, "vmcnt range; LDS of a CU");
};
template <int NI, int NS>
__global__ __launch_bounds__(64 * kSums) void k_lora_shrink_ring(ShrinkArgs p, int chunks)
{
    using R = ShrinkRing<NI, NS>;
    constexpr int MI = R::MI;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int turn = mm_turn(blockIdx.x, *p.list.tiles_n);
    if (turn < 0) return;
    const Tile t = p.list.tiles[turn];
    if (t.a >= p.L) return;
    const ShrinkJob& job = p.job[blockIdx.z / chunks];
    const int j0 = (int)(blockIdx.z % chunks) * 16 * NI, K = job.K;
    const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem + wave * R::RING;
    // this lane's segments: row lane / 8 of each piece, segments as MmSide has them
    const int r8 = lane >> 3;
    auto segment = [&](int piece) { return (lane & 7) ^ (((piece * 8 + r8) >> 1) & 7); };
    const uint16_t *px[R::AP], *pf[R::BP];
#pragma unroll
    for (int i = 0; i < R::AP; i++)
        px[i] = job.x + (int64_t)p.list.order[t.first + min(8 * i + r8, t.count - 1)] * job.ldx + segment(i) * 8;
#pragma unroll
    for (int j = 0; j < R::BP; j++)
        pf[j] = job.f + ((int64_t)t.a * p.r + min(j0 + 8 * j + r8, p.r - 1)) * K + segment(j) * 8;
    // the wave's step q: 64 k of its slice q / PER
    constexpr int PER = kSlice / 64;
    auto begin_of = [&](int q) { return ((q / PER) * kSums + wave) * kSlice + q % PER * 64; };
    int steps = 0;
    for (int k = wave * kSlice; k < K; k += kSums * kSlice) steps += (min(K - k, kSlice) + 63) / 64;
    auto copy = [&](int q) {
        const int k = begin_of(q);
        const uint32_t to = ring0 + (uint32_t)(q % NS) * R::STAGE;
        auto one = [&](const uint16_t* from, int piece, uint32_t at) {
            const bool in = k + segment(piece) * 8 < K;           // (K a multiple of 8: whole segments)
            dma16(in ? (const void*)(from + k) : (const void*)&g_mm_zeros[lane], __builtin_amdgcn_readfirstlane(at));
        };
#pragma unroll
        for (int i = 0; i < R::AP; i++) one(px[i], i, to + i * 1024);
#pragma unroll
        for (int j = 0; j < R::BP; j++) one(pf[j], j, to + R::B_OFF + j * 1024);
    };
    const int r16 = lane & 15, kq = lane >> 4;
    MmReader<kTile, false, MI> ra;
    MmReader<16 * NI, false, NI> rb;
    ra.begin(0, lane);
    rb.begin(0, lane);
    v4f acc[MI][NI], sum[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++) acc[i][j] = sum[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < NS; q++)
        if (q < steps) copy(q);
    for (int q = 0; q < steps; q++) {
        // step q is whole once only later ones' copies are out
        if (q + NS <= steps) wait_vm<R::OPS * (NS - 1)>();
        else wait_vm<0>();
        asm volatile("" ::: "memory");
        const uint8_t* st = smem + wave * R::RING + (q % NS) * R::STAGE;
        v8bf a[2][MI], b[2][NI];
#pragma unroll
        for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int i = 0; i < MI; i++) a[s][i] = ra.read(st, i, s);
#pragma unroll
            for (int j = 0; j < NI; j++) b[s][j] = rb.read(st + R::B_OFF, j, s);
        }
        // the slot is free once its operands are in registers
        if (q + NS < steps) {
            __builtin_amdgcn_s_waitcnt(0xC07F);                   // lgkmcnt(0)
            asm volatile("" ::: "memory");
            copy(q + NS);
        }
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[s][j], a[s][i], acc[i][j], 0, 0, 0);
        if ((q + 1) % PER == 0 || q + 1 == steps) {
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                }
        }
    }
    __syncthreads();                                    // (every ring is read)
    float* sums = reinterpret_cast<float*>(smem);       // [kSums][kTile][LD]
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
            *reinterpret_cast<float4*>(sums + (wave * kTile + 16 * i + r16) * R::LD + 16 * j + 4 * kq) =
                make_float4(sum[i][j][0], sum[i][j][1], sum[i][j][2], sum[i][j][3]);
    __syncthreads();
    const float scale = p.scale[t.a];
#pragma unroll
    for (int q = 0; q < NI; q++) {
        const int at = q * 256 + tid, row = at / (4 * NI), k = at % (4 * NI) * 4;
        if (row >= t.count || j0 + k >= p.rp) continue;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kSums; w++) {
            const float4 f = *reinterpret_cast<const float4*>(sums + (w * kTile + row) * R::LD + k);
            v[0] = w ? v[0] + f.x : f.x;
            v[1] = w ? v[1] + f.y : f.y;
            v[2] = w ? v[2] + f.z : f.z;
            v[3] = w ? v[3] + f.w : f.w;
        }
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = j0 + k + e < p.r ? v[e] * scale : 0.0f;
        store_u(job.u + (int64_t)(t.first + row) * 2 * p.rp + j0 + k, p.rp, v);
    }
}

struct ExpandArgs {
    int M, N, L, r, rp;
    const int32_t* ids;
    const uint16_t* u;                          // [M][2][rp], by row, or by place
    const uint16_t* f;                          // factor [L][r][N]
    const void* y; int64_t ldy;                 // added to (null: zeros)
    void* out; int64_t ldo;
    int in_place;                               // out is y: rows without an adapter are there already
    Listing list;
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

// The factor's 16 RC ranks from j0 on by 64 columns from c0 on, adapter a, into registers, and from there
// into a wave's LDS, where transposing reads make operands of them.  Columns are dealt so that a lane ends with
// 16 consecutive ones: of the instruction's column i of tile t it is 16 (i / 4) + 4 t + i % 4.
template <int RC>
__device__ __forceinline__ void load_factor(const uint16_t* f, int a, int r, int j0, int c0, int N, v4u32 (&v)[2 * RC])
{
    const int lane = threadIdx.x & 63, s = lane & 7;
#pragma unroll
    for (int q = 0; q < 2 * RC; q++) {
        const int j = j0 + 8 * q + (lane >> 3);
        v[q] = v4u32{0u, 0u, 0u, 0u};
        if (j < r && c0 + 8 * s < N) v[q] = load8(f + ((int64_t)a * r + j) * N, c0 + 8 * s, N);
    }
}
template <int RC>
__device__ __forceinline__ void stage_factor(const v4u32 (&v)[2 * RC], uint8_t* to)
{
    const int lane = threadIdx.x & 63, s = lane & 7;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 2 * RC; q++) {
        const int j = 8 * q + (lane >> 3), swizzle = column_swizzle<64>(j);
        // the segment's halves: columns 16 (s / 2) + 4 t + 0 .. 3 for t = 2 (s % 2), + 1
#pragma unroll
        for (int h = 0; h < 2; h++)
            *reinterpret_cast<uint2*>(to + j * 128 + ((2 * (s & 1) + h) ^ swizzle) * 32 + (s >> 1) * 8) =
                make_uint2(v[q][2 * h], v[q][2 * h + 1]);
    }
    __builtin_amdgcn_wave_barrier();
}

// Few rows: a wave has 64 columns of a 16-row tile, once for each adapter among its rows.  A step of
// the contraction is 16 ranks twice, by u and by what its rounding left.  64 rows and adapters, N = 4096, rank 16: 6.5 us,
// a chain of loads (ids, u and factor, y).
template <int RC, typename T>
__global__ __launch_bounds__(256) void k_lora_expand(ExpandArgs p)
{
    __shared__ __align__(128) uint8_t lds[4][16 * RC * 128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int columns = (p.N + 255) / 256;                    // blocks along a row first
    const int c0 = ((int)(blockIdx.x % columns) * 4 + wave) * 64, n = c0 + 16 * kq;
    if (c0 >= p.N) return;                                    // (no barrier below: waves are on their own)
    uint8_t* mine = lds[wave];
    MmReader<64, true, 4> reader;
    reader.begin_at(0, lane, 8 * (kq & 1));
    const int m = (int)(blockIdx.x / columns) * 16 + r16, row = min(m, p.M - 1);
    const int id = adapter_of(p.ids, m, p.M, p.L);
    const bool real = m < p.M && n < p.N;
    const uint16_t* urow = p.u + ((int64_t)row * 2 + (kq >> 1)) * p.rp + 8 * (kq & 1);
    T* orow = static_cast<T*>(p.out) + (int64_t)row * p.ldo;
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; e++) y[e] = 0.0f;
    if (p.y && real) load16f(static_cast<const T*>(p.y) + (int64_t)row * p.ldy, n, p.N, y);
    if (blockIdx.y == 0 && real && id < 0 && !p.in_place) store16f(orow, n, p.N, y);
    each_adapter(lane < 16 ? id : -1, blockIdx.y, gridDim.y, [&](int a, uint64_t) {
        v4f acc[4];
#pragma unroll
        for (int t = 0; t < 4; t++) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int j0 = 0; j0 < p.r; j0 += 16 * RC) {
            v4u32 u[RC];
#pragma unroll
            for (int c = 0; c < RC; c++) {
                u[c] = v4u32{0u, 0u, 0u, 0u};
                // (rows of other adapters give results that nobody takes; a lane has its part of the contraction
                // where its columns are past the end, too)
                if (id == a && j0 + 16 * c < p.rp) u[c] = *reinterpret_cast<const v4u32*>(urow + j0 + 16 * c);
            }
            v4u32 f[2 * RC];
            load_factor<RC>(p.f, a, p.r, j0, c0, p.N, f);
            stage_factor<RC>(f, mine);
#pragma unroll
            for (int c = 0; c < RC; c++)
#pragma unroll
                for (int t = 0; t < 4; t++)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(reader.read_at(mine, t, 16 * c),
                                                                     __builtin_bit_cast(v8bf, u[c]), acc[t], 0, 0, 0);
        }
        if (id == a && real) {
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; e++) v[e] = y[e] + acc[e >> 2][e & 3];
            store16f(orow, n, p.N, v);
        }
    });
}

// Eight values of a row from column n on, as fp32; past N zeros.
template <typename T>
struct Eight {
    v4u32 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* row, int n, int N)
    {
        if constexpr (sizeof(T) == 2) {
            w[0] = load8(row, n, N);
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (n + 4 * h + 4 <= N) {
                    w[h] = *reinterpret_cast<const v4u32_any*>(row + n + 4 * h);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++) w[h][e] = n + 4 * h + e < N ? __float_as_uint(row[n + 4 * h + e]) : 0u;
                }
            }
        }
    }
    __device__ __forceinline__ float operator[](int e) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e >> 2][e & 3]);
        else return __uint_as_float(e & 1 ? w[0][e >> 1] & 0xFFFF0000u : w[0][e >> 1] << 16);
    }
};
template <typename T>
__device__ __forceinline__ void store8f(T* row, int n, int N, const float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        const v4u32 w = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
        if (n + 8 <= N) {
            *reinterpret_cast<v4u32_any*>(row + n) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (n + e < N) row[n + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (n + 4 * h + 4 <= N) {
                *reinterpret_cast<v4u32_any*>(row + n + 4 * h) =
                    v4u32{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                          __float_as_uint(v[4 * h + 3])};
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + 4 * h + e < N) row[n + 4 * h + e] = v[4 * h + e];
            }
        }
    }
}

// A tile of the list by 256 columns per block, a wave 64 of them.  y is on its way while the tile's u, for
// all waves, and the factor, for each, are staged in LDS; the sums pass through LDS to where neighbouring lanes
// have neighbouring columns, as y came (as the instruction leaves them, a lane's row is far from its
// neighbour's, and the L1 takes a lane at a time).
// ONE: all ranks at once (RC chosen so); else 16 RC of them in turn, staged anew for each row tile (whose sums then need
// no more registers): 8192 rows, N = K = 4096, 16 adapters, the whole call at ranks 64 / 128 / 256 / 512 77 / 130 / 220 / 393 us.
// 8192 rows, N = 4096, rank 64: 41 us, 3.3 TB/s, three blocks a CU (registers); a fourth spills and is slower.
template <int RC>
struct ExpandLds {
    static constexpr int FACTOR = 16 * RC * 128, SUMS = 16 * 256;     // a wave's part of the factor, then of the sums: 16 rows
    uint8_t us[kTile * 16 * RC * 4];                                  // (16 RC ranks of a row, twice)
    uint8_t wave[4][FACTOR > SUMS ? FACTOR : SUMS];
};
template <int RC, typename T, bool ONE>
__device__ __forceinline__ void expand_tile(const ExpandArgs& p, int block, ExpandLds<RC>& shared)
{
    uint8_t* us = shared.us;
    auto& lds = shared.wave;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int blocks = (p.N + 255) / 256;                      // along a row, which go first
    const Tile t = p.list.tiles[block / blocks];
    const bool none = t.a >= p.L;
    if (t.count == 0 || (none && p.in_place)) return;
    const int c = block % blocks * 256 + 64 * wave, s8 = lane & 7, n = c + 8 * s8;
    // this lane's rows 8 q + lane / 8, and its columns n .. + 7
    int m[8];
#pragma unroll
    for (int q = 0; q < 8; q++) m[q] = 8 * q + (lane >> 3) < t.count ? p.list.order[t.first + 8 * q + (lane >> 3)] : -1;
    v4u32 f[2 * RC];
    if (ONE && !none) load_factor<RC>(p.f, t.a, p.r, 0, c, p.N, f);
    Eight<T> y[8];
#pragma unroll
    for (int q = 0; q < 8; q++) {
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; h++) y[q].w[h] = v4u32{0u, 0u, 0u, 0u};
        if (p.y && m[q] >= 0 && n < p.N) y[q].load(static_cast<const T*>(p.y) + (int64_t)m[q] * p.ldy, n, p.N);
    }
    // Where 16-byte segments go, so that the lanes that are served together (0-3, 12-15 and 20-27 of each 32, and
    // the others; of a write eight in a row) hit distinct banks.
    auto u_at = [](int i, int sg) {
        if constexpr (RC == 1) return i * 64 + (sg ^ ((i >> 3 & 1) * 3)) * 16;
        else if constexpr (RC == 2) return i * 128 + (sg ^ (i >> 1 & 7)) * 16;
        else return i * 256 + (sg ^ (i & 15)) * 16;
    };
    auto sum_at = [](int i, int sg) { return i * 64 + (sg ^ ((i >> 1 & 1) | (i & 1) << 1 | (i & 12))) * 4; };
    MmReader<64, true, 4> reader;
    reader.begin_at(0, lane, 8 * (kq & 1));
    auto stage_u = [&](int j0) {
        constexpr int SEGS = 4 * RC, EACH = kTile * SEGS / 256;       // 16-byte segments of a row: half u, half what it left
#pragma unroll
        for (int q = 0; q < EACH; q++) {
            const int i = (q * 256 + tid) / SEGS, sg = (q * 256 + tid) % SEGS, j = j0 + sg % (SEGS / 2) * 8;
            v4u32 v = {0u, 0u, 0u, 0u};
            if (i < t.count && j < p.rp)
                v = *reinterpret_cast<const v4u32*>(p.u + ((int64_t)(t.first + i) * 2 + sg / (SEGS / 2)) * p.rp + j);
            *reinterpret_cast<v4u32*>(us + u_at(i, sg)) = v;
        }
    };
    v8bf b[RC][4];
    auto operands = [&]() {
#pragma unroll
        for (int k = 0; k < RC; k++)
#pragma unroll
            for (int w = 0; w < 4; w++) b[k][w] = reader.read_at(lds[wave], w, 16 * k);
    };
    if (ONE && !none) {
        stage_u(0);
        stage_factor<RC>(f, lds[wave]);
        __syncthreads();
        operands();
    }
    float* sums = reinterpret_cast<float*>(lds[wave]);
#pragma unroll
    for (int i = 0; i < kTile / 16; i++) {
        if (16 * i >= t.count) break;
        v4f acc[4];
#pragma unroll
        for (int w = 0; w < 4; w++) acc[w] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int j0 = 0; j0 < (none ? 0 : ONE ? 1 : p.r); j0 += 16 * RC) {
            if constexpr (!ONE) {
                __syncthreads();                               // (the ranks, or the sums, before are read)
                stage_u(j0);
                load_factor<RC>(p.f, t.a, p.r, j0, c, p.N, f);
                stage_factor<RC>(f, lds[wave]);
                __syncthreads();
                operands();
            }
#pragma unroll
            for (int k = 0; k < RC; k++) {
                const v8bf u = *reinterpret_cast<const v8bf*>(us + u_at(16 * i + r16, (kq >> 1) * 2 * RC + 2 * k + (kq & 1)));
#pragma unroll
                for (int w = 0; w < 4; w++) acc[w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[k][w], u, acc[w], 0, 0, 0);
            }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 4; k++)
            *reinterpret_cast<float4*>(sums + sum_at(r16, 4 * kq + k)) = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int q = 2 * i + h, r = 8 * h + (lane >> 3);
            const float4 lo = *reinterpret_cast<const float4*>(sums + sum_at(r, 2 * s8));
            const float4 hi = *reinterpret_cast<const float4*>(sums + sum_at(r, 2 * s8 + 1));
            if (m[q] < 0 || n >= p.N) continue;
            const float add[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            float v[8];
            // (a row without an adapter stays what it is, a negative zero too)
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = none ? y[q][e] : y[q][e] + add[e];
            store8f(static_cast<T*>(p.out) + (int64_t)m[q] * p.ldo, n, p.N, v);
        }
    }
}

template <int RC, typename T, bool ONE>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) void k_lora_expand_tile(ExpandArgs p)
{
    __shared__ __align__(128) ExpandLds<RC> shared;
    expand_tile<RC, T, ONE>(p, blockIdx.x, shared);
}

struct OuterJob {
    const uint16_t* u;                          // [M][2][rp], by row, or by place
    const uint16_t* x; int64_t ldx; int N;      // rows, columns
    void* d;                                    // [L][r][N]
    int bf16, blocks;                           // column blocks of 64
};
struct OuterArgs {
    int M, L, r, rp, accumulate;
    const int32_t* ids;
    OuterJob job[2];
    Listing list;
};

// Sums over the rows of one adapter: 16 RC ranks by 64 columns per block.  The adapter's rows
// are its part of the list, or listed here, 2048 rows at a time, in order; the waves take 32 of
// them in turn, the next ones on their way while these are multiplied, and add up in the order
// of the waves.
constexpr int kOuterRows = 2048;
template <int RC, bool LISTED>
struct OuterLds {
    static constexpr int UW = 32 * RC, XB = 32 * 128, UB = 32 * UW * 2;   // ranks of a row (twice 16 RC), bytes of a step
    uint8_t wave[4][XB + UB];
    uint16_t listed[LISTED ? 8 : kOuterRows];
    int counts[4];
};
template <int RC, bool LISTED>
__device__ __forceinline__ void outer_block(const OuterArgs& p, int block, int a, int chunk, OuterLds<RC, LISTED>& shared)
{
    constexpr int UW = 32 * RC, XB = 32 * 128;
    auto& lds = shared.wave;
    uint16_t* listed = shared.listed;
    int* counts = shared.counts;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const bool second = block >= p.job[0].blocks;
    const OuterJob& job = p.job[second];
    const int c0 = (block - (second ? p.job[0].blocks : 0)) * 64, j0 = chunk * 16 * RC;
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
    // n rows: row(i) of x, place(i) of u
    auto sums = [&](int n, auto row, auto place) {
        // 32 of them: where they are, a step ahead of them; columns and ranks in registers, zeros past the end
        constexpr int DEEP = RC <= 2 ? 2 : 1;                  // steps of the wave on their way
        constexpr int SEGS = UW / 8;                           // of a row of u: half for u, half for what it left
        int at_row[4];
        v4u32 xv[DEEP][4], uv[DEEP][2 * RC];
        auto find = [&](int s) {
#pragma unroll
            for (int q = 0; q < 4; q++) at_row[q] = 32 * s + 8 * q + (lane >> 3) < n ? row(32 * s + 8 * q + (lane >> 3)) : -1;
        };
        auto load = [&](int s, v4u32 (&x)[4], v4u32 (&u)[2 * RC]) {
            // (opaque: the addresses' parts are made anew, or they take the registers of the loads on their way)
            int l = lane;
            asm volatile("" : "+v"(l));
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int c = c0 + 8 * (l & 7);
                x[q] = v4u32{0u, 0u, 0u, 0u};
                if (at_row[q] >= 0 && c < job.N) x[q] = load8(job.x + (int64_t)at_row[q] * job.ldx, c, job.N);
            }
#pragma unroll
            for (int q = 0; q < 2 * RC; q++) {
                const int at = q * 64 + l, i = 32 * s + at / SEGS, sg = at % SEGS;
                const int j = j0 + (sg % (SEGS / 2)) * 8;
                u[q] = v4u32{0u, 0u, 0u, 0u};
                if (i < n && j < p.rp)
                    u[q] = *reinterpret_cast<const v4u32*>(job.u + ((int64_t)place(i) * 2 + sg / (SEGS / 2)) * p.rp + j);
            }
        };
        auto step = [&](int s, v4u32 (&x)[4], v4u32 (&u)[2 * RC]) {
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int i = 8 * q + (lane >> 3);
                *reinterpret_cast<v4u32*>(xs + i * 128 + ((lane & 7) ^ (2 * column_swizzle<64>(i))) * 16) = x[q];
            }
#pragma unroll
            for (int q = 0; q < 2 * RC; q++) {
                const int at = q * 64 + lane, i = at / SEGS;
                *reinterpret_cast<v4u32*>(us + i * UW * 2 + ((at % SEGS) ^ (2 * column_swizzle<UW>(i))) * 16) = u[q];
            }
            load(s + 4 * DEEP, x, u);
            find(s + 4 * DEEP + 4);
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
        };
        // (steps past the end load zeros)
        const int steps = (n + 31) / 32;
        if (wave >= steps) return;
#pragma unroll
        for (int d = 0; d < DEEP; d++) {
            find(wave + 4 * d);
            load(wave + 4 * d, xv[d], uv[d]);
        }
        find(wave + 4 * DEEP);
        for (int s = wave; s < steps; s += 4 * DEEP)
#pragma unroll
            for (int d = 0; d < DEEP; d++) step(s + 4 * d, xv[d], uv[d]);
    };
    int any = 0;
    if constexpr (LISTED) {
        const int begin = p.list.begin[a];
        any = p.list.begin[a + 1] - begin;
        const int* order = p.list.order + begin;
        sums(any, [&](int i) { return order[i]; }, [&](int i) { return begin + i; });
    } else {
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
                if (has >> e & 1) listed[at++] = (uint16_t)(8 * tid + e);
            __syncthreads();
            any |= n;
            auto row = [&](int i) { return seg + listed[i]; };
            sums(n, row, row);
        }
    }
    if (any == 0 && p.accumulate) return;          // (adding a sum of nothing would turn -0 into 0)
    // The sums of the waves that had steps, in their order, to where neighbouring lanes have neighbouring columns (in
    // the instruction's result, lane: rank 16 c + r16, columns 16 t + 4 kq .. + 3): 16-byte segments XORed by the row,
    // or sixteen lanes would write to the same banks.
    float* total = reinterpret_cast<float*>(lds);
    static_assert(sizeof(lds) >= 16 * RC * 64 * 4, "the sums fit");
    auto total_at = [&](int j, int sg) { return total + j * 64 + (sg ^ (j & 15)) * 4; };
    const int waves = LISTED ? max(1, min(4, (any + 31) / 32)) : 4;
    for (int w = 0; w < 4; w++) {
        if (w >= waves) break;
        __syncthreads();
        if (wave == w) {
#pragma unroll
            for (int c = 0; c < RC; c++)
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    float4* to = reinterpret_cast<float4*>(total_at(16 * c + r16, 4 * t + kq));
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
    auto store = [&](auto* d) {
        using T = std::remove_reference_t<decltype(*d)>;
#pragma unroll 1
        for (int i = tid; i < 16 * RC * 8; i += 256) {
            const int jr = i >> 3, sg = i & 7, j = j0 + jr, c = c0 + 8 * sg;
            if (j >= p.r || c >= job.N) continue;
            T* row = d + ((int64_t)a * p.r + j) * job.N;
            const float4 lo = *reinterpret_cast<const float4*>(total_at(jr, 2 * sg)), hi = *reinterpret_cast<const float4*>(total_at(jr, 2 * sg + 1));
            float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            if (p.accumulate) {
                Eight<T> old;
                old.load(row, c, job.N);
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = old[e] + v[e];
            }
            store8f(row, c, job.N, v);
        }
    };
    if (job.bf16) store(static_cast<uint16_t*>(job.d));
    else store(static_cast<float*>(job.d));
}

template <int RC, bool LISTED>
__global__ __launch_bounds__(256) void k_lora_outer(OuterArgs p)
{
    __shared__ __align__(128) OuterLds<RC, LISTED> shared;
    outer_block<RC, LISTED>(p, blockIdx.x, blockIdx.y, blockIdx.z, shared);
}

// dx, and the gradients of the factors: the longer blocks of these first, all ranks at once.  8192 rows, 2048 x 4096,
// rank 32, 8 adapters: 50 us, 4 TB/s; in two launches 35 and 38.  The bound keeps three blocks a CU (two: 10 us more).
template <int RC, typename T>
__global__ __launch_bounds__(256, RC < 4 ? 3 : 2) void k_lora_gradients(OuterArgs o, int columns, int outer, ExpandArgs e)
{
    __shared__ __align__(128) union {
        ExpandLds<RC> expand;
        OuterLds<RC, true> outer;
    } shared;
    const int block = blockIdx.x;
    if (block < outer) outer_block<RC, true>(o, block % columns, block / columns, 0, shared.outer);
    else expand_tile<RC, T, true>(e, block - outer, shared.expand);
}

// ---- host ----
// Whether the rows are listed first.  Unlisted, a tile of 16 rows is gone over once for each adapter among them, up to
// min(L, 16) times; listed, a tile of 64 has one, but the list takes a launch of 7 to 10 us.  Times in us, K = N = 4096,
// rank 16, unlisted / listed, rows in any order (in runs):
//                3 adapters                     16 adapters
//   rows     forward       backward       forward          backward
//    512   13/21 (13/21)  22/22 (22/22)   22/21 (14/21)    50/35 (36/34)
//   1024   18/22 (16/22)  33/27 (30/27)   35/25 (16/24)    72/41 (42/41)
//   2048   25/27 (19/28)  46/32 (37/32)   53/30 (20/29)   103/46 (52/44)
//   8192   63/48 (47/49) 122/78 (95/77)  159/50 (49/49)   304/87 (123/84)
// The order is not known here: the rules lie between.  Above 1024 adapters, K = N = 1024, rank 16:
//                      2047 adapters                   4096                            16384
//   rows     forward        backward        forward         backward         forward          backward
//   1024   33/43 (15/28)  392/170 (294/90)  33/58 (15/43)  664/255 (553/164)                 2238/733 (2121/625)
//   2048   46/55 (16/28)  496/220 (346/95)  47/78 (16/45)  847/333 (637/168)                 2732/841 (2401/651)
//   8192  134/74 (29/39) 1503/304 (1055/121) 141/135 (29/61) 2584/567 (2039/208) 160/296 (31/146) 8572/1372 (7957/710)
// Backward, an unlisted block of an adapter's sums looks through all rows; forward, a tile never has more than 16.
bool listed_first(int M, int L, bool backward)
{
    const int64_t work = (int64_t)M * std::min(L, 16);
    return backward ? work > 1000 : work > 8192 && L <= 1024;
}
int64_t most_tiles(int64_t M, int64_t L) { return M / kTile + std::min<int64_t>(M, L + 1); }

template <bool MANY>
hipError_t launch_list(int M, int L, const int32_t* ids, const Listing& list, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_lora_list<MANY>;
    constexpr int COUNTERS = (16 + 2) * 4, MOST = MANY ? kListAdapters : 1024;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), COUNTERS * MOST, allowed); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), COUNTERS * std::min(L + 1, MOST), s, M, L, ids, list, (int)most_tiles(M, L));
    return hipGetLastError();
}
hipError_t run_list(int M, int L, const int32_t* ids, const Listing& list, hipStream_t s)
{
    return L + 1 > 1024 ? launch_list<true>(M, L, ids, list, s) : launch_list<false>(M, L, ids, list, s);
}

template <int NJ, bool LISTED>
hipError_t launch_shrink(const ShrinkArgs& p, int jobs, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_lora_shrink<NJ, LISTED>;
    constexpr int BYTES = shrink_bytes<NJ>();
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), BYTES, allowed); e != hipSuccess) return e;
    const int chunks = (int)over(p.r, 16 * NJ);
    const int64_t tiles = LISTED ? most_tiles(p.M, p.L) : over(p.M, 16);
    // a block for each adapter that a tile's rows may have, where there are few tiles
    const int slots = LISTED ? kTile / 16 : (int)std::max<int64_t>(1, std::min<int64_t>(16, 1024 / tiles));
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles, (unsigned)slots, (unsigned)(chunks * jobs)), dim3(64 * kShrinkWaves), BYTES,
                       s, p, chunks);
    return hipGetLastError();
}
template <bool LISTED>
hipError_t shrink_by_rank(const ShrinkArgs& p, int jobs, hipStream_t s)
{
    if (p.r <= 16) return launch_shrink<1, LISTED>(p, jobs, s);
    if (p.r <= 32) return launch_shrink<2, LISTED>(p, jobs, s);
    return launch_shrink<4, LISTED>(p, jobs, s);
}
template <int NI, int NS>
hipError_t launch_ring(const ShrinkArgs& p, int jobs, hipStream_t s)
{
    static LdsAllowed allowed;
    const auto kernel = k_lora_shrink_ring<NI, NS>;
    using R = ShrinkRing<NI, NS>;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), R::BYTES, allowed); e != hipSuccess) return e;
    const int chunks = (int)over(p.r, 16 * NI);
    hipLaunchKernelGGL(kernel, dim3((unsigned)most_tiles(p.M, p.L), 1, (unsigned)(chunks * jobs)), dim3(64 * kSums), R::BYTES, s,
                       p, chunks);
    return hipGetLastError();
}
hipError_t run_shrink(const ShrinkArgs& p, int jobs, hipStream_t s)
{
    if (!p.list.order) return shrink_by_rank<false>(p, jobs, s);
    for (int j = 0; j < jobs; j++)
        if (!in_place(p.job[j].x, p.job[j].K, p.job[j].ldx) || !aligned_to(p.job[j].f, 16)) return shrink_by_rank<true>(p, jobs, s);
    if (p.r <= 16) return launch_ring<1, 4>(p, jobs, s);
    if (p.r <= 32) return launch_ring<2, 3>(p, jobs, s);
    return launch_ring<4, 2>(p, jobs, s);
}

template <int RC>
hipError_t launch_expand(const ExpandArgs& p, int bf16, hipStream_t s)
{
    if (p.list.order) {
        const int64_t blocks = over(p.N, 256) * most_tiles(p.M, p.L);
        if (blocks > INT32_MAX) return hipErrorInvalidValue;
        auto run = [&](auto one) {
            constexpr bool ONE = decltype(one)::value;
            if (bf16) hipLaunchKernelGGL((k_lora_expand_tile<RC, uint16_t, ONE>), dim3((unsigned)blocks), dim3(256), 0, s, p);
            else hipLaunchKernelGGL((k_lora_expand_tile<RC, float, ONE>), dim3((unsigned)blocks), dim3(256), 0, s, p);
        };
        if (RC < 4 || p.r <= 64) run(std::true_type{});
        else if constexpr (RC == 4) run(std::false_type{});
        return hipGetLastError();
    }
    const int64_t blocks = over(p.N, 256) * over(p.M, 16);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    // (a wave for each adapter that a tile's rows may have, where there are few tiles)
    const dim3 grid((unsigned)blocks, (unsigned)std::max<int64_t>(1, std::min<int64_t>(16, 2048 / blocks)));
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

template <int RC, bool LISTED>
hipError_t launch_outer(const OuterArgs& p, hipStream_t s)
{
    hipLaunchKernelGGL((k_lora_outer<RC, LISTED>), dim3((unsigned)(p.job[0].blocks + p.job[1].blocks), (unsigned)p.L,
                                                        (unsigned)over(p.r, 16 * RC)), dim3(256), 0, s, p);
    return hipGetLastError();
}
template <bool LISTED>
hipError_t outer_by_rank(const OuterArgs& p, hipStream_t s)
{
    if (p.r <= 16) return launch_outer<1, LISTED>(p, s);
    if (p.r <= 32) return launch_outer<2, LISTED>(p, s);
    return launch_outer<4, LISTED>(p, s);
}
hipError_t run_outer(const OuterArgs& p, hipStream_t s)
{
    return p.list.order ? outer_by_rank<true>(p, s) : outer_by_rank<false>(p, s);
}

// Both gradients, in one launch where the rows are listed and all ranks fit a block.
template <int RC>
hipError_t launch_gradients(const OuterArgs& o, const ExpandArgs& e, int bf16, hipStream_t s)
{
    const int64_t columns = o.job[0].blocks + o.job[1].blocks, outer = columns * o.L, all = outer + over(e.N, 256) * most_tiles(e.M, e.L);
    if (all > INT32_MAX) return hipErrorInvalidValue;
    if (bf16) hipLaunchKernelGGL((k_lora_gradients<RC, uint16_t>), dim3((unsigned)all), dim3(256), 0, s, o, (int)columns, (int)outer, e);
    else hipLaunchKernelGGL((k_lora_gradients<RC, float>), dim3((unsigned)all), dim3(256), 0, s, o, (int)columns, (int)outer, e);
    return hipGetLastError();
}
hipError_t run_gradients(const OuterArgs& o, const ExpandArgs& e, int bf16, hipStream_t s)
{
    if (o.list.order && o.r <= 64) {
        if (o.r <= 16) return launch_gradients<1>(o, e, bf16, s);
        if (o.r <= 32) return launch_gradients<2>(o, e, bf16, s);
        return launch_gradients<4>(o, e, bf16, s);
    }
    if (const hipError_t x = run_expand(e, bf16, s); x != hipSuccess) return x;
    return run_outer(o, s);
}

int ranks(int r) { return (r + 15) / 16 * 16; }
size_t lora_u(int64_t M, int r) { return up256((size_t)(M * 2 * ranks(r) * 2)); }
size_t lora_list(int M, int L, bool backward)
{
    if (!listed_first(M, L, backward)) return 0;
    return up256((size_t)M * 4) + up256((size_t)(L + 2) * 4) + 256 + up256((size_t)most_tiles(M, L) * sizeof(Tile));
}
Listing listing(uint8_t* ws, int M, int L, bool backward)
{
    if (!listed_first(M, L, backward)) return Listing{};
    Listing l;
    l.order = reinterpret_cast<int*>(ws);
    l.begin = reinterpret_cast<int*>(ws += up256((size_t)M * 4));
    l.tiles_n = reinterpret_cast<int*>(ws += up256((size_t)(L + 2) * 4));
    l.tiles = reinterpret_cast<Tile*>(ws += 256);
    return l;
}

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
    return lora_list(p->M, p->L, backward != 0) + lora_u(p->M, p->r) * (backward ? 2 : 1);
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
    if (ws_bytes < moe_lora_workspace_bytes(p, 0)) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Listing list = listing(ws, p->M, p->L, false);
    if (list.order && run_list(p->M, p->L, ids, list, s) != hipSuccess) return V4MOE_ELAUNCH;
    uint16_t* u = reinterpret_cast<uint16_t*>(ws + lora_list(p->M, p->L, false));
    const int rp = ranks(p->r);
    const ShrinkArgs sh{p->M, p->L, p->r, rp, ids, scale, {{x, ldx, p->K, a, u}, {}}, list};
    if (run_shrink(sh, 1, s) != hipSuccess) return V4MOE_ELAUNCH;
    const ExpandArgs ex{p->M, p->N, p->L, p->r, rp, ids, u, b, y, ldy, out, ldo, out == y, list};
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
    if (ws_bytes < moe_lora_workspace_bytes(p, 1)) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Listing list = listing(ws, p->M, p->L, true);
    if (list.order && run_list(p->M, p->L, ids, list, s) != hipSuccess) return V4MOE_ELAUNCH;
    ws += lora_list(p->M, p->L, true);
    uint16_t* du = reinterpret_cast<uint16_t*>(ws);
    uint16_t* u = reinterpret_cast<uint16_t*>(ws + lora_u(p->M, p->r));
    const int rp = ranks(p->r);
    if (p->M > 0) {
        ShrinkArgs sh{p->M, p->L, p->r, rp, ids, scale, {}, list};
        int jobs = 0;
        if (dx || da) sh.job[jobs++] = ShrinkJob{dy, lddy, p->N, b, du};
        if (db) sh.job[jobs++] = ShrinkJob{x, ldx, p->K, a, u};
        if (jobs == 2 && p->K > p->N) std::swap(sh.job[0], sh.job[1]);       // (the longer one's blocks begin first)
        if (run_shrink(sh, jobs, s) != hipSuccess) return V4MOE_ELAUNCH;
    }
    const ExpandArgs ex{p->M, p->K, p->L, p->r, rp, ids, du, a, base, ldbase, dx, lddx, base == dx, list};
    OuterArgs o{p->M, p->L, p->r, rp, accumulate != 0, ids, {}, list};
    int jobs = 0;
    if (da) o.job[jobs++] = OuterJob{du, x, ldx, p->K, da, da_type == V4MOE_TYPE_BF16, (int)over(p->K, 64)};
    if (db) o.job[jobs++] = OuterJob{u, dy, lddy, p->N, db, db_type == V4MOE_TYPE_BF16, (int)over(p->N, 64)};
    const int bf16 = dx_type == V4MOE_TYPE_BF16;
    const bool rows = dx && p->M > 0;
    if ((rows && jobs > 0 ? run_gradients(o, ex, bf16, s) : rows ? run_expand(ex, bf16, s) : jobs > 0 ? run_outer(o, s) : hipSuccess) !=
        hipSuccess)
        return V4MOE_ELAUNCH;
    return V4MOE_OK;
}

}  // extern "C"
