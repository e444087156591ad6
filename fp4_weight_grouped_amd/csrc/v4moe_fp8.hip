// v4moe_fp8.hip -- dense products of E4M3 operands with an fp32 scale for each
// 128 of the contraction, and the quantisers that make those operands: the
// projections that stand around the MoE layer, in the layer's payload format.
//
//   quantise   s = fp32(amax / 448) over a group, 1 where that is zero; code =
//              E4M3(fp32(x / s)), nearest even, saturating.  Groups: 128
//              consecutive elements of a row (activations), of a column (the
//              operands of a weight gradient), or a 128x128 block (weights).
//              A group with an infinity or NaN gets scale NaN and codes 0, so
//              that every result it takes part in is NaN.
//   product    C[m][n] = sum over chunks c of 128 of
//                  as[c][m] * bs[n, c] * sum_{k in c} A[m][k] B[n][k],
//              each chunk's sum by one block-scaled matrix instruction (fp32
//              result), the chunks added by fused multiply-adds in increasing
//              c whatever the tile, so a row of C does not depend on the
//              other rows of the call.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

#include <hip/hip_runtime.h>

namespace v4moe {

namespace {

// What a 16-byte segment past the end of the contraction is copied from.
__device__ const uint4 g_zeros[64] = {};

template <typename T>
__device__ __forceinline__ float load_f32(const T* p);
template <>
__device__ __forceinline__ float load_f32<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_f32<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

// Eight consecutive elements, `n` of them inside the array (the rest read as
// zero); vec: the address is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&f)[8])
{
    if (vec && n >= 8) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; u++) {
                f[2 * u] = bf16_to_f32(q[u] & 0xFFFFu);
                f[2 * u + 1] = bf16_to_f32(q[u] >> 16);
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 8; u++) f[u] = u < n ? load_f32(p + u) : 0.0f;
    }
}

// Magnitudes are compared as their bits: a NaN is then larger than everything.
__device__ __forceinline__ uint32_t mag_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Scale of a group from the bits of its largest magnitude.
__device__ __forceinline__ float group_scale(uint32_t mag)
{
    if (mag >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float s = __uint_as_float(mag) / 448.0f;
    return s > 0.0f ? s : 1.0f;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s)
{
    if (s != s) return 0u;
    return e4m3x2(a / s, b / s) | (e4m3x2(c / s, d / s) << 16);
}

// One 128x128 tile of x [R][C] per block: thread t holds rows 8(t/16) .. +7,
// columns 8(t%16) .. +7.  Bound by HBM (a read of x, a byte or two written per
// element); the tile is read once for both orders.
//   ROWS: q [R][ldq], s [ceil(C/128)][R]: groups of 128 columns of a row
//   COLS: qt [C][ldqt], st [ceil(R/128)][C]: groups of 128 rows of a column
//   BLOCK: q, qt, s [ceil(R/128)][ceil(C/128)]: one group per tile
// Rows of q are written up to C rounded up to 16, zeros past C (qt likewise).
enum { kQuantRows = 1, kQuantCols = 2, kQuantBlock = 4 };
template <typename T, int MODE>
__global__ __launch_bounds__(256) void k_fp8_quant(int R, int C, const T* __restrict__ x, int64_t ldx, int vec,
                                                   uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s,
                                                   uint8_t* __restrict__ qt, int64_t ldqt, float* __restrict__ st)
{
    __shared__ uint32_t mx[4][128];
    __shared__ __align__(16) uint8_t tq[128][144];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int c0 = blockIdx.x * 128, r0 = blockIdx.y * 128;
    const int rt = 8 * (t >> 4), ct = 8 * (t & 15);
    const int nc = C - c0 - ct;                        // columns of this thread inside x
    float f[8][8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = r0 + rt + i;
        load8(x + (int64_t)min(r, R - 1) * ldx + min(c0 + ct, C - 1), r < R ? nc : 0, vec, f[i]);
    }
    const int cpad = (C + 15) / 16 * 16, rpad = (R + 15) / 16 * 16;
    if constexpr (MODE & kQuantRows) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 8; u++) m = max(m, mag_bits(f[i][u]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
            const float sc = group_scale(m);
            const int r = r0 + rt + i;
            if (r < R) {
                if (c0 + ct < cpad)
                    *reinterpret_cast<uint2*>(q + (int64_t)r * ldq + c0 + ct) =
                        make_uint2(codes4(f[i][0], f[i][1], f[i][2], f[i][3], sc),
                                   codes4(f[i][4], f[i][5], f[i][6], f[i][7], sc));
                if ((t & 15) == 0) s[(int64_t)blockIdx.x * R + r] = sc;
            }
        }
    }
    if constexpr (MODE & (kQuantCols | kQuantBlock)) {
        uint32_t m[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            m[u] = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) m[u] = max(m[u], mag_bits(f[i][u]));
            m[u] = max(m[u], (uint32_t)__shfl_xor((int)m[u], 16));
            m[u] = max(m[u], (uint32_t)__shfl_xor((int)m[u], 32));
            if (lane < 16) mx[wave][ct + u] = m[u];
        }
        __syncthreads();
        float sc[8];
        if constexpr (MODE & kQuantBlock) {
            uint32_t b = max(max(mx[0][lane], mx[1][lane]), max(mx[2][lane], mx[3][lane]));
            b = max(b, max(max(mx[0][64 + lane], mx[1][64 + lane]), max(mx[2][64 + lane], mx[3][64 + lane])));
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o));
#pragma unroll
            for (int u = 0; u < 8; u++) sc[u] = group_scale(b);
            if (t == 0) s[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sc[0];
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (r0 + rt + i < R && c0 + ct < cpad)
                    *reinterpret_cast<uint2*>(q + (int64_t)(r0 + rt + i) * ldq + c0 + ct) =
                        make_uint2(codes4(f[i][0], f[i][1], f[i][2], f[i][3], sc[0]),
                                   codes4(f[i][4], f[i][5], f[i][6], f[i][7], sc[0]));
        } else {
#pragma unroll
            for (int u = 0; u < 8; u++)
                sc[u] = group_scale(max(max(mx[0][ct + u], mx[1][ct + u]), max(mx[2][ct + u], mx[3][ct + u])));
            if (lane < 16 && wave == 0) {
#pragma unroll
                for (int u = 0; u < 8; u++)
                    if (u < nc) st[(int64_t)blockIdx.y * C + c0 + ct + u] = sc[u];
            }
        }
        // the codes transposed through LDS, then 16-byte stores along the rows
#pragma unroll
        for (int u = 0; u < 8; u++)
            *reinterpret_cast<uint2*>(&tq[ct + u][rt]) =
                make_uint2(codes4(f[0][u], f[1][u], f[2][u], f[3][u], sc[u]),
                           codes4(f[4][u], f[5][u], f[6][u], f[7][u], sc[u]));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = i * 256 + t, c = p >> 3, seg = p & 7;
            if (c0 + c < C && r0 + 16 * seg < rpad)
                *reinterpret_cast<uint4*>(qt + (int64_t)(c0 + c) * ldqt + r0 + 16 * seg) =
                    *reinterpret_cast<const uint4*>(&tq[c][16 * seg]);
        }
    }
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------
struct GemmArgs {
    int M, N, K;
    const uint8_t* a; int64_t lda; const float* as;     // A [M][lda], as [ceil(K/128)][M]
    const uint8_t* b; int64_t ldb; const float* bs;     // B [N][ldb]
    int64_t bs_n, bs_k;                                  // block scales: bs[(n/128)*bs_n + c*bs_k]; ROWS: bs [c][N]
    void* c; int64_t ldc;
    int c_bf16, accumulate, vec;                         // vec: C rows allow 4-column stores
};

// Both operands E4M3, no hardware scale (E8M0 127 = 2^0).  Weights (rows of B)
// are the instruction's first operand: lane l gets rows 4(l/16) .. +3 of B for
// row l%16 of A, so the activation scale is one value per lane.
__device__ __forceinline__ v4f mfma_e4m3(v8i w, v8i x)
{
    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, 127, 0, 127);
}

template <int WM, int WN, int MI, int NI, int NS, bool ROWS>
struct GemmTile {
    static constexpr int NW = WM * WN, BM = WM * MI * 16, BN = WN * NI * 16;
    static constexpr int AJ = (BM / 8 + NW - 1) / NW, BJ = (BN / 8 + NW - 1) / NW;    // 1 KiB pieces per wave
    static constexpr int AS = (BM + 63) / 64, BS = ROWS ? (BN + 63) / 64 : 0;         // 64-scale pieces
    static constexpr int SJ = (AS + BS + NW - 1) / NW;
    static constexpr int OPS = AJ + BJ + SJ;                                           // copies per wave and stage
    static constexpr int A_OFF = 0, B_OFF = BM * 128, S_OFF = B_OFF + BN * 128;
    static constexpr int STAGE = S_OFF + (AS + BS) * 256;
    static constexpr int BYTES = NS * STAGE;
    static_assert(OPS * (NS - 2) < 64 && NS >= 2, "vmcnt range");
    static_assert(NI * 16 <= 128 && 128 % (NI * 16) == 0, "a wave's rows of B lie in one 128-row block");
};

// A tile of C per block: WM x WN waves, each with MI x NI tiles of 16x16.
// Operand rows are staged in LDS, a chunk of 128 per stage, by direct-to-LDS
// copies NS-1 stages ahead; 16-byte segments are XOR-swizzled by (row/2)%8, so
// the 16 rows of an operand read hit distinct banks.
template <int WM, int WN, int MI, int NI, int NS, bool ROWS>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_gemm(GemmArgs g, int tiles_m, int tiles_n)
{
    using L = GemmTile<WM, WN, MI, NI, NS, ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tm = (int)blockIdx.x % tiles_m, tn = (int)blockIdx.x / tiles_m;
    const int m0 = tm * L::BM, n0 = tn * L::BN;
    const int nch = (g.K + 127) / 128;
    const uint8_t* abase = g.a + (int64_t)m0 * g.lda;
    const uint8_t* bbase = g.b + (int64_t)n0 * g.ldb;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;

    // byte offsets of this lane's 16-byte segments from the tile's first row
    uint32_t aoff[L::AJ], boff[L::BJ];
    int seg[L::AJ > L::BJ ? L::AJ : L::BJ];
#pragma unroll
    for (int j = 0; j < L::AJ; j++) {
        const int p = min(wave + j * L::NW, L::BM / 8 - 1), r = p * 8 + (lane >> 3);
        aoff[j] = (uint32_t)(min(r, g.M - 1 - m0) * (int)g.lda + (((lane & 7) ^ ((r >> 1) & 7)) * 16));
    }
#pragma unroll
    for (int j = 0; j < L::BJ; j++) {
        const int p = min(wave + j * L::NW, L::BN / 8 - 1), r = p * 8 + (lane >> 3);
        boff[j] = (uint32_t)(min(r, g.N - 1 - n0) * (int)g.ldb + (((lane & 7) ^ ((r >> 1) & 7)) * 16));
    }
    (void)seg;
    auto issue = [&](int c) {
        const uint32_t slot = lds0 + (uint32_t)(c % NS) * L::STAGE;
        const uint8_t *ac = abase + (int64_t)c * 128, *bc = bbase + (int64_t)c * 128;
        const int left = g.K - c * 128;              // bytes of a row inside the contraction
#pragma unroll
        for (int j = 0; j < L::AJ; j++) {
            const int p = min(wave + j * L::NW, L::BM / 8 - 1), r = p * 8 + (lane >> 3);
            const int sg = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
            if (left >= 128) dma16s(ac, aoff[j], slot + L::A_OFF + p * 1024);
            else dma16(sg < left ? (const void*)(ac + aoff[j]) : (const void*)&g_zeros[lane], slot + L::A_OFF + p * 1024);
        }
#pragma unroll
        for (int j = 0; j < L::BJ; j++) {
            const int p = min(wave + j * L::NW, L::BN / 8 - 1), r = p * 8 + (lane >> 3);
            const int sg = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
            if (left >= 128) dma16s(bc, boff[j], slot + L::B_OFF + p * 1024);
            else dma16(sg < left ? (const void*)(bc + boff[j]) : (const void*)&g_zeros[lane], slot + L::B_OFF + p * 1024);
        }
#pragma unroll
        for (int j = 0; j < L::SJ; j++) {
            const int p = min(wave + j * L::NW, L::AS + L::BS - 1);
            if (p < L::AS)
                dma4s(g.as + (int64_t)c * g.M, (uint32_t)min(m0 + p * 64 + lane, g.M - 1) * 4u, slot + L::S_OFF + p * 256);
            else
                dma4s(g.bs + (int64_t)c * g.N, (uint32_t)min(n0 + (p - L::AS) * 64 + lane, g.N - 1) * 4u,
                      slot + L::S_OFF + p * 256);
        }
    };

    const int wm = wave / WN, wn = wave % WN;
    const int arow = wm * MI * 16 + (lane & 15), brow = wn * NI * 16 + (lane & 15), kq = lane >> 4;
    const int nblk = min((n0 + wn * NI * 16), g.N - 1) >> 7;
    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
    for (int c = 0; c < NS - 1; c++)
        if (c < nch) issue(c);
    for (int c = 0; c < nch; c++) {
        // stage c has landed once at most the copies of the later stages are out
        if (c + NS - 2 < nch) wait_vm<L::OPS * (NS - 2)>();
        else wait_vm<0>();
        __syncthreads();
        if (c + NS - 1 < nch) issue(c + NS - 1);     // into the slot every wave left before the barrier
        const uint8_t* st = smem + (c % NS) * L::STAGE;
        auto frag = [&](const uint8_t* base, int row) {
            const int sw = (row >> 1) & 7;
            const uint4 lo = *reinterpret_cast<const uint4*>(base + row * 128 + ((kq ^ sw) * 16));
            const uint4 hi = *reinterpret_cast<const uint4*>(base + row * 128 + (((4 + kq) ^ sw) * 16));
            return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        };
        v8i bf[NI];
#pragma unroll
        for (int j = 0; j < NI; j++) bf[j] = frag(st + L::B_OFF, brow + 16 * j);
        float bs = 1.0f;
        float4 br[ROWS ? NI : 1];
        if constexpr (ROWS) {
#pragma unroll
            for (int j = 0; j < NI; j++)
                br[j] = *reinterpret_cast<const float4*>(st + L::S_OFF + L::AS * 256 + (wn * NI * 16 + 16 * j + 4 * kq) * 4);
        } else {
            bs = g.bs[nblk * g.bs_n + c * g.bs_k];
        }
#pragma unroll
        for (int i = 0; i < MI; i++) {
            const v8i af = frag(st + L::A_OFF, arow + 16 * i);
            const float sa = *reinterpret_cast<const float*>(st + L::S_OFF + (arow + 16 * i) * 4) * bs;
#pragma unroll
            for (int j = 0; j < NI; j++) {
                const v4f p = mfma_e4m3(bf[j], af);
                if constexpr (ROWS) {
                    acc[i][j][0] = fmaf(sa * br[j].x, p[0], acc[i][j][0]);
                    acc[i][j][1] = fmaf(sa * br[j].y, p[1], acc[i][j][1]);
                    acc[i][j][2] = fmaf(sa * br[j].z, p[2], acc[i][j][2]);
                    acc[i][j][3] = fmaf(sa * br[j].w, p[3], acc[i][j][3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[i][j][e] = fmaf(sa, p[e], acc[i][j][e]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MI; i++) {
        const int m = m0 + arow + 16 * i;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int n = n0 + wn * NI * 16 + 16 * j + 4 * kq, nv = min(4, g.N - n);
            if (nv <= 0) continue;
            v4f v = acc[i][j];
            if (g.c_bf16) {
                uint16_t* o = static_cast<uint16_t*>(g.c) + (int64_t)m * g.ldc + n;
                if (g.accumulate)
                    for (int e = 0; e < nv; e++) v[e] += bf16_to_f32(o[e]);
                const uint32_t lo = bf16x2(v[0], v[1]), hi = bf16x2(v[2], v[3]);
                if (g.vec && nv == 4) *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
                else
                    for (int e = 0; e < nv; e++) o[e] = (uint16_t)((e & 2 ? hi : lo) >> (16 * (e & 1)));
            } else {
                float* o = static_cast<float*>(g.c) + (int64_t)m * g.ldc + n;
                if (g.accumulate)
                    for (int e = 0; e < nv; e++) v[e] += o[e];
                if (g.vec && nv == 4) *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    for (int e = 0; e < nv; e++) o[e] = v[e];
            }
        }
    }
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }
inline int64_t chunks(int64_t v) { return (v + 127) / 128; }
inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename T>
hipError_t launch_quant(int mode, int R, int C, const T* x, int64_t ldx, uint8_t* q, int64_t ldq, float* s, uint8_t* qt,
                        int64_t ldqt, float* st, hipStream_t stream)
{
    const int vec = aligned_to(x, 16) && ldx % (16 / (int)sizeof(T)) == 0;
    const dim3 grid((unsigned)chunks(C), (unsigned)chunks(R));
    auto run = [&](auto m) {
        hipLaunchKernelGGL((k_fp8_quant<T, decltype(m)::value>), grid, dim3(256), 0, stream, R, C, x, ldx, vec, q, ldq, s,
                           qt, ldqt, st);
    };
    switch (mode) {
    case kQuantRows: run(std::integral_constant<int, kQuantRows>{}); break;
    case kQuantCols: run(std::integral_constant<int, kQuantCols>{}); break;
    case kQuantRows | kQuantCols: run(std::integral_constant<int, kQuantRows | kQuantCols>{}); break;
    default: run(std::integral_constant<int, kQuantBlock>{}); break;
    }
    return hipGetLastError();
}

hipError_t run_quant(int mode, int R, int C, const void* x, int type, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                     uint8_t* qt, int64_t ldqt, float* st, hipStream_t stream)
{
    if (type == V4MOE_TYPE_F32)
        return launch_quant(mode, R, C, static_cast<const float*>(x), ldx, q, ldq, s, qt, ldqt, st, stream);
    return launch_quant(mode, R, C, static_cast<const uint16_t*>(x), ldx, q, ldq, s, qt, ldqt, st, stream);
}

template <int WM, int WN, int MI, int NI, int NS, bool ROWS>
hipError_t launch_gemm(const GemmArgs& g, hipStream_t s)
{
    using L = GemmTile<WM, WN, MI, NI, NS, ROWS>;
    const auto kernel = k_fp8_gemm<WM, WN, MI, NI, NS, ROWS>;
    if (L::BYTES > 65536) {
        static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
        if (e != hipSuccess) return e;
    }
    const int tm = (g.M + L::BM - 1) / L::BM, tn = (g.N + L::BN - 1) / L::BN;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(64 * L::NW), L::BYTES, s, g, tm, tn);
    return hipGetLastError();
}

hipError_t run_gemm(const GemmArgs& g, bool rows, hipStream_t s)
{
    return rows ? launch_gemm<2, 2, 2, 2, 3, true>(g, s) : launch_gemm<2, 2, 2, 2, 3, false>(g, s);
}

bool type_ok(int t) { return t == V4MOE_TYPE_F32 || t == V4MOE_TYPE_BF16; }
size_t type_size(int t) { return t == V4MOE_TYPE_F32 ? 4 : 2; }
constexpr int64_t kMaxSide = 1 << 22;     // rows times this many bytes of a tile stay below 2^31

// x [R][C] of a type with leading dimension ld
int check_matrix(const void* x, int type, int64_t R, int64_t C, int64_t ld)
{
    if (!type_ok(type) || ld < C || ld > (1ll << 40)) return V4MOE_EDIMS;
    if (R > 0 && C > 0 && !x) return V4MOE_ENULL;
    return aligned_to(x, type_size(type)) ? V4MOE_OK : V4MOE_EALIGN;
}
bool side_ok(int64_t n) { return n >= 0 && n <= kMaxSide; }

struct LinearLayout {
    size_t xq, xs, dq, ds, xt, xts, dt, dts, total;
};
LinearLayout linear_layout(int64_t M, int64_t N, int64_t K, bool backward)
{
    LinearLayout L{};
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
    if (!backward) {
        L.xq = take(M * up16(K));
        L.xs = take(chunks(K) * M * 4);
    } else {
        L.dq = take(M * up16(N));
        L.ds = take(chunks(N) * M * 4);
        L.dt = take(N * up16(M));
        L.dts = take(chunks(M) * N * 4);
        L.xt = take(K * up16(M));
        L.xts = take(chunks(M) * K * 4);
    }
    L.total = o;
    return L;
}

int check_fp8mat(const v4moe_fp8mat* w, bool q, bool qt)
{
    if (!w) return V4MOE_ENULL;
    if (w->N < 1 || w->K < 1 || !side_ok(w->N) || !side_ok(w->K)) return V4MOE_EDIMS;
    if ((q && !w->q) || (qt && !w->qt) || !w->blk) return V4MOE_ENULL;
    if ((q && !aligned_to(w->q, 16)) || (qt && !aligned_to(w->qt, 16)) || !aligned_to(w->blk, 4)) return V4MOE_EALIGN;
    return V4MOE_OK;
}

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) int moe_fp8_quantize(int32_t M, int32_t K, const void* x, int32_t type,
                                                            int64_t ldx, uint8_t* q, float* s, uint8_t* qt, float* st,
                                                            void* stream)
{
    if (!side_ok(M) || !side_ok(K)) return V4MOE_EDIMS;
    if (const int rc = check_matrix(x, type, M, K, ldx)) return rc;
    if ((q != nullptr) != (s != nullptr) || (qt != nullptr) != (st != nullptr) || (!q && !qt)) return V4MOE_ENULL;
    if (!aligned_to(q, 16) || !aligned_to(qt, 16) || !aligned_to(s, 4) || !aligned_to(st, 4)) return V4MOE_EALIGN;
    if (M == 0 || K == 0) return V4MOE_OK;
    if (!device_ready()) return V4MOE_EDEVICE;
    const int mode = (q ? kQuantRows : 0) | (qt ? kQuantCols : 0);
    return run_quant(mode, M, K, x, type, ldx, q, up16(K), s, qt, up16(M), st, static_cast<hipStream_t>(stream)) ==
                   hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_fp8_quantize_weights(int32_t N, int32_t K, const void* w, int32_t type,
                                                                    int64_t ldw, uint8_t* q, uint8_t* qt, float* blk,
                                                                    void* stream)
{
    if (N < 1 || K < 1 || !side_ok(N) || !side_ok(K)) return V4MOE_EDIMS;
    if (const int rc = check_matrix(w, type, N, K, ldw)) return rc;
    if (!q || !qt || !blk) return V4MOE_ENULL;
    if (!aligned_to(q, 16) || !aligned_to(qt, 16) || !aligned_to(blk, 4)) return V4MOE_EALIGN;
    if (!device_ready()) return V4MOE_EDEVICE;
    return run_quant(kQuantBlock, N, K, w, type, ldw, q, up16(K), blk, qt, up16(N), nullptr,
                     static_cast<hipStream_t>(stream)) == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_fp8_gemm(const v4moe_gemm* p, const uint8_t* a, const float* as,
                                                        const uint8_t* b, const float* bs, void* c, void* stream)
{
    if (!p) return V4MOE_ENULL;
    if (!side_ok(p->M) || !side_ok(p->N) || !side_ok(p->K) || p->K % 16) return V4MOE_EDIMS;
    if (p->lda < p->K || p->ldb < p->K || p->lda % 16 || p->ldb % 16 || p->lda > kMaxSide || p->ldb > kMaxSide)
        return V4MOE_EDIMS;
    if (p->b_scale != V4MOE_SCALE_BLOCK && p->b_scale != V4MOE_SCALE_ROW) return V4MOE_EDIMS;
    if (const int rc = check_matrix(c, p->c_type, p->M, p->N, p->ldc)) return rc;
    if (p->M == 0 || p->N == 0) return V4MOE_OK;
    if (p->K > 0 && (!a || !as || !b || !bs)) return V4MOE_ENULL;
    if (!aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(as, 4) || !aligned_to(bs, 4)) return V4MOE_EALIGN;
    if (!device_ready()) return V4MOE_EDEVICE;
    const bool bf16 = p->c_type == V4MOE_TYPE_BF16, rows = p->b_scale == V4MOE_SCALE_ROW;
    const GemmArgs g{p->M, p->N, p->K, a, p->lda, as, b, p->ldb, bs, p->bs_n, p->bs_k, c, p->ldc, bf16, p->accumulate != 0,
                     p->ldc % 4 == 0 && aligned_to(c, bf16 ? 8 : 16)};
    return run_gemm(g, rows, static_cast<hipStream_t>(stream)) == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) size_t moe_fp8_linear_workspace_bytes(int32_t M, int32_t N, int32_t K,
                                                                             int32_t backward)
{
    if (!side_ok(M) || !side_ok(N) || !side_ok(K) || N < 1 || K < 1) return 0;
    return linear_layout(M, N, K, backward != 0).total;
}

__attribute__((visibility("default"))) int moe_fp8_linear(int32_t M, const void* x, int32_t x_type, int64_t ldx,
                                                          const v4moe_fp8mat* w, void* y, int32_t y_type, int64_t ldy,
                                                          void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_fp8mat(w, true, false)) return rc;
    const int N = w->N, K = w->K;
    if (!side_ok(M)) return V4MOE_EDIMS;
    if (const int rc = check_matrix(x, x_type, M, K, ldx)) return rc;
    if (const int rc = check_matrix(y, y_type, M, N, ldy)) return rc;
    if (M == 0) return V4MOE_OK;
    if (!workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    const LinearLayout L = linear_layout(M, N, K, false);
    if (ws_bytes < L.total) return V4MOE_EWORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* xs = reinterpret_cast<float*>(ws + L.xs);
    if (const int rc = moe_fp8_quantize(M, K, x, x_type, ldx, ws + L.xq, xs, nullptr, nullptr, stream)) return rc;
    const v4moe_gemm g{M, N, (int32_t)up16(K), V4MOE_SCALE_BLOCK, y_type, 0, up16(K), up16(K), ldy, chunks(K), 1};
    return moe_fp8_gemm(&g, ws + L.xq, xs, w->q, w->blk, y, stream);
}

__attribute__((visibility("default"))) int moe_fp8_linear_backward(
    int32_t M, const void* x, int32_t x_type, int64_t ldx, const void* dy, int32_t dy_type, int64_t lddy,
    const v4moe_fp8mat* w, void* dx, int32_t dx_type, int64_t lddx, void* dw, int32_t dw_type, int64_t lddw,
    int32_t accumulate, void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_fp8mat(w, false, dx != nullptr)) return rc;
    const int N = w->N, K = w->K;
    if (!side_ok(M)) return V4MOE_EDIMS;
    if (!dx && !dw) return V4MOE_ENULL;
    if (dw)
        if (const int rc = check_matrix(x, x_type, M, K, ldx)) return rc;
    if (const int rc = check_matrix(dy, dy_type, M, N, lddy)) return rc;
    if (dx)
        if (const int rc = check_matrix(dx, dx_type, M, K, lddx)) return rc;
    if (dw)
        if (const int rc = check_matrix(dw, dw_type, N, K, lddw)) return rc;
    const LinearLayout L = linear_layout(M, N, K, true);
    if (M > 0 && !workspace) return V4MOE_ENULL;
    if (!aligned_to(workspace, 16)) return V4MOE_EALIGN;
    if (ws_bytes < L.total) return V4MOE_EWORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    if (M > 0) {
        if (const int rc = moe_fp8_quantize(M, N, dy, dy_type, lddy, dx ? ws + L.dq : nullptr, dx ? f32(L.ds) : nullptr,
                                            dw ? ws + L.dt : nullptr, dw ? f32(L.dts) : nullptr, stream))
            return rc;
        if (dw)
            if (const int rc = moe_fp8_quantize(M, K, x, x_type, ldx, nullptr, nullptr, ws + L.xt, f32(L.xts), stream))
                return rc;
    }
    if (dx && M > 0) {
        // dx = dy W: contraction over N, block (i, c) of W^T is block (c, i) of W
        const v4moe_gemm g{M, K, (int32_t)up16(N), V4MOE_SCALE_BLOCK, dx_type, 0, up16(N), up16(N), lddx, 1, chunks(K)};
        if (const int rc = moe_fp8_gemm(&g, ws + L.dq, f32(L.ds), w->qt, w->blk, dx, stream)) return rc;
    }
    if (dw) {
        // dW = dy^T x: contraction over the tokens, both scales per row
        const v4moe_gemm g{N, K, (int32_t)up16(M), V4MOE_SCALE_ROW, dw_type, accumulate, up16(M), up16(M), lddw, 0, 0};
        if (const int rc = moe_fp8_gemm(&g, ws + L.dt, f32(L.dts), ws + L.xt, f32(L.xts), dw, stream)) return rc;
    }
    return V4MOE_OK;
}

}  // extern "C"
