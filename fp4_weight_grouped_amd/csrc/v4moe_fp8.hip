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

#include <atomic>
#include <type_traits>

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

// Sixteen bytes at any element's address, in one access: unaligned ones are the
// hardware's to split.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef v4u v4u_any __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ v4u load16(const T* p) { return *reinterpret_cast<const v4u_any*>(p); }

// Magnitudes are compared as their bits: a NaN is then larger than everything.
__device__ __forceinline__ uint32_t mag_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Scale of a group from the bits of its largest magnitude.
__device__ __forceinline__ float group_scale(uint32_t mag)
{
    if (mag >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float s = __uint_as_float(mag) / 448.0f;
    return s > 0.0f ? s : 1.0f;
}

// E4M3 codes of x / s, the quotient rounded to fp32 first.  A scale well inside
// the normal range takes y = 1/s rounded and one correction of q = x y by its
// residual: that is within 5/(2 S) of the exact quotient's last place (S the
// scale's 24-bit integer), so another fp32 than the rounded quotient can only
// come out beside a rounding boundary of E4M3 for S within 5 of a multiple of
// 2^20, and for every such S (64 on either side were tried) and every 24-bit x
// the two are equal.  The others (y = 0) divide; a NaN scale gives codes 0.
struct Divisor {
    float s, y;
    Divisor() = default;
    __device__ __forceinline__ explicit Divisor(float scale)
        : s(scale), y(scale > 0x1p-80f && scale < 0x1p80f ? 1.0f / scale : 0.0f) {}
    __device__ __forceinline__ Divisor(float scale, float inverse) : s(scale), y(inverse) {}
    __device__ __forceinline__ float corrected(float x) const
    {
        // (the residual as q s - x: where it vanishes the quotient keeps its sign, a zero's too)
        const float q = x * y;
        return fmaf(-fmaf(q, s, -x), y, q);
    }
    __device__ __forceinline__ uint32_t quick4(float a, float b, float c, float d) const
    {
        return e4m3x2(corrected(a), corrected(b)) | (e4m3x2(corrected(c), corrected(d)) << 16);
    }
    __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) const
    {
        if (y != 0.0f) return quick4(a, b, c, d);
        if (s != s) return 0u;
        return e4m3x2(a / s, b / s) | (e4m3x2(c / s, d / s) << 16);
    }
};

// Maximum over lanes by DPP (quad xor 1, xor 2, half-row mirror: 8 lanes; row
// mirror: 16), in every lane of them.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    auto step = [&](auto ctrl) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, false));
    };
    step(std::integral_constant<int, 0xB1>{});
    step(std::integral_constant<int, 0x4E>{});
    step(std::integral_constant<int, 0x141>{});
    if constexpr (LANES == 16) step(std::integral_constant<int, 0x140>{});
    return v;
}

// Eight consecutive elements as they are in memory (zeros past the array's end).
template <typename T>
struct Raw {
    static constexpr int W = sizeof(T) / 2;          // 16-byte words
    v4u w[W];
    __device__ __forceinline__ float operator[](int u) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[u >> 2][u & 3]);
        else return __uint_as_float(u & 1 ? w[0][u >> 1] & 0xFFFF0000u : w[0][u >> 1] << 16);
    }
    // the compiler takes the words for new ones
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int h = 0; h < W; h++) asm volatile("" : "+v"(w[h]));
    }
    __device__ __forceinline__ void load(const T* p, int n)
    {
        if (n >= 8) {
#pragma unroll
            for (int h = 0; h < W; h++) w[h] = load16(p + 4 * h);
        } else {
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const uint32_t f = u < n ? __float_as_uint(load_f32(p + u)) : 0u, b = sizeof(T) == 4 ? f : f >> 16;
                if constexpr (sizeof(T) == 4) w[u >> 2][u & 3] = b;
                else w[0][u >> 1] = u & 1 ? w[0][u >> 1] | (b << 16) : b;
            }
        }
    }
};

// The largest magnitudes of word i of several Raw: fp32 one per word, bf16 two
// (their bits compare as integers), so half the instructions.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ uint32_t mag_word(uint32_t w) { return w & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu); }
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b)
{
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                       __builtin_bit_cast(u16x2, b)));
}
// ... and of a word alone, as the bits of an fp32
template <typename T>
__device__ __forceinline__ uint32_t word_mag(uint32_t w)
{
    if constexpr (sizeof(T) == 4) return w;
    else return max(w & 0xFFFF0000u, w << 16);
}
template <typename T>
__device__ __forceinline__ uint32_t largest(const Raw<T>& r)
{
    uint32_t m = mag_word<T>(r.w[0][0]);
#pragma unroll
    for (int i = 1; i < 4 * Raw<T>::W; i++) m = max_word<T>(m, mag_word<T>(r.w[i >> 2][i & 3]));
    return word_mag<T>(m);
}

// Groups along rows: x [R][C] -> q [R][ldq] (up to C rounded up to 16, zeros
// past C), s [ceil(C/128)][R].  Eight lanes per group, sixteen elements each; a
// block takes 2^lg consecutive groups of a row (at most a wave's eight) and
// 32 / 2^lg rows.  Bound by HBM: 8192x4096 bf16 19.0 to 19.6 us, 102 MB at 5.3 TB/s
// (an element-wise copy of 4 GiB: 6.2; sixteen lanes per group, whose scales are then
// twice the work, and a second correction of each quotient: 23 us, all of them issuing).
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_quant_rows(int R, int C, int lg, const T* __restrict__ x, int64_t ldx,
                                                        uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s)
{
    const int g = threadIdx.x >> 3;
    const int r = blockIdx.x * (32 >> lg) + (g >> lg), c = ((int)blockIdx.y << lg) + (g & ((1 << lg) - 1));
    if (r >= R || c * 128 >= C) return;                   // whole groups of lanes
    const int at = c * 128 + 16 * (threadIdx.x & 7);
    Raw<T> f[2];
#pragma unroll
    for (int h = 0; h < 2; h++) f[h].load(x + (int64_t)r * ldx + min(at + 8 * h, C - 1), C - at - 8 * h);
    const Divisor d(group_scale(lanes_max<8>(max(largest(f[0]), largest(f[1])))));
    uint4 codes;
    if (d.y != 0.0f)
        codes = make_uint4(d.quick4(f[0][0], f[0][1], f[0][2], f[0][3]), d.quick4(f[0][4], f[0][5], f[0][6], f[0][7]),
                           d.quick4(f[1][0], f[1][1], f[1][2], f[1][3]), d.quick4(f[1][4], f[1][5], f[1][6], f[1][7]));
    else
        codes = make_uint4(d.codes4(f[0][0], f[0][1], f[0][2], f[0][3]), d.codes4(f[0][4], f[0][5], f[0][6], f[0][7]),
                           d.codes4(f[1][0], f[1][1], f[1][2], f[1][3]), d.codes4(f[1][4], f[1][5], f[1][6], f[1][7]));
    if (at < C) *reinterpret_cast<uint4*>(q + (int64_t)r * ldq + at) = codes;
    if ((threadIdx.x & 7) == 0) s[(int64_t)c * R + r] = d.s;
}

// One 128x128 tile of x [R][C] per block, read once for both orders: thread t
// holds rows 4(t/16) .. +3, columns 8(t%16) .. +7 as they are in memory.  Bound by
// HBM, next to the tile's own latency and instructions: 16384x4096 fp32 weights
// 78 us (403 MB, 5.2 TB/s; 83 with a branch per row); 8192x2048 bf16 in both orders
// and 8192x4096 by columns in one launch 34 us (169 MB, 5.0 TB/s).  What helps is waves per CU (eight rows
// per thread took 47 us for the latter where four took 40, with the elements kept
// as floats or the next tile's loads out a tile ahead 60) and fewer instructions
// (40 -> 35: bf16 magnitudes two to an operation, their maxima over lanes by
// permutes of the vector unit, a column's scale inverted by one thread, one
// correction of each quotient).
//   ROWS: q [R][ldq], s [ceil(C/128)][R]: groups of 128 columns of a row
//   COLS: qt [C][ldqt], st [ceil(R/128)][C]: groups of 128 rows of a column
//   BLOCK: q, qt, s [ceil(R/128)][ceil(C/128)]: one group per tile
// Rows of q are written up to C rounded up to 16, zeros past C (qt likewise).
enum { kQuantRows = 1, kQuantCols = 2, kQuantBlock = 4 };
template <typename T>
struct QuantJob {
    int R, C;
    const T* x; int64_t ldx;
    uint8_t* q; int64_t ldq;
    float* s;
    uint8_t* qt; int64_t ldqt;
    float* st;
    int tiles() const { return (int)(((int64_t)R + 127) / 128 * (((int64_t)C + 127) / 128)); }
};
constexpr int kQuantThreads = 512;
struct QuantLds {
    __align__(16) uint32_t mx[kQuantThreads / 64][128];
    __align__(16) uint8_t tq[128 * 128];
};
template <typename T, int MODE>
__device__ __forceinline__ void quant_tile(const QuantJob<T>& job, int tile, QuantLds& lds)
{
    constexpr int NR = 4, NW = kQuantThreads / 64;      // rows per thread, waves
    const int R = job.R, C = job.C;
    const T* __restrict__ x = job.x;
    uint8_t* __restrict__ q = job.q;
    float* __restrict__ s = job.s;
    uint8_t* __restrict__ qt = job.qt;
    float* __restrict__ st = job.st;
    const int64_t ldx = job.ldx, ldq = job.ldq, ldqt = job.ldqt;
    auto& mx = lds.mx;
    auto& tq = lds.tq;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int rt = NR * (t >> 4), ct = 8 * (t & 15);
    const int cpad = (C + 15) / 16 * 16, rpad = (R + 15) / 16 * 16;
    const int nx = (C + 127) / 128;
    const int by = tile / nx, bx = tile % nx, r0 = by * 128, c0 = bx * 128;
    Raw<T> f[NR];
#pragma unroll
    for (int i = 0; i < NR; i++)
        f[i].load(x + (int64_t)min(r0 + rt + i, R - 1) * ldx + min(c0 + ct, C - 1), r0 + rt + i < R ? C - c0 - ct : 0);
    // rows' codes; together, so that no branch stands between one's divisions and the next's
    auto store_rows = [&](const Divisor (&d)[NR]) {
        uint2 codes[NR];
        bool quick = true;
#pragma unroll
        for (int i = 0; i < NR; i++) quick = quick && d[i].y != 0.0f;
        if (quick) {
#pragma unroll
            for (int i = 0; i < NR; i++)
                codes[i] = make_uint2(d[i].quick4(f[i][0], f[i][1], f[i][2], f[i][3]),
                                      d[i].quick4(f[i][4], f[i][5], f[i][6], f[i][7]));
        } else {
#pragma unroll
            for (int i = 0; i < NR; i++)
                codes[i] = make_uint2(d[i].codes4(f[i][0], f[i][1], f[i][2], f[i][3]),
                                      d[i].codes4(f[i][4], f[i][5], f[i][6], f[i][7]));
        }
#pragma unroll
        for (int i = 0; i < NR; i++)
            if (r0 + rt + i < R && c0 + ct < cpad)
                *reinterpret_cast<uint2*>(q + (int64_t)(r0 + rt + i) * ldq + c0 + ct) = codes[i];
    };
    if constexpr (MODE & kQuantRows) {
        uint32_t big[NR];
#pragma unroll
        for (int i = 0; i < NR; i++) big[i] = lanes_max<16>(largest(f[i]));
        const Divisor d[NR] = {Divisor(group_scale(big[0])), Divisor(group_scale(big[1])), Divisor(group_scale(big[2])),
                               Divisor(group_scale(big[3]))};
        store_rows(d);
        if ((t & 15) == 0) {
#pragma unroll
            for (int i = 0; i < NR; i++)
                if (r0 + rt + i < R) s[(int64_t)bx * R + r0 + rt + i] = d[i].s;
        }
    }
    // largest magnitude of each column in the wave's 16 rows, a word's columns together
    constexpr int NWORD = 4 * Raw<T>::W;
    uint32_t m[NWORD];
    // (the columns convert the elements anew: kept as floats they would cost two blocks of the CU's four)
#pragma unroll
    for (int i = 0; i < NR; i++) f[i].forget();
#pragma unroll
    for (int u = 0; u < NWORD; u++) {
        m[u] = mag_word<T>(f[0].w[u >> 2][u & 3]);
#pragma unroll
        for (int i = 1; i < NR; i++) m[u] = max_word<T>(m[u], mag_word<T>(f[i].w[u >> 2][u & 3]));
        // lanes 16 apart (odd rows of 16 for even ones), then 32 apart
        const auto a = __builtin_amdgcn_permlane16_swap(m[u], m[u], false, false);
        m[u] = max_word<T>(a[0], a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(m[u], m[u], false, false);
        m[u] = max_word<T>(b[0], b[1]);
    }
    if (lane < 16) {
#pragma unroll
        for (int h = 0; h < Raw<T>::W; h++)
            *reinterpret_cast<uint4*>(&mx[wave][(lane * Raw<T>::W + h) * 4]) =
                make_uint4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
    }
    __syncthreads();
    constexpr int WORDS = 128 * sizeof(T) / 4;           // of a tile's row
    auto word = [&](int c) {
        uint32_t v = mx[0][c];
#pragma unroll
        for (int i = 1; i < NW; i++) v = max_word<T>(v, mx[i][c]);
        return v;
    };
    Divisor d8[8];
    if constexpr (MODE & kQuantBlock) {
        uint32_t all = word_mag<T>(word(lane));
        if constexpr (WORDS == 128) all = max(all, word_mag<T>(word(64 + lane)));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) all = max(all, (uint32_t)__shfl_xor((int)all, o));
        d8[0] = Divisor(group_scale(all));
        if (t == 0) s[tile] = d8[0].s;
        const Divisor d[NR] = {d8[0], d8[0], d8[0], d8[0]};
        store_rows(d);
#pragma unroll
        for (int u = 1; u < 8; u++) d8[u] = d8[0];
    } else {
        // each column's scale and its inverse once, by one thread
        uint32_t v = 0;
        if (t < 128) v = sizeof(T) == 4 ? word(t) : t & 1 ? word(t >> 1) & 0xFFFF0000u : word(t >> 1) << 16;
        __syncthreads();
        if (t < 128) {
            const Divisor d(group_scale(v));
            mx[0][t] = __float_as_uint(d.s);
            mx[1][t] = __float_as_uint(d.y);
            if (c0 + t < C) st[(int64_t)by * C + c0 + t] = d.s;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const float4 sc = *reinterpret_cast<const float4*>(&mx[0][ct + 4 * h]);
            const float4 in = *reinterpret_cast<const float4*>(&mx[1][ct + 4 * h]);
            d8[4 * h] = Divisor(sc.x, in.x);
            d8[4 * h + 1] = Divisor(sc.y, in.y);
            d8[4 * h + 2] = Divisor(sc.z, in.z);
            d8[4 * h + 3] = Divisor(sc.w, in.w);
        }
    }
    // The codes transposed through LDS: column c's 128 bytes, their 16-byte
    // segments XORed by c/8 so that the columns a store covers spread over the
    // banks; then 16-byte stores along the rows of qt.
    bool quick = true;
#pragma unroll
    for (int u = 0; u < 8; u++) quick = quick && d8[u].y != 0.0f;
    auto column = [&](int u, uint32_t codes) {
        const int c = ct + u, r4 = t >> 4;
        *reinterpret_cast<uint32_t*>(tq + c * 128 + (((r4 >> 2) ^ (c >> 3 & 7)) * 16) + (r4 & 3) * 4) = codes;
    };
    if (quick) {
#pragma unroll
        for (int u = 0; u < 8; u++) column(u, d8[u].quick4(f[0][u], f[1][u], f[2][u], f[3][u]));
    } else {
#pragma unroll
        for (int u = 0; u < 8; u++) column(u, d8[u].codes4(f[0][u], f[1][u], f[2][u], f[3][u]));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int p = i * 512 + t, c = p >> 3, seg = p & 7;
        if (c0 + c < C && r0 + 16 * seg < rpad)
            *reinterpret_cast<uint4*>(qt + (int64_t)(c0 + c) * ldqt + r0 + 16 * seg) =
                *reinterpret_cast<const uint4*>(tq + c * 128 + ((seg ^ (c >> 3 & 7)) * 16));
    }
}

template <typename T, int MODE>
__global__ __launch_bounds__(kQuantThreads) void k_fp8_quant(QuantJob<T> job)
{
    __shared__ QuantLds lds;
    quant_tile<T, MODE>(job, blockIdx.x, lds);
}
// The operands of a backward in one launch: the incoming gradient (rows for the
// data gradient, columns for the weights'), then the activations (columns).
template <typename T, int MODE>
__global__ __launch_bounds__(kQuantThreads) void k_fp8_quant_pair(QuantJob<T> a, int tiles_a, QuantJob<T> b)
{
    __shared__ QuantLds lds;
    if ((int)blockIdx.x < tiles_a) quant_tile<T, MODE>(a, blockIdx.x, lds);
    else quant_tile<T, kQuantCols>(b, blockIdx.x - tiles_a, lds);
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
    int c_bf16, accumulate;
};

// Both operands E4M3, no hardware scale (E8M0 127 = 2^0).  Weights (rows of B)
// are the instruction's first operand: lane l gets rows 4(l/16) .. +3 of B for
// row l%16 of A, so the activation scale is one value per lane.
__device__ __forceinline__ v4f mfma_e4m3(v8i w, v8i x)
{
    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, 127, 0, 127);
}

// A wave's MI x NI tiles to C, 16 rows at a time through LDS (two buffers of
// 16 rows): a lane's four columns become 16-byte stores along the rows, whole
// lines where a row's part is one (straight from the registers the stores cost
// 22 us of 139 at 8192 x 4096).  16-byte segments XOR-swizzled by the row.  S: the
// type staged, fp32 where C is added to, so that a bf16 C takes the sum rounded once.
template <bool STREAM, int MI, int NI, typename S, typename T>
__device__ __forceinline__ void store_tile(const v4f (&acc)[MI][NI], uint8_t* stage, T* __restrict__ c, const GemmArgs& g,
                                           int m0, int n0)
{
    constexpr int ES = sizeof(S), RB = NI * 16 * ES, LR = RB / 16, PER = 16 / ES;    // bytes, lanes per row; elements per lane
    constexpr int RP = 64 / LR;                                                    // rows per pass
    const int lane = threadIdx.x & 63, r16 = lane & 15, kq = lane >> 4;
#pragma unroll
    for (int i = 0; i < MI; i++) {
        uint8_t* buf = stage + (i & 1) * (16 * NI * 16 * 4);
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int at = (16 * j + 4 * kq) * ES;
            uint8_t* d = buf + r16 * RB + (((at >> 4) ^ (r16 & (LR - 1))) << 4) + (at & 15);
            if constexpr (ES == 2) *reinterpret_cast<uint2*>(d) = make_uint2(bf16x2(acc[i][j][0], acc[i][j][1]),
                                                                             bf16x2(acc[i][j][2], acc[i][j][3]));
            else *reinterpret_cast<float4*>(d) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 16; q += RP) {
            const int r = q + lane / LR, sg = lane % LR;
            if (r >= 16) continue;                                     // (RP > 16: half the lanes)
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * RB + ((sg ^ (r & (LR - 1))) << 4));
            const int m = m0 + 16 * i + r, n = n0 + sg * PER;
            if (m >= g.M || n >= g.N) continue;
            T* o = c + (int64_t)m * g.ldc + n;
            if constexpr (sizeof(S) == sizeof(T)) {
                if (n + PER <= g.N && !g.accumulate) {
                    const v4u w4 = {v.x, v.y, v.z, v.w};
                    if (STREAM) __builtin_nontemporal_store(w4, reinterpret_cast<v4u_any*>(o));
                    else *reinterpret_cast<v4u_any*>(o) = w4;
                    continue;
                }
            }
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < PER; e++) {
                if (n + e >= g.N) break;
                if constexpr (ES == 2) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                else if constexpr (sizeof(T) == 2) o[e] = (uint16_t)bf16x2(bf16_to_f32(o[e]) + __uint_as_float(w[e]), 0.0f);
                else o[e] = g.accumulate ? o[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int WM, int WN, int MI, int NI, int NS, int KC, bool ROWS>
struct GemmTile {
    static constexpr int NW = WM * WN, BM = WM * MI * 16, BN = WN * NI * 16;
    static constexpr int AJ = (BM / 8 + NW - 1) / NW, BJ = (BN / 8 + NW - 1) / NW;    // 1 KiB pieces per wave
    static constexpr int AS = (BM + 63) / 64, BS = ROWS ? (BN + 63) / 64 : 0;         // 64-scale pieces
    static constexpr int SJ = (AS + BS + NW - 1) / NW;
    static constexpr int OPS = AJ + BJ + SJ;                                           // copies per wave and chunk
    static constexpr int A_OFF = 0, B_OFF = BM * 128, S_OFF = B_OFF + BN * 128;
    static constexpr int CHUNK = S_OFF + (AS + BS) * 256, STAGE = KC * CHUNK;
    static constexpr int BYTES = NS * STAGE;
    static_assert(NW * 2 * 16 * NI * 16 * 4 <= BYTES, "staging of C fits the ring");
    static_assert(NW > 1, "the barrier, not only the order of one wave, frees a slot");
    static_assert(OPS * KC * (NS - 1) < 64 && NS >= 2, "vmcnt range");
    static_assert(NI * 16 <= 128 && 128 % (NI * 16) == 0, "a wave's rows of B lie in one 128-row block");
};

// The tile of a block of a product.  Blocks go to the eight XCDs in turn: an XCD x takes the
// x-th eighth of the tiles, in columns of eight tiles of m, so that the blocks
// that run together on one XCD share operand rows in its L2.
__device__ __forceinline__ void tile_of(int block, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int n = tiles_m * tiles_n, x = block & 7, i = block >> 3;
    const int each = n >> 3, rest = n & 7;
    const int t = x * each + min(x, rest) + i;
    const int col = t / (8 * tiles_n), rows = min(8, tiles_m - col * 8), in = t - col * 8 * tiles_n;
    tm = col * 8 + in % rows;
    tn = in / rows;
}

// A tile of C per block: WM x WN waves, each with MI x NI tiles of 16x16.
// Operand rows are staged in LDS, KC chunks of 128 per stage (and barrier), by
// direct-to-LDS copies NS-1 stages ahead; 16-byte segments are XOR-swizzled by (row/2)%8, so
// the 16 rows of an operand read hit distinct banks.
template <int WM, int WN, int MI, int NI, int NS, int KC, bool ROWS>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, int block, int tiles_m, int tiles_n)
{
    using L = GemmTile<WM, WN, MI, NI, NS, KC, ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    tile_of(block, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * L::BM, n0 = tn * L::BN;
    const int nch = (g.K + 127) / 128;
    const uint8_t* abase = g.a + (int64_t)m0 * g.lda;
    const uint8_t* bbase = g.b + (int64_t)n0 * g.ldb;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;

    // byte offsets of this lane's 16-byte segments from the tile's first row
    uint32_t aoff[L::AJ], boff[L::BJ];
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
    // this wave's copies of chunk c into the slot of chunk `at`; tail: the last, shorter chunk, zeros past its end
    auto issue = [&](int at, int c, auto tail) {
        const uint32_t slot = lds0 + (uint32_t)(at / KC % NS) * L::STAGE + (uint32_t)(at % KC) * L::CHUNK;
        const uint8_t *ac = abase + (int64_t)c * 128, *bc = bbase + (int64_t)c * 128;
        auto copy = [&](const uint8_t* base, uint32_t off, int p, uint32_t to) {
            const uint32_t dst = __builtin_amdgcn_readfirstlane(to);
            if constexpr (decltype(tail)::value) {
                const int r = p * 8 + (lane >> 3), sg = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
                dma16(sg < (g.K & 127) ? (const void*)(base + off) : (const void*)&g_zeros[lane], dst);
            } else {
                dma16s(base, off, dst);
            }
        };
#pragma unroll
        for (int j = 0; j < L::AJ; j++) {
            const int p = min(wave + j * L::NW, L::BM / 8 - 1);
            copy(ac, aoff[j], p, slot + L::A_OFF + p * 1024);
        }
#pragma unroll
        for (int j = 0; j < L::BJ; j++) {
            const int p = min(wave + j * L::NW, L::BN / 8 - 1);
            copy(bc, boff[j], p, slot + L::B_OFF + p * 1024);
        }
#pragma unroll
        for (int j = 0; j < L::SJ; j++) {
            const int p = min(wave + j * L::NW, L::AS + L::BS - 1);
            const bool is_a = p < L::AS;
            const float* base = is_a ? g.as + (int64_t)c * g.M : g.bs + (int64_t)c * g.N;
            const int row = is_a ? m0 + p * 64 : n0 + (p - L::AS) * 64;
            dma4s(base, (uint32_t)min(row + lane, (is_a ? g.M : g.N) - 1) * 4u,
                  __builtin_amdgcn_readfirstlane(slot + L::S_OFF + p * 256));
        }
    };

    const int wm = wave / WN, wn = wave % WN;
    const int arow = wm * MI * 16 + (lane & 15), brow = wn * NI * 16 + (lane & 15), kq = lane >> 4;
    // the wave's block scales, a scalar load a chunk ahead: a vector load would
    // wait for the copies issued before it
    typedef const __attribute__((address_space(4))) float* cfloat;
    const cfloat bsp = (cfloat)(uintptr_t)(g.bs + (ROWS ? 0 : (min(n0 + wn * NI * 16, g.N - 1) >> 7) * g.bs_n));
    float bs_next = ROWS || nch == 0 ? 1.0f : bsp[0];
    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // this lane's operand segments: rows 16 apart share the swizzle
    const int sw = (lane >> 1) & 7;
    const int alo = L::A_OFF + arow * 128 + ((kq ^ sw) * 16), ahi = L::A_OFF + arow * 128 + (((4 + kq) ^ sw) * 16);
    const int blo = L::B_OFF + brow * 128 + ((kq ^ sw) * 16), bhi = L::B_OFF + brow * 128 + (((4 + kq) ^ sw) * 16);
    auto frag = [&](const uint8_t* st, int lo, int hi, int tile) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + lo + tile * 2048);
        const uint4 y = *reinterpret_cast<const uint4*>(st + hi + tile * 2048);
        return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };
    // Small wave tiles have all of a chunk's operands in registers, large ones two row tiles of A, or three where
    // the products of one are too few to cover the read of the next (8192x4096x4096 125.5 -> 121.7 us; 64-row
    // wave tiles and row scales lose by it: 2048x4096x8192 86 -> 111).
    constexpr bool SMALL = MI * NI <= 4;
    constexpr int D = MI >= 8 && !ROWS ? 3 : 2;
    v8i af[SMALL && MI > 2 ? MI : D], bf[NI];
    float sa[MI], bs = 1.0f;
    float4 br[ROWS ? NI : 1];
    v4f p[NI];
    // operands that every step of chunk c needs, and its first row tiles
    auto open = [&](int c) {
        const uint8_t* st = smem + (c / KC % NS) * L::STAGE + (c % KC) * L::CHUNK;
#pragma unroll
        for (int i = 0; i < (SMALL ? MI : D - 1); i++) af[i] = frag(st, alo, ahi, i);
#pragma unroll
        for (int j = 0; j < NI; j++) bf[j] = frag(st, blo, bhi, j);
#pragma unroll
        for (int i = 0; i < MI; i++) sa[i] = *reinterpret_cast<const float*>(st + L::S_OFF + (arow + 16 * i) * 4);
        if constexpr (ROWS) {
#pragma unroll
            for (int j = 0; j < NI; j++)
                br[j] = *reinterpret_cast<const float4*>(st + L::S_OFF + L::AS * 256 + (wn * NI * 16 + 16 * j + 4 * kq) * 4);
        } else {
            bs = bs_next;
            bs_next = bsp[min(c + 1, nch - 1) * g.bs_k];
        }
    };
    auto add_to = [&](v4f& a, const v4f& v, float s, float4 r) {
        if constexpr (ROWS) {
            a[0] = fmaf(s * r.x, v[0], a[0]);
            a[1] = fmaf(s * r.y, v[1], a[1]);
            a[2] = fmaf(s * r.z, v[2], a[2]);
            a[3] = fmaf(s * r.w, v[3], a[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) a[e] = fmaf(s, v[e], a[e]);
        }
    };
    auto add = [&](int i, int j, float s, float4 r) { add_to(acc[i][j], p[j], s, r); };
    // Products of chunk c, whose operands open() has begun: row tile i's go out
    // while the previous tile's are added; mid() runs once every operand is in
    // registers, next() once the last products are out.
    // (a small tile reads the next chunk's operands before its own products, which cover their latency)
    auto chunk = [&](int c, auto mid, auto next) {
        if constexpr (SMALL) {
            mid();
            v8i a0[MI], b0[NI];
            float s0[MI];
            float4 r0[ROWS ? NI : 1];
#pragma unroll
            for (int i = 0; i < MI; i++) a0[i] = af[i], s0[i] = sa[i] * bs;
#pragma unroll
            for (int j = 0; j < NI; j++) b0[j] = bf[j];
#pragma unroll
            for (int j = 0; j < (ROWS ? NI : 1); j++) r0[j] = br[j];
            next();
            v4f v[MI][NI];
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) v[i][j] = mfma_e4m3(b0[j], a0[i]);
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) add_to(acc[i][j], v[i][j], s0[i], r0[ROWS ? j : 0]);
            return;
        }
        const uint8_t* st = smem + (c / KC % NS) * L::STAGE + (c % KC) * L::CHUNK;
#pragma unroll
        for (int i = 0; i < MI - 1; i++) {
            if (i + D - 1 < MI) af[(i + D - 1) % D] = frag(st, alo, ahi, i + D - 1);
#pragma unroll
            for (int j = 0; j < NI; j++) {
                if (i > 0) add(i - 1, j, sa[i - 1] * bs, br[ROWS ? j : 0]);
                p[j] = mfma_e4m3(bf[j], af[i % D]);
            }
        }
        mid();
#pragma unroll
        for (int j = 0; j < NI; j++) {
            if (MI > 1) add(MI - 2, j, sa[MI > 1 ? MI - 2 : 0] * bs, br[ROWS ? j : 0]);
            p[j] = mfma_e4m3(bf[j], af[(MI - 1) % D]);
        }
        // (with row scales the last tile is added first: both chunks' would not fit the registers)
        const float last = sa[MI - 1] * bs;
        if (!ROWS) next();
#pragma unroll
        for (int j = 0; j < NI; j++) add(MI - 1, j, last, br[ROWS ? j : 0]);
        if (ROWS) next();
    };
    const std::false_type whole;
    const std::true_type tail;
    const int full = g.K >> 7;
    auto issue_stage = [&](int g0) {
#pragma unroll
        for (int k = 0; k < KC; k++) issue(g0 * KC + k, min(g0 * KC + k, full - 1), whole);
    };
    if (full > 0) {
#pragma unroll
        for (int g0 = 0; g0 < NS; g0++) issue_stage(g0);
        wait_vm<L::OPS * KC * (NS - 1)>();
        __syncthreads();
        open(0);
    }
    // The barrier in a stage's last chunk frees its slot and makes the next stage
    // whole: only copies of later stages are then out.  Copies past the last chunk
    // fetch it again, into slots that are not read any more.
    const int stages = (full + KC - 1) / KC;
    int c = 0;
    for (int g0 = 0; g0 < stages - 1; g0++) {
#pragma unroll
        for (int k = 0; k < KC - 1; k++, c++) chunk(c, []() {}, [&]() { open(c + 1); });
        chunk(c, [&]() { wait_vm<L::OPS * KC * (NS - 2)>(); __syncthreads(); },
              [&]() { issue_stage(g0 + NS); open(c + 1); });
        c++;
    }
    if (KC > 1)
        for (; c < full - 1; c++) chunk(c, []() {}, [&]() { open(c + 1); });
    for (; c < nch; c++) {
        if (c == full) {
            wait_vm<0>();
            __syncthreads();
            issue(c, c, tail);
            wait_vm<0>();
            __syncthreads();
            open(c);
        }
        chunk(c, []() {}, []() {});
    }
    wait_vm<0>();
    __syncthreads();   // every wave is done with the ring: it becomes staging space
    uint8_t* stage = smem + wave * (2 * 16 * NI * 16 * 4);
    const int mw = m0 + wm * MI * 16, nw = n0 + wn * NI * 16;
    constexpr bool STREAM = L::BM * L::BN >= 128 * 128;
    if (!g.c_bf16) store_tile<STREAM, MI, NI, float>(acc, stage, static_cast<float*>(g.c), g, mw, nw);
    else if (g.accumulate) store_tile<STREAM, MI, NI, float>(acc, stage, static_cast<uint16_t*>(g.c), g, mw, nw);
    else store_tile<STREAM, MI, NI, uint16_t>(acc, stage, static_cast<uint16_t*>(g.c), g, mw, nw);
}

template <int WM, int WN, int MI, int NI, int NS, int KC, bool ROWS>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_gemm(GemmArgs g, int tiles_m, int tiles_n)
{
    gemm_tile<WM, WN, MI, NI, NS, KC, ROWS>(g, blockIdx.x, tiles_m, tiles_n);
}
// The two products of a backward in one launch, a's blocks first: block scales
// for the data gradient, row scales for the weights'.
template <int WM, int WN, int MI, int NI, int NS, int KC>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_gemm_pair(GemmArgs a, int am, int an, GemmArgs b, int bm, int bn)
{
    const int n = am * an;
    if ((int)blockIdx.x < n) gemm_tile<WM, WN, MI, NI, NS, KC, false>(a, blockIdx.x, am, an);
    else gemm_tile<WM, WN, MI, NI, NS, KC, true>(b, blockIdx.x - n, bm, bn);
}

// Few rows: the chunks of a tile of (16 MT) x (16 NT) are spread over the NW
// waves of a block, each loading its operands straight into registers, so that
// a block's whole stretch of weights is in flight at once and nothing waits
// for a barrier per chunk.  The chunk sums meet in LDS, where one thread per
// four columns adds them in increasing chunk order: the same operations, and
// so the same bits, as k_fp8_gemm.  X (MT = 1): A is x itself (bf16), each
// chunk quantised by the wave that needs it, in every block: 16 rows cost less
// than a launch of their own.
// Bound by latency: one row by 4096x2048 5.8 us, the 8.4 MB of weights at 1.4 TB/s;
// 16 rows of codes by 4096x4096 6.6 us, 2.5 TB/s.  Longer contractions are held up by
// the rounds, each wave with the operands of one chunk on their way and every round
// with a barrier and the addition of its sums: one row by 4096x8192 14.4 to 15 us, 2.2 TB/s,
// where 33.5 MB of weights would take 5.4 at a copy's rate.
template <int MT, int NT, int NW, bool ROWS, bool X>
struct SplitLds {
    static constexpr int P = 16 * MT * (16 * NT + 4);          // floats of a chunk's products (rows padded)
    static constexpr int S = 16 * MT + (ROWS ? 16 * NT : 0);   // its scales
    static constexpr int BYTES = 2 * NW * (P + S) * 4;         // two rounds
    static_assert(MT * NT * 64 <= NW * 64 && (!X || (MT == 1 && !ROWS)), "a thread per four columns");
    static_assert(NW % 8 == 0, "chunks are added eight at a time");
};
template <int MT, int NT, int NW, bool ROWS, bool X>
__global__ __launch_bounds__(64 * NW) void k_fp8_split(GemmArgs g, const uint16_t* __restrict__ x, int64_t ldx, int kx)
{
    using L = SplitLds<MT, NT, NW, ROWS, X>;
    extern __shared__ __align__(16) float lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
    const int nch = (g.K + 127) / 128;

    const uint8_t* brow[NT];
    const uint8_t* arow[MT];
#pragma unroll
    for (int j = 0; j < NT; j++) brow[j] = g.b + (int64_t)min(n0 + 16 * j + r16, g.N - 1) * g.ldb + 16 * kq;
    if constexpr (!X) {
#pragma unroll
        for (int i = 0; i < MT; i++) arow[i] = g.a + (int64_t)min(m0 + 16 * i + r16, g.M - 1) * g.lda + 16 * kq;
    }
    const uint16_t* xrow = X ? x + (int64_t)min(m0 + r16, g.M - 1) * ldx + 16 * kq : nullptr;

    struct Operands {
        uint4 b[NT][2], a[MT][2], xv[X ? 4 : 1];
        float sa[MT], sb[ROWS ? NT : 1];
    };
    // this lane's segments kq and 4 + kq of chunk c, zeros past the end (by their address: no branch between loads)
    typedef const __attribute__((address_space(1))) v4u* gptr;
    const gptr zeros = (gptr)&g_zeros[lane];
    auto fetch = [&](bool in, const void* p) {
        const gptr q = in ? (gptr)p : zeros;
        const v4u v = *q;
        return make_uint4(v.x, v.y, v.z, v.w);
    };
    // a zero the compiler does not know, so that the block scale is a vector load like the rest and
    // is waited for with them
    int opaque;
    asm("v_mov_b32 %0, 0" : "=v"(opaque));
    auto load = [&](int c, Operands& o) {
        const int left = g.K - c * 128;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const bool in = 64 * h + 16 * kq < left;
#pragma unroll
            for (int j = 0; j < NT; j++) o.b[j][h] = fetch(in, brow[j] + c * 128 + 64 * h);
            if constexpr (X) {
                const int xl = kx - c * 128 - 64 * h - 16 * kq;       // elements of x left (kx a multiple of 8)
#pragma unroll
                for (int u = 0; u < 2; u++)
                    o.xv[2 * h + u] = fetch(8 * u < xl, xrow + c * 128 + 64 * h + 8 * u);
            } else {
#pragma unroll
                for (int i = 0; i < MT; i++) o.a[i][h] = fetch(in, arow[i] + c * 128 + 64 * h);
            }
        }
        if constexpr (!X) {
#pragma unroll
            for (int i = 0; i < MT; i++) o.sa[i] = g.as[(int64_t)c * g.M + min(m0 + 16 * i + r16, g.M - 1)];
        }
#pragma unroll
        for (int j = 0; j < (ROWS ? NT : 1); j++)
            o.sb[j] = ROWS ? g.bs[(int64_t)c * g.N + min(n0 + 16 * j + r16, g.N - 1)]
                           : g.bs[(min(n0, g.N - 1) >> 7) * g.bs_n + c * g.bs_k + opaque];
    };
    auto v8 = [](const uint4& lo, const uint4& hi) {
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const int em = tid / (4 * NT), en = 4 * (tid % (4 * NT));    // this thread's row and first column of the tile
    const bool owner = tid < MT * NT * 64;
    Operands o;
    if (wave < nch) load(wave, o);
    for (int r = 0; r * NW < nch; r++) {
        const int c = r * NW + wave;
        float* slot = lds + ((r & 1) * NW + wave) * (L::P + L::S);
        if (c < nch) {
            v8i a[MT], b[NT];
            float s[MT];
            if constexpr (X) {
                float f[32];
                uint32_t m = 0;
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const uint32_t q[4] = {o.xv[u].x, o.xv[u].y, o.xv[u].z, o.xv[u].w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        f[8 * u + 2 * e] = bf16_to_f32(q[e] & 0xFFFFu);
                        f[8 * u + 2 * e + 1] = bf16_to_f32(q[e] >> 16);
                        m = max(m, max(mag_bits(f[8 * u + 2 * e]), mag_bits(f[8 * u + 2 * e + 1])));
                    }
                }
                m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32));
                const Divisor d(group_scale(m));
                s[0] = d.s;
#pragma unroll
                for (int u = 0; u < 8; u++) a[0][u] = (int)d.codes4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < MT; i++) a[i] = v8(o.a[i][0], o.a[i][1]), s[i] = o.sa[i];
            }
#pragma unroll
            for (int j = 0; j < NT; j++) b[j] = v8(o.b[j][0], o.b[j][1]);
            if (kq == 0) {
#pragma unroll
                for (int i = 0; i < MT; i++) slot[L::P + 16 * i + r16] = ROWS ? s[i] : s[i] * o.sb[0];
                if constexpr (ROWS) {
#pragma unroll
                    for (int j = 0; j < NT; j++) slot[L::P + 16 * MT + 16 * j + r16] = o.sb[j];
                }
            }
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const v4f p = mfma_e4m3(b[j], a[i]);
                    *reinterpret_cast<float4*>(slot + (16 * i + r16) * (16 * NT + 4) + 16 * j + 4 * kq) =
                        make_float4(p[0], p[1], p[2], p[3]);
                }
            if (c + NW < nch) load(c + NW, o);
        }
        __syncthreads();     // (two rounds' slots: a round is read before its slots are written again)
        if (owner) {
            const float* p = lds + (r & 1) * NW * (L::P + L::S);
            auto add = [&](float4 v, float s, float4 b) {
                if constexpr (ROWS) {
                    acc[0] = fmaf(s * b.x, v.x, acc[0]);
                    acc[1] = fmaf(s * b.y, v.y, acc[1]);
                    acc[2] = fmaf(s * b.z, v.z, acc[2]);
                    acc[3] = fmaf(s * b.w, v.w, acc[3]);
                } else {
                    acc[0] = fmaf(s, v.x, acc[0]);
                    acc[1] = fmaf(s, v.y, acc[1]);
                    acc[2] = fmaf(s, v.z, acc[2]);
                    acc[3] = fmaf(s, v.w, acc[3]);
                }
            };
            auto product = [&](int w) {
                return *reinterpret_cast<const float4*>(p + w * (L::P + L::S) + em * (16 * NT + 4) + en);
            };
            auto scale = [&](int w) { return p[w * (L::P + L::S) + L::P + em]; };
            auto rows = [&](int w) {
                return ROWS ? *reinterpret_cast<const float4*>(p + w * (L::P + L::S) + L::P + 16 * MT + en) : float4{};
            };
            const int n = nch - r * NW;
            if (n >= NW) {
                // eight chunks' values read together: an add then waits for none of its own
#pragma unroll
                for (int w0 = 0; w0 < NW; w0 += 8) {
                    float4 v[8], b[8];
                    float s[8];
#pragma unroll
                    for (int w = 0; w < 8; w++) v[w] = product(w0 + w), s[w] = scale(w0 + w), b[w] = rows(w0 + w);
#pragma unroll
                    for (int w = 0; w < 8; w++) add(v[w], s[w], b[w]);
                }
            } else {
                for (int w = 0; w < n; w++) add(product(w), scale(w), rows(w));
            }
        }
    }
    const int m = m0 + em, n = n0 + en;
    if (!owner || m >= g.M) return;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if (n + e >= g.N) break;
        if (g.c_bf16) {
            uint16_t* o = static_cast<uint16_t*>(g.c) + (int64_t)m * g.ldc + n + e;
            *o = (uint16_t)bf16x2(g.accumulate ? bf16_to_f32(*o) + acc[e] : acc[e], 0.0f);
        } else {
            float* o = static_cast<float*>(g.c) + (int64_t)m * g.ldc + n + e;
            *o = g.accumulate ? *o + acc[e] : acc[e];
        }
    }
}

inline int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }
inline int64_t chunks(int64_t v) { return (v + 127) / 128; }

template <typename T>
hipError_t launch_quant(int mode, int R, int C, const T* x, int64_t ldx, uint8_t* q, int64_t ldq, float* s, uint8_t* qt,
                        int64_t ldqt, float* st, hipStream_t stream)
{
    if (mode == kQuantRows) {
        // groups of a row in a block: a power of two up to eight
        const int lg = chunks(C) >= 8 ? 3 : chunks(C) >= 4 ? 2 : chunks(C) >= 2 ? 1 : 0, per = 32 >> lg;
        const dim3 grid((unsigned)((R + per - 1) / per), (unsigned)((chunks(C) + (1 << lg) - 1) >> lg));
        hipLaunchKernelGGL(k_fp8_quant_rows<T>, grid, dim3(256), 0, stream, R, C, lg, x, ldx, q, ldq, s);
        return hipGetLastError();
    }
    const QuantJob<T> job{R, C, x, ldx, q, ldq, s, qt, ldqt, st};
    auto run = [&](auto m) {
        hipLaunchKernelGGL((k_fp8_quant<T, decltype(m)::value>), dim3((unsigned)job.tiles()), dim3(kQuantThreads), 0, stream,
                           job);
    };
    switch (mode) {
    case kQuantCols: run(std::integral_constant<int, kQuantCols>{}); break;
    case kQuantRows | kQuantCols: run(std::integral_constant<int, kQuantRows | kQuantCols>{}); break;
    default: run(std::integral_constant<int, kQuantBlock>{}); break;
    }
    return hipGetLastError();
}

// dy and x of a backward, of one type; rows: dy's codes by rows too
template <typename T>
hipError_t launch_quant_pair(const QuantJob<T>& dy, const QuantJob<T>& x, bool rows, hipStream_t stream)
{
    const int a = dy.tiles(), b = x.tiles();
    if ((int64_t)a + b > INT32_MAX) return hipErrorInvalidValue;
    if (rows)
        hipLaunchKernelGGL((k_fp8_quant_pair<T, kQuantRows | kQuantCols>), dim3((unsigned)(a + b)), dim3(kQuantThreads), 0,
                           stream, dy, a, x);
    else
        hipLaunchKernelGGL((k_fp8_quant_pair<T, kQuantCols>), dim3((unsigned)(a + b)), dim3(kQuantThreads), 0, stream, dy, a,
                           x);
    return hipGetLastError();
}

hipError_t run_quant(int mode, int R, int C, const void* x, int type, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                     uint8_t* qt, int64_t ldqt, float* st, hipStream_t stream)
{
    if (type == V4MOE_TYPE_F32)
        return launch_quant(mode, R, C, static_cast<const float*>(x), ldx, q, ldq, s, qt, ldqt, st, stream);
    return launch_quant(mode, R, C, static_cast<const uint16_t*>(x), ldx, q, ldq, s, qt, ldqt, st, stream);
}

// Lets a kernel have more than 64 KiB of LDS, once per device (or again by host threads that come to it at once).
using LdsAllowed = std::atomic<bool>[kMaxDevices];
hipError_t allow_lds(const void* kernel, int bytes, LdsAllowed& done)
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

template <int WM, int WN, int MI, int NI, int NS, int KC, bool ROWS>
hipError_t launch_gemm(const GemmArgs& g, hipStream_t s)
{
    using L = GemmTile<WM, WN, MI, NI, NS, KC, ROWS>;
    const auto kernel = k_fp8_gemm<WM, WN, MI, NI, NS, KC, ROWS>;
    static LdsAllowed allowed;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const int tm = (g.M + L::BM - 1) / L::BM, tn = (g.N + L::BN - 1) / L::BN;
    if ((int64_t)tm * tn > INT32_MAX / 8) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(64 * L::NW), L::BYTES, s, g, tm, tn);
    return hipGetLastError();
}

template <int MT, int NT, int NW, bool ROWS, bool X>
hipError_t launch_split(const GemmArgs& g, hipStream_t s, const uint16_t* x = nullptr, int64_t ldx = 0, int kx = 0)
{
    using L = SplitLds<MT, NT, NW, ROWS, X>;
    const auto kernel = k_fp8_split<MT, NT, NW, ROWS, X>;
    static LdsAllowed allowed;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    const dim3 grid((unsigned)((g.N + 16 * NT - 1) / (16 * NT)), (unsigned)((g.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * NW), L::BYTES, s, g, x, ldx, kx);
    return hipGetLastError();
}

// The product's variants.  A call takes the one of the least time in this table,
// by the rounds its tiles make (a round is one tile per CU): microseconds at
// K = 4096, N = 4096 and M = 16 .. 8192, in a graph of many calls.  Times are nearly
// proportional to K, so the order holds for others; two blocks of the tiles up to
// 128x128 share a CU, so that a second round costs less than the first.  Rounds that
// come from N instead read weights of their own, and from memory where no cache holds
// them, which the table does not know: one row by 16384x4096, one round of 16x64 tiles,
// takes 16.5 us (67 MB, 4.1 TB/s), 16 rows by 7168x4096 11.5.
//                 rounds:  1       2      3      4     each further
//   k_fp8_split   16x16     6.6    10.2   14.0   17.8   3.7
//   k_fp8_gemm    16x64     9.2    12.3   16.0   20.3   4.0
//                 32x64    10.2    13.2   17.4   22.5   4.2
//                 64x64    12.5    15.7   24.6   29.1   8.4
//                 128x128  23      34     52     73     19
//                 256x256  58      124    186    248    62
// (Tiles between them were timed and lie on or above the line these make: 128x64
// at 512x4096x4096 17.8 us next to 15.8, at 1024x4096x4096 23.9 next to 24.1;
// 128x256 at 2048x4096x8192 83.5 next to 84.6.)
// What bounds them: the small tiles the bytes of their operands through a CU's
// vector memory path (the 32x64 tiles of 128x4096x4096 move 0.4 MB a CU in about 7
// of their 10 us; deeper rings, two to four chunks a stage and scales through
// LDS left that as it was), the large ones the matrix pipe next to the copies.
// At 8192x4096x4096 (122 us in a long run of launches, 2.25 PFLOP/s; 129 to 160 in the
// first tens of milliseconds of load, at lower clocks; matrix pipe half busy)
// copies of the kernel that leave work out take, of 128 us with two row tiles of A
// in registers: no stores of C 115 us, no copies into LDS 104, no scaling of the
// chunk sums 116, neither 87, and without operand reads too 81 us, which is the
// products (65 us at the pipe's rate) and the ends of the tiles.  64x64 takes two chunks a stage (one: 13.1 / 18.8 / 32.3 us).
struct Variant {
    int bm, bn;
    float us[4], further;
};
constexpr Variant kVariants[] = {
    {16, 16, {6.6f, 10.2f, 14.0f, 17.8f}, 3.7f},   {16, 64, {9.2f, 12.3f, 16.0f, 20.3f}, 4.0f},
    {32, 64, {10.2f, 13.2f, 17.4f, 22.5f}, 4.2f},  {64, 64, {12.5f, 15.7f, 24.6f, 29.1f}, 8.4f},
    {128, 128, {23.0f, 34.0f, 52.0f, 73.0f}, 19.0f}, {256, 256, {58.0f, 124.0f, 186.0f, 248.0f}, 62.0f}};
int64_t tiles_of(const Variant& k, int64_t M, int64_t N) { return ((M + k.bm - 1) / k.bm) * ((N + k.bn - 1) / k.bn); }
float time_of(const Variant& k, int64_t tiles)
{
    const int64_t rounds = (tiles + 255) / 256;
    return rounds <= 4 ? k.us[rounds - 1] : k.us[3] + k.further * (float)(rounds - 4);
}
int choose_variant(int64_t M, int64_t N)
{
    int best = 0;
    float least = 0.0f;
    for (int v = 0; v < 6; v++) {
        const float us = time_of(kVariants[v], tiles_of(kVariants[v], M, N));
        if (v == 0 || us < least) best = v, least = us;
    }
    return best;
}

template <bool ROWS>
hipError_t run_gemm(const GemmArgs& g, hipStream_t s)
{
    switch (choose_variant(g.M, g.N)) {
    case 0: return launch_split<1, 1, 8, ROWS, false>(g, s);
    case 1: return launch_gemm<1, 4, 1, 1, 4, 1, ROWS>(g, s);
    case 2: return launch_gemm<2, 2, 1, 2, 4, 1, ROWS>(g, s);
    case 3: return launch_gemm<2, 2, 2, 2, 2, 2, ROWS>(g, s);
    case 4: // with row scales four waves of 64x64 take 250 registers: eight of 64x32 (115) run ahead further
        // (2048x2048x4096 27.6 -> 25.3 us; without, 8192x4096x2048 73.3 -> 79.7)
        if constexpr (ROWS) return launch_gemm<2, 4, 4, 2, 2, 1, ROWS>(g, s);
        else return launch_gemm<2, 2, 4, 4, 2, 1, ROWS>(g, s);
    default: return launch_gemm<2, 4, 8, 4, 2, 1, ROWS>(g, s);
    }
}

template <int WM, int WN, int MI, int NI, int NS, int KC>
hipError_t launch_gemm_pair(const GemmArgs& a, const GemmArgs& b, hipStream_t s)
{
    using L = GemmTile<WM, WN, MI, NI, NS, KC, true>;          // (the larger LDS of the two)
    const auto kernel = k_fp8_gemm_pair<WM, WN, MI, NI, NS, KC>;
    static LdsAllowed allowed;
    if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::BYTES, allowed); e != hipSuccess) return e;
    auto over = [](int n, int b) { return (n + b - 1) / b; };
    const int am = over(a.M, L::BM), an = over(a.N, L::BN), bm = over(b.M, L::BM), bn = over(b.N, L::BN);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(am * an + bm * bn)), dim3(64 * L::NW), L::BYTES, s, a, am, an, b, bm, bn);
    return hipGetLastError();
}

// A backward's products (block scales, row scales): in one launch of one of the
// small tiles where the table has that shorter, the contractions weighing in: one
// product's last round is then filled by the other's tiles, and a launch falls
// away (1237x1999x1001, 320 and 512 tiles of 64x64: 13.4 + 10.6 us apart, 20.9
// together, and 33.8 -> 29.9 of the whole call).
hipError_t run_gemm_pair(const GemmArgs& a, const GemmArgs& b, hipStream_t s)
{
    auto alone = [](const GemmArgs& g) {
        const Variant& k = kVariants[choose_variant(g.M, g.N)];
        return time_of(k, tiles_of(k, g.M, g.N)) * (float)g.K;
    };
    float least = alone(a) + alone(b);
    int best = 0;
    for (int v = 1; v <= 3; v++) {
        const int64_t na = tiles_of(kVariants[v], a.M, a.N), nb = tiles_of(kVariants[v], b.M, b.N);
        const float us = time_of(kVariants[v], na + nb) * (float)((double)(na * a.K + nb * b.K) / (double)(na + nb));
        if (us < least) best = v, least = us;
    }
    switch (best) {
    case 1: return launch_gemm_pair<1, 4, 1, 1, 4, 1>(a, b, s);
    case 2: return launch_gemm_pair<2, 2, 1, 2, 4, 1>(a, b, s);
    case 3: return launch_gemm_pair<2, 2, 2, 2, 2, 2>(a, b, s);
    }
    if (const hipError_t e = run_gemm<false>(a, s); e != hipSuccess) return e;
    return run_gemm<true>(b, s);
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
GemmArgs gemm_args(const v4moe_gemm& p, const uint8_t* a, const float* as, const uint8_t* b, const float* bs, void* c)
{
    return GemmArgs{p.M, p.N, p.K, a, p.lda, as, b, p.ldb, bs, p.bs_n, p.bs_k, c, p.ldc,
                    p.c_type == V4MOE_TYPE_BF16, p.accumulate != 0};
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
    const GemmArgs g = gemm_args(*p, a, as, b, bs, c);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = p->b_scale == V4MOE_SCALE_ROW ? run_gemm<true>(g, s) : run_gemm<false>(g, s);
    return e == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
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
    const int K16 = (int)up16(K), y_bf16 = y_type == V4MOE_TYPE_BF16;
    if (x_type == V4MOE_TYPE_BF16 && K % 8 == 0 && ldx % 8 == 0 && aligned_to(x, 16) && choose_variant(M, N) == 0) {
        // few rows: the product quantises x itself
        if (!device_ready()) return V4MOE_EDEVICE;
        const GemmArgs g{M, N, K16, nullptr, 0, nullptr, w->q, K16, w->blk, chunks(K), 1, y, ldy, y_bf16, 0};
        const hipStream_t s = static_cast<hipStream_t>(stream);
        const uint16_t* xb = static_cast<const uint16_t*>(x);
        // Sixteen waves (and chunks) at a time where a CU has one tile and more than eight chunks to do: one row by
        // 4096x2048 5.8 us (eight waves: 6.5), by 4096x4096 8.7 (10.5), by 4096x8192 14.4 (19.2).  Two tiles a CU
        // (which this variant is chosen for where N is at most 16 and the rows are 4112 to 8192) gain by eight:
        // 8192 rows by 16x2048 11.5 us (sixteen waves: 13.4), by 16x4096 17.9 (21.4).
        const bool many = chunks(K) > 8 && tiles_of(kVariants[0], M, N) <= 256;
        const hipError_t e = many ? launch_split<1, 1, 16, false, true>(g, s, xb, ldx, K)
                                  : launch_split<1, 1, 8, false, true>(g, s, xb, ldx, K);
        return e == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* xs = reinterpret_cast<float*>(ws + L.xs);
    if (const int rc = moe_fp8_quantize(M, K, x, x_type, ldx, ws + L.xq, xs, nullptr, nullptr, stream)) return rc;
    const v4moe_gemm g{M, N, K16, V4MOE_SCALE_BLOCK, y_type, 0, K16, K16, ldy, chunks(K), 1};
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
    if (M > 0 && dw) {
        // both operands' columns, and dy's rows, in one launch where they are of one type
        const bool one = x_type == dy_type;
        if (!device_ready()) return V4MOE_EDEVICE;
        const hipStream_t s = static_cast<hipStream_t>(stream);
        auto both = [&](auto* as) {
            using T = std::remove_pointer_t<decltype(as)>;
            const QuantJob<T> a{M, N, static_cast<const T*>(dy), lddy, ws + L.dq, up16(N), f32(L.ds),
                                ws + L.dt, up16(M), f32(L.dts)};
            const QuantJob<T> b{M, K, static_cast<const T*>(x), ldx, nullptr, 0, nullptr, ws + L.xt, up16(M), f32(L.xts)};
            return launch_quant_pair(a, b, dx != nullptr, s);
        };
        if (one) {
            const hipError_t e =
                x_type == V4MOE_TYPE_F32 ? both(static_cast<float*>(nullptr)) : both(static_cast<uint16_t*>(nullptr));
            if (e != hipSuccess) return V4MOE_ELAUNCH;
        } else {
            if (const int rc = moe_fp8_quantize(M, N, dy, dy_type, lddy, dx ? ws + L.dq : nullptr, dx ? f32(L.ds) : nullptr,
                                                ws + L.dt, f32(L.dts), stream))
                return rc;
            if (const int rc = moe_fp8_quantize(M, K, x, x_type, ldx, nullptr, nullptr, ws + L.xt, f32(L.xts), stream))
                return rc;
        }
    } else if (M > 0) {
        if (const int rc = moe_fp8_quantize(M, N, dy, dy_type, lddy, ws + L.dq, f32(L.ds), nullptr, nullptr, stream))
            return rc;
    }
    // dx = dy W: contraction over N, block (i, c) of W^T is block (c, i) of W
    const v4moe_gemm gx{M, K, (int32_t)up16(N), V4MOE_SCALE_BLOCK, dx_type, 0, up16(N), up16(N), lddx, 1, chunks(K)};
    // dW = dy^T x: contraction over the tokens, both scales per row
    const v4moe_gemm gw{N, K, (int32_t)up16(M), V4MOE_SCALE_ROW, dw_type, accumulate, up16(M), up16(M), lddw, 0, 0};
    if (dx && dw && M > 0) {
        const GemmArgs a = gemm_args(gx, ws + L.dq, f32(L.ds), w->qt, w->blk, dx);
        const GemmArgs b = gemm_args(gw, ws + L.dt, f32(L.dts), ws + L.xt, f32(L.xts), dw);
        return run_gemm_pair(a, b, static_cast<hipStream_t>(stream)) == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
    }
    if (dx && M > 0) return moe_fp8_gemm(&gx, ws + L.dq, f32(L.ds), w->qt, w->blk, dx, stream);
    if (dw && (M > 0 || !accumulate))      // (adding a sum of nothing would turn -0 into 0)
        return moe_fp8_gemm(&gw, ws + L.dt, f32(L.dts), ws + L.xt, f32(L.xts), dw, stream);
    return V4MOE_OK;
}

}  // extern "C"
