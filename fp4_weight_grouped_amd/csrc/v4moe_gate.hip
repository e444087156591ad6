// v4moe_gate.hip -- routing from given logits, and its gradient.
//
// Per token, with z the logits (masked: NaN or <= -1e30; capped at 1e30):
//   s_e   = 1 / (1 + exp(-z)) | exp(z - max) / sum | sqrt(max(z, 0) + log1p(exp(-|z|)))
//   key_e = s_e + bias_e, -inf for masked experts and NaN
//   a group's value is the sum of its two largest keys that are not -inf; the
//   topk_groups largest groups stay, ties to the lower group; the topk largest
//   keys of those are picked in order, ties to the lower id
//   w_j   = scale * s_j [/ sum of the picked s], 0 where the key is -inf
// Scores and keys are fp32, every operation rounded once (the library is built
// without contraction), so the picks are a function of the logits alone.  The
// softmax's sum is taken in fp64, over neighbours, their pairs and so on, which
// is the same tree however many lanes a token has.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace v4moe {

namespace {

constexpr float kMask = 1e30f;
constexpr float kInf = __builtin_inff();

// EPL consecutive logits of a row from expert e0 on, -inf past E: one access
// where the row has them all (at any element's address).
template <typename T, int EPL>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, float (&z)[EPL])
{
    typedef T vec __attribute__((ext_vector_type(EPL)));
    typedef vec vec_any __attribute__((aligned(sizeof(T))));
    auto f32 = [](T v) {
        if constexpr (sizeof(T) == 4) return (float)v;
        else return bf16_to_f32(v);
    };
    if (e0 + EPL <= E) {
        const vec v = *reinterpret_cast<const vec_any*>(row + e0);
#pragma unroll
        for (int q = 0; q < EPL; q++) z[q] = f32(v[q]);
    } else {
#pragma unroll
        for (int q = 0; q < EPL; q++) z[q] = e0 + q < E ? f32(row[e0 + q]) : -kInf;
    }
}
template <typename T, int EPL>
__device__ __forceinline__ void store_logits(T* row, int e0, int E, const float (&z)[EPL])
{
    typedef T vec __attribute__((ext_vector_type(EPL)));
    typedef vec vec_any __attribute__((aligned(sizeof(T))));
    vec v;
#pragma unroll
    for (int q = 0; q < EPL; q++) {
        if constexpr (sizeof(T) == 4) v[q] = z[q];
        else v[q] = (T)bf16x2(z[q], 0.0f);
    }
    if (e0 + EPL <= E) {
        *reinterpret_cast<vec_any*>(row + e0) = v;
    } else {
#pragma unroll
        for (int q = 0; q < EPL; q++)
            if (e0 + q < E) row[e0 + q] = v[q];
    }
}

// -inf for a masked logit, and for NaN
__device__ __forceinline__ float clean(float z) { return z > -kMask ? fminf(z, kMask) : -kInf; }

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))); }
__device__ __forceinline__ float sqrt_softplus(float z) { return sqrtf(softplus(z)); }

// One step of a reduction over lanes: v as lane pattern CTRL brings it (DPP),
// `none` where it brings nothing.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false);
}
// Sum over the 16 lanes of a row, in every one of them.
__device__ __forceinline__ float row_sum(float v)
{
    auto add = [&](uint32_t o) { v += __uint_as_float(o); };
    add(dpp<0xB1>(0, __float_as_uint(v)));
    add(dpp<0x4E>(0, __float_as_uint(v)));
    add(dpp<0x141>(0, __float_as_uint(v)));
    add(dpp<0x140>(0, __float_as_uint(v)));
    return v;
}
// Order-preserving map of floats (no NaN) to unsigned integers; -inf is kNone.
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_of(float f)
{
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }

// Maximum over the LPT lanes of a token, in every one of them: the rows of 16
// by DPP, then rows by permutes that swap them (16 and 32 lanes apart).
template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v)
{
    v = max(v, dpp<0xB1>(0, v));
    v = max(v, dpp<0x4E>(0, v));
    v = max(v, dpp<0x141>(0, v));
    v = max(v, dpp<0x140>(0, v));
    if constexpr (LPT >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(a[0], a[1]);
    }
    if constexpr (LPT >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(a[0], a[1]);
    }
    return v;
}
// ... their sum
template <int LPT>
__device__ __forceinline__ float token_sum(float v)
{
    v = row_sum(v);
    if constexpr (LPT >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if constexpr (LPT >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ double token_sum(double v)
{
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o);
    return v;
}
// The lowest set bit of each token's LPT bits.
template <int LPT>
__device__ __forceinline__ uint64_t first_of(uint64_t m)
{
    if constexpr (LPT == 64) {
        return m & (0 - m);
    } else {
        uint64_t r = 0;
#pragma unroll
        for (int i = 0; i < 64; i += LPT) {
            const uint32_t f = (uint32_t)(m >> i) & (uint32_t)((1ull << LPT) - 1);
            r |= (uint64_t)(f & (0u - f)) << i;
        }
        return r;
    }
}

// Sorts N values downwards (Batcher's odd-even merges).
template <int N>
__device__ __forceinline__ void sort_down(uint64_t (&k)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int d = p; d >= 1; d /= 2)
#pragma unroll
            for (int j = d % p; j + d < N; j += 2 * d)
#pragma unroll
                for (int i = 0; i < d; i++) {
                    const int x = i + j, y = x + d;
                    if (y < N && x / (2 * p) == y / (2 * p)) {
                        // (as a mask: one comparison, where the compiler would take a maximum and a minimum)
                        const bool swap = __builtin_amdgcn_inverse_ballot_w64(__ballot(k[y] > k[x]));
                        const uint64_t hi = swap ? k[y] : k[x], lo = swap ? k[x] : k[y];
                        k[x] = hi;
                        k[y] = lo;
                    }
                }
}

// LPT lanes per token (64 / LPT tokens per wave); a token's lane l holds experts
// l EPL .. + EPL - 1, so that of equal keys the lowest lane has the lowest id.
// Each lane sorts its keys once, into LDS; a round takes the maximum over the
// token's lanes, and the first lane that has it notes the expert and reads its next.
// The groups' two largest keys are found by LPT / groups lanes each: the lanes
// that hold them where the experts fill the token's lanes and the groups are a
// power of two, otherwise over keys staged in LDS, as groups need not end with a
// lane.  Bound by the instructions a token takes, for a sigmoid half of them the
// exponentials and divisions of its scores: T = 8192, E = 256, top-8 of four of
// eight groups 8.5 us in a run of calls, 9.2 alone, where its 8.9 MB would take 2 (rescanning a lane's keys
// after each pick, and one token a wave, 10.7; lists in registers 9.3).
template <typename T, int EPL, int LPT>
__global__ __launch_bounds__(256) void k_gate(v4moe_gate g, const T* __restrict__ logits, int64_t ld,
                                              const float* __restrict__ bias, int32_t* __restrict__ ids,
                                              float* __restrict__ w)
{
    constexpr int TOK = 64 / LPT, MAXE = EPL * LPT;
    __shared__ __align__(16) uint32_t staged_[4][TOK][MAXE];     // keys, then scores
    __shared__ uint32_t values_[4][TOK][LPT];                    // of the groups
    __shared__ uint32_t lists_[4][64][EPL + 1];                  // each lane's keys in order
    __shared__ int32_t picks_[4][TOK][16];
    const int lane = threadIdx.x & (LPT - 1), tok = (threadIdx.x & 63) / LPT;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), t0 = (blockIdx.x * 4 + wave) * TOK;
    if (t0 >= g.T) return;
    const int t = min(t0 + tok, g.T - 1);               // (past the last token: it again, not stored)
    auto& staged = staged_[wave][tok];
    auto& values = values_[wave][tok];
    auto& picks = picks_[wave][tok];
    const int e0 = lane * EPL;
    float s[EPL];
    uint32_t key[EPL];
    load_logits<T, EPL>(logits + (int64_t)t * ld, e0, g.E, s);
    float b[EPL];                                        // what the selection adds: -inf where the logit is masked
#pragma unroll
    for (int q = 0; q < EPL; q++) b[q] = 0.0f;
    if (bias) load_logits<float, EPL>(bias, e0, g.E, b);
#pragma unroll
    for (int q = 0; q < EPL; q++) {
        s[q] = clean(s[q]);
        if (s[q] == -kInf) b[q] = -kInf;
    }
    if (g.score == V4MOE_SCORE_SOFTMAX) {
        uint32_t best = kNone;
#pragma unroll
        for (int q = 0; q < EPL; q++) best = max(best, order_of(s[q]));
        best = token_max<LPT>(best);
        const float m = best == kNone ? 0.0f : float_of(best);
        // (pairs of neighbours, their pairs, ...: the same sums however the experts lie over the lanes)
        double p[EPL];
#pragma unroll
        for (int q = 0; q < EPL; q++) {
            s[q] = expf(s[q] - m);
            p[q] = (double)s[q];
        }
#pragma unroll
        for (int d = 1; d < EPL; d *= 2)
#pragma unroll
            for (int q = 0; q < EPL; q += 2 * d) p[q] += p[q + d];
        const float total = (float)token_sum<LPT>(p[0]);
#pragma unroll
        for (int q = 0; q < EPL; q++) s[q] = total > 0.0f ? s[q] / total : 0.0f;
    } else if (g.score == V4MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int q = 0; q < EPL; q++) s[q] = sigmoid(s[q]);
    } else {
#pragma unroll
        for (int q = 0; q < EPL; q++) s[q] = sqrt_softplus(s[q]);
    }
#pragma unroll
    for (int q = 0; q < EPL; q++) key[q] = order_of(fmaxf(s[q] + b[q], -kInf));      // (NaN: -inf)
    if (g.groups > 1) {
        const int size = g.E / g.groups;
        // 2^shift lanes per group, the group's two largest keys in each of them
        const int shift = __builtin_ctz(LPT) - (32 - __builtin_clz(g.groups - 1)), per = 1 << shift;
        const int mine = lane >> shift;
        uint32_t a = kNone, c = kNone;              // largest and second
        auto merge = [&](uint32_t oa, uint32_t oc) {
            c = max(min(a, oa), max(c, oc));
            a = max(a, oa);
        };
        const bool own = g.E == MAXE && (g.groups & (g.groups - 1)) == 0;      // those lanes hold the group's keys
        if (own) {
#pragma unroll
            for (int q = 0; q < EPL; q++) merge(key[q], kNone);
        } else {
            // lane i of them takes the group's keys i, i + 2^shift, ... out of LDS
#pragma unroll
            for (int q = 0; q < EPL; q++) staged[e0 + q] = key[q];
            __builtin_amdgcn_wave_barrier();
            if (mine < g.groups)
                for (int i = lane & (per - 1); i < size; i += per) merge(staged[mine * size + i], kNone);
        }
        if (per > 1) merge(dpp<0xB1>(kNone, a), dpp<0xB1>(kNone, c));
        if (per > 2) merge(dpp<0x4E>(kNone, a), dpp<0x4E>(kNone, c));
        if (per > 4) merge(dpp<0x141>(kNone, a), dpp<0x141>(kNone, c));
        if (per > 8) merge(dpp<0x140>(kNone, a), dpp<0x140>(kNone, c));
        if (per > 16) merge((uint32_t)__shfl_xor((int)a, 16), (uint32_t)__shfl_xor((int)c, 16));
        const uint32_t v = c == kNone ? a : order_of(float_of(a) + float_of(c));
        if ((lane & (per - 1)) == 0) values[mine] = v;
        __builtin_amdgcn_wave_barrier();
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < g.groups; o++)
            rank += values[o] >= v + (o < mine ? 0u : 1u) ? 1 : 0;      // larger, or as large with a lower number
        const bool keep = mine < g.groups && rank < g.topk_groups;
        if (own) {
            if (!keep) {
#pragma unroll
                for (int q = 0; q < EPL; q++) key[q] = kNone;
            }
        } else {
            const uint64_t kept = __ballot(keep) >> (tok * LPT);
            const float inv = 1.0f / (float)size;
#pragma unroll
            for (int q = 0; q < EPL; q++) {
                // (e0 + q) / size: exact below 2^20
                const int group = min((int)(((float)(e0 + q) + 0.5f) * inv), g.groups - 1);
                if (!((kept >> (group << shift)) & 1)) key[q] = kNone;
            }
        }
    }
    // the lane's keys in order, with EPL - 1 - q below each: of equal ones the lowest expert is the largest
    uint64_t list[EPL];
#pragma unroll
    for (int q = 0; q < EPL; q++) {
        list[q] = (uint64_t)key[q] << 32 | (uint32_t)(EPL - 1 - q);
        staged[e0 + q] = __float_as_uint(s[q]);
    }
    sort_down(list);
    std::conditional_t<(EPL > 8), uint64_t, uint32_t> order = 0;        // the q of each, four bits
    uint32_t* next = lists_[wave][threadIdx.x & 63];
#pragma unroll
    for (int q = 0; q < EPL; q++) {
        order |= (decltype(order))(EPL - 1 - (uint32_t)list[q]) << (4 * q);
        next[q] = (uint32_t)(list[q] >> 32);
    }
    next[EPL] = kNone;
    uint32_t best = (uint32_t)(list[0] >> 32), taken = 0;
    int picked = 0;
    for (int j = 0; j < g.topk; j++) {
        const uint32_t m = token_max<LPT>(best);
        const uint64_t hit = __ballot(best == m && m != kNone);
        if (hit == 0) break;
        if (m != kNone) picked = j + 1;
        if (__builtin_amdgcn_inverse_ballot_w64(first_of<LPT>(hit))) {
            const uint32_t q = (uint32_t)order & 15;
            best = *++next;
            order >>= 4;
            picks[j] = e0 + (int)q;
            taken |= 1u << q;
        }
    }
    // fewer unmasked experts than slots: the lowest others, weight 0
    if (__ballot(picked < g.topk)) {
        for (int j = 0; j < g.topk; j++) {
            const uint32_t open = ~taken & ((1u << EPL) - 1);
            const int q = open ? __builtin_ctz(open) : EPL;
            const uint64_t hit = __ballot(j >= picked && q < EPL && e0 + q < g.E);
            if (__builtin_amdgcn_inverse_ballot_w64(first_of<LPT>(hit))) {
                picks[j] = e0 + q;
                taken |= 1u << q;
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
    int my_e = 0;
    float my_s = 0.0f;
    if (lane < g.topk) {
        my_e = picks[lane];
        if (lane < picked) my_s = __uint_as_float(staged[my_e]);
    }
    const float sum = g.renorm ? row_sum(my_s) : 1.0f;       // (topk <= 16: lanes past it hold 0)
    if (lane < g.topk && t0 + tok < g.T) {
        ids[(int64_t)t * g.topk + lane] = my_e;
        w[(int64_t)t * g.topk + lane] = (sum > 0.0f ? my_s / sum : 0.0f) * g.scale;
    }
}

// Gradient with respect to the logits.  A slot of weight zero (a filler, or a
// score that underflowed) has none.  With u_j = s_j / S renormalised (S the sum of
// the live s), s_j otherwise, and f the score's logarithmic derivative,
//   dz_j = scale d_j u_j f(z_j),  d_j = sum_i u_i (dw_j - dw_i) renormalised, dw_j otherwise,
//   f = 1 / (1 + exp(z)) | sigmoid(z) / (2 softplus(z)) | 1, the softmax's other part
//       -p_e sum_j scale d_j p_j at every logit.
// Shares are formed first and the score itself is never divided by: S and s may lie
// below fp32's normal numbers (a sigmoid's row of logits near -88) where the weights
// and the gradient do not.  For a softmax the last sum is zero where the weights are
// renormalised, which leaves only the picked logits and, as p_j / S = e_j / (sum of the picked e),
// no need of the others.  LPT lanes per token, lane j < topk its slot j; the
// picked logits' parts reach the lanes that write them through LDS.  Bound by HBM
// and the order of a token's loads (the row, then ids, then w, dw and the picked
// logits, each waited for): where the softmax reaches every logit, T = 19647, E = 256,
// fp32, 11 to 13 us for 42 MB, 11.5 in a run of calls, 3.6 TB/s (12.2 with one token
// a wave).  Elsewhere only the rows' zeros and picks are written: sigmoid,
// renormalised, top-8 of the same, 10.5 to 13 us, 22 MB.
template <typename T, int EPL, int LPT>
__global__ __launch_bounds__(256) void k_gate_backward(v4moe_gate g, const T* __restrict__ logits, int64_t ld,
                                                       const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                       const float* __restrict__ dw, T* __restrict__ dl, int64_t ldd)
{
    constexpr int TOK = 64 / LPT;
    __shared__ __align__(16) float staged[4][TOK][EPL * LPT];
    const int lane = threadIdx.x & (LPT - 1), tok = (threadIdx.x & 63) / LPT;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), t0 = (blockIdx.x * 4 + wave) * TOK;
    if (t0 >= g.T) return;
    const int t = min(t0 + tok, g.T - 1);               // (past the last token: it again, not stored)
    const int e0 = lane * EPL;
    const T* row = logits + (int64_t)t * ld;
    const bool soft = g.score == V4MOE_SCORE_SOFTMAX, dense = soft && !g.renorm;
    float p[EPL];
    if (dense) load_logits<T, EPL>(row, e0, g.E, p);
    const bool slot = lane < g.topk;
    const int64_t at = (int64_t)t * g.topk + lane;
    const int my_e = slot ? ids[at] : -1;
    const bool valid = my_e >= 0 && my_e < g.E;      // an id out of range (an input error) gets no gradient
    const bool live = valid && w[at] != 0.0f;
    const float my_dw = live ? dw[at] : 0.0f;
    float z = -kInf;
    if (live) {
        if constexpr (sizeof(T) == 4) z = clean(row[my_e]);
        else z = clean(bf16_to_f32(row[my_e]));
    }
    float m = 0.0f, total = 1.0f;
    if (soft) {
        uint32_t best = order_of(z);
        if (dense) {
#pragma unroll
            for (int q = 0; q < EPL; q++) {
                p[q] = clean(p[q]);
                best = max(best, order_of(p[q]));
            }
        }
        best = token_max<LPT>(best);
        m = best == kNone ? 0.0f : float_of(best);
    }
    if (dense) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < EPL; q++) {
            p[q] = expf(p[q] - m);
            sum += p[q];
        }
        total = token_sum<LPT>(sum);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int q = 0; q < EPL; q++) p[q] *= inv;
    }
    float s = 0.0f;
    if (live) s = soft ? expf(z - m) / total : g.score == V4MOE_SCORE_SIGMOID ? sigmoid(z) : sqrt_softplus(z);
    float u = s, d = my_dw;
    if (g.renorm) {
        const float S = row_sum(s);                  // (lanes past topk <= 16 hold 0)
        u = S > 0.0f ? s / S : 0.0f;
        d = 0.0f;
#pragma unroll 4
        for (int j = 0; j < g.topk; j++) d += __shfl(u, j, 16) * (my_dw - __shfl(my_dw, j, 16));
    }
    float dz = g.scale * d * u;
    if (g.score == V4MOE_SCORE_SIGMOID) dz *= 1.0f / (1.0f + expf(z));
    // (below -16 sigmoid / softplus = 1 - exp(z) / 2 + ... is 1 in fp32; neither needs to be a normal number)
    else if (!soft) dz *= z < -16.0f ? 0.5f : sigmoid(z) / (2.0f * softplus(z));
    if (!live || s == 0.0f) dz = 0.0f;
    float* st = staged[wave][tok];
    const float dot = dense ? token_sum<LPT>(dz) : 0.0f;
#pragma unroll
    for (int q = 0; q < EPL; q++) st[e0 + q] = dense ? -p[q] * dot : 0.0f;
    __builtin_amdgcn_wave_barrier();
    if (valid) st[my_e] += dz;                       // (ids of a row are distinct)
    __builtin_amdgcn_wave_barrier();
    float out[EPL];
#pragma unroll
    for (int q = 0; q < EPL; q++) out[q] = st[e0 + q];
    if (t0 + tok < g.T) store_logits<T, EPL>(dl + (int64_t)t * ldd, e0, g.E, out);
}

// Calls f with the experts per lane and the lanes per token, which hold at least
// `lanes` groups and a row of E.  Several tokens to a wave share its reductions,
// but each lane then has more experts to itself: one token a wave until that
// fills the card (1024 SIMDs, four waves each).  Routing over E = 256, eight of
// four groups' experts, one and two tokens a wave: T = 1 4.0 and 4.5 us, 2048 5.1
// and 5.5, 4096 6.3 and 5.9, 8192 9.7 and 8.5, 20000 19.4 and 16.6; four of 16
// lanes, sixteen experts each, 20000 17.5.  E = 128, one and four: 2048 4.6 and 5.5,
// 4096 5.5 and 5.6, 8192 7.8 and 6.1.
template <typename F>
void for_row(int T, int E, int lanes, F f)
{
    const std::integral_constant<int, 16> quarter;
    const std::integral_constant<int, 32> half;
    const std::integral_constant<int, 64> whole;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    const std::integral_constant<int, 16> sixteen;
    const bool many = T >= 4096;
    if (many && lanes <= 16 && E <= 32) f(two, quarter);
    else if (many && lanes <= 16 && E <= 64) f(four, quarter);
    else if (many && lanes <= 16 && E <= 128) f(eight, quarter);
    else if (many && lanes <= 32 && E <= 256) f(eight, half);
    else if (E <= 64) f(one, whole);
    else if (E <= 128) f(two, whole);
    else if (E <= 256) f(four, whole);
    else if (E <= 512) f(eight, whole);
    else f(sixteen, whole);
}

int check_gate(const v4moe_gate* g, int32_t type, const void* logits, int64_t ld)
{
    if (!g) return V4MOE_ENULL;
    if (g->T < 0 || g->T > (1 << 24) || g->E < 1 || g->E > 1024 || g->topk < 1 || g->topk > 16) return V4MOE_EDIMS;
    if (g->score < V4MOE_SCORE_SIGMOID || g->score > V4MOE_SCORE_SQRTSOFTPLUS) return V4MOE_EDIMS;
    if (g->groups < 1 || g->groups > 64 || g->E % g->groups) return V4MOE_EDIMS;
    if (g->topk_groups < 1 || g->topk_groups > g->groups) return V4MOE_EDIMS;
    if (g->topk > g->topk_groups * (g->E / g->groups)) return V4MOE_EDIMS;
    if (type != V4MOE_TYPE_F32 && type != V4MOE_TYPE_BF16) return V4MOE_EDIMS;
    if (ld < g->E || ld > (1ll << 40)) return V4MOE_EDIMS;
    if (g->T == 0) return V4MOE_OK;
    if (!logits) return V4MOE_ENULL;
    return reinterpret_cast<uintptr_t>(logits) % (type == V4MOE_TYPE_F32 ? 4 : 2) ? V4MOE_EALIGN : V4MOE_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T>
hipError_t launch_gate(const v4moe_gate& g, const void* logits, int64_t ld, const float* bias, int32_t* ids, float* w,
                       hipStream_t s)
{
    for_row(g.T, g.E, g.groups, [&](auto epl, auto lpt) {
        constexpr int PER = 4 * 64 / decltype(lpt)::value;        // tokens per block
        hipLaunchKernelGGL((k_gate<T, decltype(epl)::value, decltype(lpt)::value>), dim3((unsigned)((g.T + PER - 1) / PER)),
                           dim3(256), 0, s, g, static_cast<const T*>(logits), ld, bias, ids, w);
    });
    return hipGetLastError();
}
template <typename T>
hipError_t launch_gate_backward(const v4moe_gate& g, const void* logits, int64_t ld, const int32_t* ids, const float* w,
                                const float* dw, void* dl, int64_t ldd, hipStream_t s)
{
    for_row(g.T, g.E, 1, [&](auto epl, auto lpt) {
        constexpr int PER = 4 * 64 / decltype(lpt)::value;
        hipLaunchKernelGGL((k_gate_backward<T, decltype(epl)::value, decltype(lpt)::value>),
                           dim3((unsigned)((g.T + PER - 1) / PER)), dim3(256), 0, s, g, static_cast<const T*>(logits), ld,
                           ids, w, dw, static_cast<T*>(dl), ldd);
    });
    return hipGetLastError();
}

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) int moe_gate(const v4moe_gate* g, const void* logits, int32_t type, int64_t ld,
                                                    const float* bias, int32_t* topk_ids, float* topk_w, void* stream)
{
    if (const int rc = check_gate(g, type, logits, ld)) return rc;
    if (g->T == 0) return V4MOE_OK;
    if (!topk_ids || !topk_w) return V4MOE_ENULL;
    if (!aligned4(bias) || !aligned4(topk_ids) || !aligned4(topk_w)) return V4MOE_EALIGN;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = type == V4MOE_TYPE_F32 ? launch_gate<float>(*g, logits, ld, bias, topk_ids, topk_w, s)
                                                : launch_gate<uint16_t>(*g, logits, ld, bias, topk_ids, topk_w, s);
    return e == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

__attribute__((visibility("default"))) int moe_gate_backward(const v4moe_gate* g, const void* logits, int32_t type,
                                                             int64_t ld, const int32_t* topk_ids, const float* topk_w,
                                                             const float* dw, void* dlogits, int64_t ldd, void* stream)
{
    if (const int rc = check_gate(g, type, logits, ld)) return rc;
    if (ldd < g->E || ldd > (1ll << 40)) return V4MOE_EDIMS;
    if (g->T == 0) return V4MOE_OK;
    if (!topk_ids || !topk_w || !dw || !dlogits) return V4MOE_ENULL;
    if (!aligned4(topk_ids) || !aligned4(topk_w) || !aligned4(dw) ||
        reinterpret_cast<uintptr_t>(dlogits) % (type == V4MOE_TYPE_F32 ? 4 : 2))
        return V4MOE_EALIGN;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e =
        type == V4MOE_TYPE_F32
            ? launch_gate_backward<float>(*g, logits, ld, topk_ids, topk_w, dw, dlogits, ldd, s)
            : launch_gate_backward<uint16_t>(*g, logits, ld, topk_ids, topk_w, dw, dlogits, ldd, s);
    return e == hipSuccess ? V4MOE_OK : V4MOE_ELAUNCH;
}

}  // extern "C"
