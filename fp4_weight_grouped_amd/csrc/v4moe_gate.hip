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
// softmax's sum is taken in fp64: rounded to fp32 it does not depend on the
// order of the terms, and so neither do the picks.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

#include <hip/hip_runtime.h>

namespace v4moe {

namespace {

constexpr float kMask = 1e30f;
constexpr float kInf = __builtin_inff();

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)bf16x2(v, 0.0f); }

// -inf for a masked logit, and for NaN
__device__ __forceinline__ float clean(float z) { return z > -kMask ? fminf(z, kMask) : -kInf; }

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
__device__ __forceinline__ float sqrt_softplus(float z) { return sqrtf(fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z)))); }

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// z -> scores, in place; lane l holds experts l + 64q.  Softmax leaves the
// maximum and the sum in m and total.
template <int NQ>
__device__ __forceinline__ void scores(int score, float (&z)[NQ], float& m, float& total)
{
    if (score == V4MOE_SCORE_SOFTMAX) {
        m = -kInf;
#pragma unroll
        for (int q = 0; q < NQ; q++) m = fmaxf(m, z[q]);
        m = wave_max(m);
        m = m == -kInf ? 0.0f : m;
        double sum = 0.0;
#pragma unroll
        for (int q = 0; q < NQ; q++) {
            z[q] = expf(z[q] - m);
            sum += (double)z[q];
        }
        total = (float)wave_sum(sum);
#pragma unroll
        for (int q = 0; q < NQ; q++) z[q] = total > 0.0f ? z[q] / total : 0.0f;
    } else {
#pragma unroll
        for (int q = 0; q < NQ; q++)
            z[q] = score == V4MOE_SCORE_SIGMOID ? sigmoid(z[q]) : sqrt_softplus(z[q]);
    }
}

// Larger key first, then the lower id.
__device__ __forceinline__ bool ahead(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

// One wave per token; lane l holds experts l + 64q, q < NQ.
template <typename T, int NQ>
__global__ __launch_bounds__(256) void k_gate(v4moe_gate g, const T* __restrict__ logits, int64_t ld,
                                              const float* __restrict__ bias, int32_t* __restrict__ ids,
                                              float* __restrict__ w)
{
    __shared__ float keys[4][NQ * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wave;
    const bool on = t < g.T;
    const T* row = logits + (int64_t)(on ? t : 0) * ld;
    float s[NQ], key[NQ];
    bool masked[NQ];
#pragma unroll
    for (int q = 0; q < NQ; q++) {
        const int e = lane + 64 * q;
        s[q] = e < g.E ? clean(load_logit(row + e)) : -kInf;
        masked[q] = s[q] == -kInf;
    }
    float m = 0.0f, total = 0.0f;
    scores<NQ>(g.score, s, m, total);
#pragma unroll
    for (int q = 0; q < NQ; q++) {
        const int e = lane + 64 * q;
        const float k = bias && e < g.E ? s[q] + bias[e] : s[q];
        key[q] = masked[q] || k != k ? -kInf : k;
    }
    if (g.groups > 1) {
        // lane i < groups: group i's value, then its rank among the groups
        const int size = g.E / g.groups;
#pragma unroll
        for (int q = 0; q < NQ; q++) keys[wave][lane + 64 * q] = key[q];
        __syncthreads();
        float a = -kInf, b = -kInf;
        if (lane < g.groups)
            for (int i = 0; i < size; i++) {
                const float k = keys[wave][lane * size + i];
                b = fmaxf(b, fminf(a, k));
                a = fmaxf(a, k);
            }
        const float v = b == -kInf ? a : a + b;
        int rank = 0;
        for (int o = 0; o < g.groups; o++) rank += ahead(__shfl(v, o), o, v, lane);
        const uint64_t kept = __ballot(lane < g.groups && rank < g.topk_groups);
#pragma unroll
        for (int q = 0; q < NQ; q++) {
            const int e = lane + 64 * q;
            if (e < g.E && !((kept >> (e / size)) & 1)) key[q] = -kInf;
        }
    }
    // topk rounds of a wave maximum; a picked expert leaves by its id
    float my_s = 0.0f;
    int my_e = 0;
    uint32_t taken = 0;
    for (int j = 0; j < g.topk; j++) {
        float bk = -kInf, bs = 0.0f;
        int be = 1 << 30;
#pragma unroll
        for (int q = 0; q < NQ; q++) {
            const int e = lane + 64 * q;
            if (e < g.E && !((taken >> q) & 1) && ahead(key[q], e, bk, be)) bk = key[q], bs = s[q], be = e;
        }
        for (int o = 1; o < 64; o <<= 1) {
            const float ok = __shfl_xor(bk, o), os = __shfl_xor(bs, o);
            const int oe = __shfl_xor(be, o);
            if (ahead(ok, oe, bk, be)) bk = ok, bs = os, be = oe;
        }
        if ((be & 63) == lane) taken |= 1u << (be >> 6);
        if (lane == j) my_e = be, my_s = bk == -kInf ? 0.0f : bs;
    }
    float sum = 1.0f;
    if (g.renorm) {
        sum = 0.0f;
        for (int j = 0; j < g.topk; j++) sum += __shfl(my_s, j);
    }
    if (on && lane < g.topk) {
        ids[(int64_t)t * g.topk + lane] = my_e;
        w[(int64_t)t * g.topk + lane] = (sum > 0.0f ? my_s / sum : 0.0f) * g.scale;
    }
}

// Gradient with respect to the logits.  A slot of weight zero (a filler, or a
// score that underflowed) has none.  With a_j = dw_j over the live slots:
//   renormalised: q_j = s_j / S, ds_j = scale / S * sum_i q_i (dw_j - dw_i)
//   otherwise:    ds_j = scale * dw_j
//   dz = ds s (1 - s) | ds sigmoid(z) / (2 s) | p_e (ds_e [picked] - sum_j ds_j p_j),
// the softmax's last sum zero where the weights are renormalised, which leaves
// only the picked logits and, as p_j / S = e_j / (sum of the picked e),
// no need of the others.
template <typename T, int NQ>
__global__ __launch_bounds__(256) void k_gate_backward(v4moe_gate g, const T* __restrict__ logits, int64_t ld,
                                                       const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                       const float* __restrict__ dw, T* __restrict__ dl, int64_t ldd)
{
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= g.T) return;
    const T* row = logits + (int64_t)t * ld;
    const bool slot = lane < g.topk;
    const int64_t at = (int64_t)t * g.topk + lane;
    const int my_e = slot ? ids[at] : -1;
    const bool valid = my_e >= 0 && my_e < g.E;      // an id out of range (an input error) gets no gradient
    const bool live = valid && w[at] != 0.0f;
    const float my_dw = live ? dw[at] : 0.0f;
    const float z = live ? clean(load_logit(row + my_e)) : -kInf;
    const bool soft = g.score == V4MOE_SCORE_SOFTMAX, dense = soft && !g.renorm;
    float p[NQ];
#pragma unroll
    for (int q = 0; q < NQ; q++) p[q] = 0.0f;
    float m = 0.0f, total = 1.0f;
    if (dense) {
#pragma unroll
        for (int q = 0; q < NQ; q++) {
            const int e = lane + 64 * q;
            p[q] = e < g.E ? clean(load_logit(row + e)) : -kInf;
        }
        scores<NQ>(g.score, p, m, total);
    } else if (soft) {
        m = wave_max(z);
    }
    float s = 0.0f;
    if (live) s = soft ? expf(z - m) / total : g.score == V4MOE_SCORE_SIGMOID ? sigmoid(z) : sqrt_softplus(z);
    float ds = live ? g.scale * my_dw : 0.0f;
    if (g.renorm) {
        float S = 0.0f, d = 0.0f;
        for (int j = 0; j < g.topk; j++) S += __shfl(s, j);
        for (int j = 0; j < g.topk; j++) d += __shfl(s, j) * (my_dw - __shfl(my_dw, j));
        ds = live && S > 0.0f ? g.scale * (d / S) / S : 0.0f;
    }
    float dz;
    if (soft) dz = ds * s;
    else if (g.score == V4MOE_SCORE_SIGMOID) dz = ds * s * (1.0f / (1.0f + expf(z)));
    else dz = ds * sigmoid(z) / (2.0f * s);
    if (!live || s == 0.0f) dz = 0.0f;
    if (dense) {
        float dot = 0.0f;
        for (int j = 0; j < g.topk; j++) dot += __shfl(dz, j);
#pragma unroll
        for (int q = 0; q < NQ; q++) p[q] = -p[q] * dot;
    }
    for (int j = 0; j < g.topk; j++) {
        const int e = __shfl(valid ? my_e : -1, j);
        const float v = __shfl(dz, j);
        if (e >= 0 && (e & 63) == lane) {
#pragma unroll
            for (int q = 0; q < NQ; q++)
                if (q == (e >> 6)) p[q] += v;
        }
    }
    T* out = dl + (int64_t)t * ldd;
#pragma unroll
    for (int q = 0; q < NQ; q++) {
        const int e = lane + 64 * q;
        if (e < g.E) store_logit(out + e, p[q]);
    }
}

// calls f with the number of 64-expert steps of a row
template <typename F>
void for_row(int E, F f)
{
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 128) f(std::integral_constant<int, 2>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else if (E <= 512) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
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
    for_row(g.E, [&](auto n) {
        hipLaunchKernelGGL((k_gate<T, decltype(n)::value>), dim3((unsigned)((g.T + 3) / 4)), dim3(256), 0, s, g,
                           static_cast<const T*>(logits), ld, bias, ids, w);
    });
    return hipGetLastError();
}
template <typename T>
hipError_t launch_gate_backward(const v4moe_gate& g, const void* logits, int64_t ld, const int32_t* ids, const float* w,
                                const float* dw, void* dl, int64_t ldd, hipStream_t s)
{
    for_row(g.E, [&](auto n) {
        hipLaunchKernelGGL((k_gate_backward<T, decltype(n)::value>), dim3((unsigned)((g.T + 3) / 4)), dim3(256), 0, s, g,
                           static_cast<const T*>(logits), ld, ids, w, dw, static_cast<T*>(dl), ldd);
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
