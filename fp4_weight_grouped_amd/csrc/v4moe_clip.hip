// v4moe_clip.hip -- the norm of all gradients together, and the gradients
// scaled down to a largest norm.
//
//   norm = sqrt(sum over every element of g^2), coef = norm > max ? max / norm : 1,
//   out = g * coef (rounded once to the gradient's type)
// Squares are summed in fp64: nothing overflows or vanishes that fp32 holds,
// and at the rate the gradients arrive from HBM the conversion and the fma
// are hidden.  No atomics: a block sums the chunks b, b + grid, ... in order
// and one thread per partial adds them in a fixed tree, so the norm is the same
// bits on every run.  Bound by HBM: every gradient is read for the norm, and
// read again and written once the norm is known.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

#include <hip/hip_runtime.h>

namespace v4moe {

namespace {

constexpr int kTensors = 96;          // tensors per launch: their table travels in the kernel's arguments (< 4 KiB)
constexpr int kChunk = 16384;         // elements per chunk: one block's unit of work
constexpr int kMaxBlocks = 2048;      // partial sums per launch
constexpr int64_t kMaxElements = 1ll << 36;   // of a tensor: a launch's chunks then fit 31 bits

struct Entry {
    const void* g;
    void* out;
    int64_t n;
    int32_t first;                    // chunks before this tensor
    int32_t bf16;
};
struct Table {
    Entry e[kTensors];
    int32_t count, chunks;
};
static_assert(sizeof(Table) < 3584, "kernel arguments");

// The tensor chunk c belongs to.
__device__ __forceinline__ int find(const Table& t, int c)
{
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)bf16x2(v, 0.0f); }

template <typename T>
__device__ __forceinline__ double sum_squares(const T* p, int n)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) {
        const double v = (double)to_f32(p[i]);
        s = fma(v, v, s);
    }
    return s;
}
template <typename T>
__device__ __forceinline__ void scale_to(const T* p, T* o, int n, float coef)
{
    for (int i = threadIdx.x; i < n; i += 256) o[i] = from_f32<T>(to_f32(p[i]) * coef);
}

// Sum over the block, in every thread; fixed tree.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[4];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(256) void k_grad_squares(Table t, double* __restrict__ partial)
{
    double s = 0.0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = t.e[find(t, c)];
        const int64_t at = (int64_t)(c - e.first) * kChunk;
        const int n = (int)min((int64_t)kChunk, e.n - at);
        s += e.bf16 ? sum_squares(static_cast<const uint16_t*>(e.g) + at, n)
                    : sum_squares(static_cast<const float*>(e.g) + at, n);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_grad_norm(int n, const double* __restrict__ partial, float* __restrict__ norm)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) s += partial[i];
    s = block_sum(s);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ __launch_bounds__(256) void k_grad_scale(Table t, const float* __restrict__ norm, float max_norm)
{
    // a norm that is not finite leaves the gradients as they are: the caller sees it and drops the step
    const float v = *norm;
    const float coef = v > max_norm && v < __builtin_inff() ? max_norm / v : 1.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = t.e[find(t, c)];
        if (coef == 1.0f && e.out == e.g) continue;
        const int64_t at = (int64_t)(c - e.first) * kChunk;
        const int n = (int)min((int64_t)kChunk, e.n - at);
        if (e.bf16) scale_to(static_cast<const uint16_t*>(e.g) + at, static_cast<uint16_t*>(e.out) + at, n, coef);
        else scale_to(static_cast<const float*>(e.g) + at, static_cast<float*>(e.out) + at, n, coef);
    }
}

// Splits a list into launches of at most kTensors entries; f(table, blocks)
// returns false to stop.
template <typename F>
bool for_tables(int32_t count, const v4moe_tensor* t, F f)
{
    int32_t i = 0;
    while (i < count) {
        Table tab{};
        int64_t chunks = 0;
        for (; i < count && tab.count < kTensors; i++) {
            if (t[i].n == 0) continue;
            tab.e[tab.count++] = Entry{t[i].g, t[i].out ? t[i].out : const_cast<void*>(t[i].g), t[i].n, (int32_t)chunks,
                                       t[i].type == V4MOE_TYPE_BF16};
            chunks += (t[i].n + kChunk - 1) / kChunk;
        }
        if (tab.count == 0) break;
        tab.chunks = (int32_t)chunks;
        if (!f(tab, (int)(chunks < kMaxBlocks ? chunks : kMaxBlocks))) return false;
    }
    return true;
}

int check_tensors(int32_t count, const v4moe_tensor* t)
{
    if (count < 0 || count > (1 << 20)) return V4MOE_EDIMS;
    if (count > 0 && !t) return V4MOE_ENULL;
    for (int32_t i = 0; i < count; i++) {
        if (t[i].n < 0 || t[i].n > kMaxElements || (t[i].type != V4MOE_TYPE_F32 && t[i].type != V4MOE_TYPE_BF16))
            return V4MOE_EDIMS;
        if (t[i].n > 0 && !t[i].g) return V4MOE_ENULL;
        const uintptr_t mask = t[i].type == V4MOE_TYPE_F32 ? 3 : 1;
        if (((uintptr_t)t[i].g | (uintptr_t)t[i].out) & mask) return V4MOE_EALIGN;
    }
    return V4MOE_OK;
}

size_t partials(int32_t count) { return (size_t)((count + kTensors - 1) / kTensors) * kMaxBlocks; }

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) size_t moe_clip_workspace_bytes(int32_t count)
{
    return count < 0 || count > (1 << 20) ? 0 : (count == 0 ? 256 : partials(count) * sizeof(double));
}

__attribute__((visibility("default"))) int moe_clip_grads(int32_t count, const v4moe_tensor* tensors, float max_norm,
                                                          float* norm, void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_tensors(count, tensors)) return rc;
    if (!(max_norm >= 0.0f)) return V4MOE_EDIMS;
    if (!norm || !workspace) return V4MOE_ENULL;
    if (((uintptr_t)norm & 3) || ((uintptr_t)workspace & 15)) return V4MOE_EALIGN;
    if (ws_bytes < moe_clip_workspace_bytes(count)) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    double* part = static_cast<double*>(workspace);
    int used = 0;
    auto launched = []() { return hipGetLastError() == hipSuccess; };
    if (!for_tables(count, tensors, [&](const Table& t, int blocks) {
            hipLaunchKernelGGL(k_grad_squares, dim3(blocks), dim3(256), 0, s, t, part + used);
            used += blocks;
            return launched();
        }))
        return V4MOE_ELAUNCH;
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, used, part, norm);
    if (!launched()) return V4MOE_ELAUNCH;
    if (!for_tables(count, tensors, [&](const Table& t, int blocks) {
            hipLaunchKernelGGL(k_grad_scale, dim3(blocks), dim3(256), 0, s, t, norm, max_norm);
            return launched();
        }))
        return V4MOE_ELAUNCH;
    return V4MOE_OK;
}

}  // extern "C"
