// v4moe_clip.hip -- the norm of all gradients together, and the gradients
// scaled down to a largest norm.
//
//   norm = sqrt(sum over every element of g^2), coef = norm > max ? max / norm : 1,
//   out = g * coef
// coef comes from the 64-bit norm where that, or coef itself, is beyond fp32: finite
// gradients are scaled whatever their norm.  It is an fp32 number where it can be (the
// product rounded once to the gradient's type); below the normal ones it would have few
// bits or none left, and the products are taken in fp64.
// Squares are summed in fp64: nothing overflows or vanishes that fp32 holds,
// and at the rate the gradients arrive from HBM the conversion and the fma
// are hidden.  No atomics: a block sums the chunks b, b + grid, ... in order,
// a fixed tree adds the blocks' sums, and every block that scales adds them
// again in the same tree, so the norm is the same bits everywhere and on every
// run.  Bound by HBM: every gradient is read for the norm, and read again and
// written once the norm is known (the last of them still from the memory-side
// cache, as the second pass goes backwards through a launch's tensors; the launches
// of a list of more than 96 go forwards).  Three fp32 tensors of 268 M elements:
// the squares 540 us, 6.0 TB/s, the scaling 1197 us, 5.4 TB/s; 23 tensors of 3.0 M
// together 5.5 and 7.4 to 8.0 us.
#include "v4moe.h"
#include "v4moe_device.h"
#include "v4moe_internal.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <memory>
#include <new>

namespace v4moe {

namespace {

constexpr int kTensors = 96;          // tensors per launch: their table travels in the kernel's arguments (< 4 KiB)
// Blocks, and so partial sums, per launch: four a CU.  Twice as many have more
// partial sums to add again in every block: 3 M fp32 elements 14.8 us (12.9), 300 M
// 683 (676); half as many leave 10 M at 25.5 (24.5).
constexpr int kMaxBlocks = 1024;
constexpr int64_t kMaxElements = 1ll << 36;   // of a tensor: a launch's chunks then fit 31 bits
constexpr int kThreads = 256;

struct Entry {
    const void* g;
    void* out;
    int64_t n;
    int32_t first;                    // chunks before this tensor
    int32_t bf16;
};
struct Table {
    Entry e[kTensors];
    int32_t count, chunks, chunk;     // chunk: elements of one, a block's unit of work
};
static_assert(sizeof(Table) < 3584 && sizeof(Entry) == 32, "kernel arguments");

// The table in LDS: the arguments lie in host memory, and each dependent read
// of them (a search takes seven) would wait for it.
__device__ __forceinline__ void stage_table(const Table& t, Entry* lds)
{
    if ((int)threadIdx.x < t.count) lds[threadIdx.x] = t.e[threadIdx.x];
    __syncthreads();
}
// The tensor chunk c belongs to.
__device__ __forceinline__ int find(const Entry* e, int count, int c)
{
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (e[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Sixteen bytes at any element's address, in one access: unaligned ones are the
// hardware's to split.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef v4u v4u_any __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ float element(const v4u& v, int i)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(v[i]);
    else return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }

template <typename T>
__device__ __forceinline__ void sum_squares(const T* p, int n, double (&s)[4])
{
    constexpr int V = 16 / sizeof(T), U = 4;             // elements per access, accesses in flight
    const int nv = n / V;
    int i = threadIdx.x;
    for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
        v4u v[U];
#pragma unroll
        for (int u = 0; u < U; u++) v[u] = *reinterpret_cast<const v4u_any*>(p + (int64_t)(i + u * kThreads) * V);
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int k = 0; k < V; k++) {
                const double d = (double)element<T>(v[u], k);
                s[k & 3] = fma(d, d, s[k & 3]);
            }
    }
    for (; i < nv; i += kThreads) {
        const v4u v = *reinterpret_cast<const v4u_any*>(p + (int64_t)i * V);
#pragma unroll
        for (int k = 0; k < V; k++) {
            const double d = (double)element<T>(v, k);
            s[k & 3] = fma(d, d, s[k & 3]);
        }
    }
    if ((int)threadIdx.x < n - nv * V) {
        const double d = (double)to_f32(p[nv * V + threadIdx.x]);
        s[0] = fma(d, d, s[0]);
    }
}
__device__ __forceinline__ float product(float g, float coef) { return g * coef; }
__device__ __forceinline__ float product(float g, double coef) { return (float)((double)g * coef); }
template <typename T, typename C>
__device__ __forceinline__ v4u scaled(const v4u& v, C coef)
{
    v4u r;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (sizeof(T) == 4) r[k] = __float_as_uint(product(element<T>(v, k), coef));
        else r[k] = bf16x2(product(element<T>(v, 2 * k), coef), product(element<T>(v, 2 * k + 1), coef));
    }
    return r;
}
template <typename T, typename C>
__device__ __forceinline__ void scale_to(const T* p, T* o, int n, C coef)
{
    constexpr int V = 16 / sizeof(T), U = 4;
    const int nv = n / V;
    int i = threadIdx.x;
    for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
        v4u v[U];
#pragma unroll
        for (int u = 0; u < U; u++) v[u] = *reinterpret_cast<const v4u_any*>(p + (int64_t)(i + u * kThreads) * V);
#pragma unroll
        for (int u = 0; u < U; u++) *reinterpret_cast<v4u_any*>(o + (int64_t)(i + u * kThreads) * V) = scaled<T>(v[u], coef);
    }
    for (; i < nv; i += kThreads)
        *reinterpret_cast<v4u_any*>(o + (int64_t)i * V) = scaled<T>(*reinterpret_cast<const v4u_any*>(p + (int64_t)i * V), coef);
    if ((int)threadIdx.x < n - nv * V) {
        const int at = nv * V + threadIdx.x;
        const float f = product(to_f32(p[at]), coef);
        if constexpr (sizeof(T) == 4) o[at] = f;
        else o[at] = (T)bf16x2(f, 0.0f);
    }
}

// Sum over the block, in every thread; fixed tree.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kThreads) void k_grad_squares(Table t, double* __restrict__ partial)
{
    __shared__ Entry tab[kTensors];
    stage_table(t, tab);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = tab[find(tab, t.count, c)];
        const int64_t at = (int64_t)(c - e.first) * t.chunk;
        const int n = (int)min((int64_t)t.chunk, e.n - at);
        if (e.bf16) sum_squares(static_cast<const uint16_t*>(e.g) + at, n, s);
        else sum_squares(static_cast<const float*>(e.g) + at, n, s);
    }
    const double v = block_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// n_partial sums of all launches of k_grad_squares -> the norm, in every block
// (block 0 of the first launch writes it); then this launch's chunks, last first.
__global__ __launch_bounds__(kThreads) void k_grad_scale(Table t, int n_partial, const double* __restrict__ partial,
                                                         float* __restrict__ norm, float max_norm)
{
    __shared__ Entry tab[kTensors];
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += kThreads) s += partial[i];
    stage_table(t, tab);
    const double exact = sqrt(block_sum(s));
    const float v = (float)exact;
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    // a norm that is not finite (in fp64: fp32 elements' squares do not overflow it) leaves the gradients as they
    // are: the caller sees it and drops the step
    const bool clip = v > max_norm && exact < __builtin_inf();
    const double ratio = clip ? (double)max_norm / exact : 1.0;
    const float coef = clip && v < __builtin_inff() ? max_norm / v : (float)ratio;
    auto scale = [&](auto by) {
        for (int c = t.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
            const Entry& e = tab[find(tab, t.count, c)];
            if (by == 1 && e.out == e.g) continue;
            const int64_t at = (int64_t)(c - e.first) * t.chunk;
            const int n = (int)min((int64_t)t.chunk, e.n - at);
            if (e.bf16) scale_to(static_cast<const uint16_t*>(e.g) + at, static_cast<uint16_t*>(e.out) + at, n, by);
            else scale_to(static_cast<const float*>(e.g) + at, static_cast<float*>(e.out) + at, n, by);
        }
    };
    if (ratio >= 0x1p-126) scale(coef);
    else scale(ratio);
}

// Elements per chunk for a list of `total`: a power of two of 1024 (one access
// per thread) to 65536, so that a small list still makes a block per CU and a
// large one spends its time in the unrolled loop: 3.0 M elements take 15 us in chunks
// of 1024 and 22 in chunks of 65536, 805 M fp32 ones 1915 and 1745.
int chunk_of(int64_t total)
{
    int chunk = 1024;
    while (chunk < 65536 && total / chunk > 2 * kMaxBlocks) chunk *= 2;
    return chunk;
}

// Splits a list into launches of at most kTensors entries; f(table, blocks)
// returns false to stop.  An empty list gives one empty table.
template <typename F>
bool for_tables(int32_t count, const v4moe_tensor* t, F f)
{
    int64_t total = 0;
    for (int32_t i = 0; i < count; i++) total += t[i].n;
    const int chunk = chunk_of(total);
    int32_t i = 0;
    do {
        Table tab;
        int64_t chunks = 0;
        tab.count = 0;
        for (; i < count && tab.count < kTensors; i++) {
            if (t[i].n == 0) continue;
            tab.e[tab.count++] = Entry{t[i].g, t[i].out ? t[i].out : const_cast<void*>(t[i].g), t[i].n, (int32_t)chunks,
                                       t[i].type == V4MOE_TYPE_BF16};
            chunks += (t[i].n + chunk - 1) / chunk;
        }
        tab.chunks = (int32_t)chunks;
        tab.chunk = chunk;
        if (!f(tab, (int)(chunks < 1 ? 1 : chunks < kMaxBlocks ? chunks : kMaxBlocks))) return false;
    } while (i < count);
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

// Whether memory that the call writes is also another entry's: blocks that scale them
// would race, and a gradient listed twice would be scaled once or twice.  An infinite
// max_norm writes nothing in place.  Ranges in order of address, each compared with
// the furthest end of those before it.
struct Range {
    uintptr_t lo, hi;
    bool written;
};
bool overlaps(int32_t count, const v4moe_tensor* t, float max_norm, Range* r)
{
    int n = 0;
    for (int32_t i = 0; i < count; i++) {
        const size_t bytes = (size_t)t[i].n * (t[i].type == V4MOE_TYPE_F32 ? 4 : 2);
        if (bytes == 0) continue;
        const uintptr_t g = (uintptr_t)t[i].g, out = (uintptr_t)t[i].out;
        const bool in_place = !out || out == g;
        r[n++] = Range{g, g + bytes, in_place && max_norm < __builtin_inff()};
        if (!in_place) r[n++] = Range{out, out + bytes, true};
    }
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (int i = 0; i < n; i++) {
        if (r[i].lo < (r[i].written ? any : written)) return true;
        any = std::max(any, r[i].hi);
        if (r[i].written) written = std::max(written, r[i].hi);
    }
    return false;
}
int check_overlaps(int32_t count, const v4moe_tensor* t, float max_norm)
{
    constexpr int kFew = 128;
    Range few[2 * kFew];
    std::unique_ptr<Range[]> many(count > kFew ? new (std::nothrow) Range[2 * (size_t)count] : nullptr);
    if (count > kFew && !many) return V4MOE_EWORKSPACE;
    return overlaps(count, t, max_norm, many ? many.get() : few) ? V4MOE_EDIMS : V4MOE_OK;
}

size_t partials(int32_t count) { return (size_t)(count / kTensors + 1) * kMaxBlocks; }

}  // namespace

}  // namespace v4moe

using namespace v4moe;

extern "C" {

__attribute__((visibility("default"))) size_t moe_clip_workspace_bytes(int32_t count)
{
    return count < 0 || count > (1 << 20) ? 0 : partials(count) * sizeof(double);
}

__attribute__((visibility("default"))) int moe_clip_grads(int32_t count, const v4moe_tensor* tensors, float max_norm,
                                                          float* norm, void* workspace, size_t ws_bytes, void* stream)
{
    if (const int rc = check_tensors(count, tensors)) return rc;
    if (!(max_norm >= 0.0f)) return V4MOE_EDIMS;
    if (const int rc = check_overlaps(count, tensors, max_norm)) return rc;
    if (!norm || !workspace) return V4MOE_ENULL;
    if (((uintptr_t)norm & 3) || ((uintptr_t)workspace & 15)) return V4MOE_EALIGN;
    if (ws_bytes < moe_clip_workspace_bytes(count)) return V4MOE_EWORKSPACE;
    if (!device_ready()) return V4MOE_EDEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    double* part = static_cast<double*>(workspace);
    int used = 0;
    auto launched = []() { return hipGetLastError() == hipSuccess; };
    if (!for_tables(count, tensors, [&](const Table& t, int blocks) {
            hipLaunchKernelGGL(k_grad_squares, dim3(blocks), dim3(kThreads), 0, s, t, part + used);
            used += blocks;
            return launched();
        }))
        return V4MOE_ELAUNCH;
    if (!for_tables(count, tensors, [&](const Table& t, int blocks) {
            hipLaunchKernelGGL(k_grad_scale, dim3(blocks), dim3(kThreads), 0, s, t, used, part, norm, max_norm);
            norm = nullptr;
            return launched();
        }))
        return V4MOE_ELAUNCH;
    return V4MOE_OK;
}

}  // extern "C"
