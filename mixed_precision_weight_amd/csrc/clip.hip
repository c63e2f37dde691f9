// clip.hip -- the global norm over many gradient tensors, and clipping by it (gfx950).
//
//   norm = sqrt(sum over every tensor and element of g^2)
//   out  = g * max_norm / norm  where norm > max_norm (and finite), else g
//
// The weak columns of every linear are the parameters weak-column tuning trains,
// so a step has one small gradient per linear: hundreds of tensors of 10^5 - 10^6
// elements. Both passes therefore run over ONE sequence of 8192-element chunks that
// walks all tensors; a block owns a run of consecutive chunks, finds its first
// tensor by bisection and then only steps forward.
//
// Pass 1 (k_clip_sumsq, one launch per kClipItems tensors: their table travels in
// the kernel arguments and is copied to the workspace for pass 2) writes one fp64
// partial per block. Squares and sums are fp64: fp32 squares overflow from 1.8e19
// on, and the fp64 rate (two instructions per element) stays far below the memory
// time. Pass 2 (k_clip_scale) adds the partials in a fixed order in every block
// (at most 1024 per launch of pass 1, read from L2: cheaper than a launch that
// reduces them first), so the result does not depend on the launch's timing, and
// scales. The product is formed in fp64 and rounded once to the tensor's type.
// A tensor that stays as it is, in place, is neither read nor written by pass 2.
//
// Bound: memory, two reads and a write of every element (the second read comes
// from the 256 MB last-level cache where the tensors fit).
#include "owq_device.h"
#include "owq_launch.h"

namespace owq {

namespace {

constexpr int kClipChunk = 8192;    // elements per chunk, both types
constexpr int kClipThreads = 256;
constexpr int kPer = kClipChunk / kClipThreads;  // elements per thread of a full chunk

struct ClipArgs {
    ClipEntry e[kClipItems];
    int32_t count;       // tensors of this launch
    int32_t chunks;      // their chunks
    int32_t table0;      // index of the first of them in the whole table
    int64_t chunk_base;  // chunks of the earlier launches
};

// Sum of one double per thread over the block; every thread returns it. Butterfly
// in the wave, then the four waves' sums in order.
__device__ __forceinline__ double block_sum(double v, double* red)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += shfl_xor_f64(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((red[0] + red[1]) + red[2]) + red[3];
}

__device__ __forceinline__ double sumsq4(float4 v, double s)
{
    s = __builtin_fma((double)v.x, (double)v.x, s);
    s = __builtin_fma((double)v.y, (double)v.y, s);
    s = __builtin_fma((double)v.z, (double)v.z, s);
    return __builtin_fma((double)v.w, (double)v.w, s);
}

__device__ __forceinline__ double sumsq_h2(uint32_t v, double s)
{
    const float lo = h2f((uint16_t)(v & 0xffffu)), hi = h2f((uint16_t)(v >> 16));
    s = __builtin_fma((double)lo, (double)lo, s);
    return __builtin_fma((double)hi, (double)hi, s);
}

// n elements at p (n <= kClipChunk). A whole chunk at a 16-byte address is read
// in 16-byte pieces, all in flight at once; anything else element by element.
__device__ __forceinline__ double chunk_sumsq(const void* base, int64_t off, int n, bool half)
{
    const int t = threadIdx.x;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (half) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + off;
        if (n == kClipChunk && ((uintptr_t)p & 15) == 0) {
            uint4 v[kPer / 8];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++)
                v[u] = reinterpret_cast<const uint4*>(p)[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++) {
                s[0] = sumsq_h2(v[u].x, s[0]);
                s[1] = sumsq_h2(v[u].y, s[1]);
                s[2] = sumsq_h2(v[u].z, s[2]);
                s[3] = sumsq_h2(v[u].w, s[3]);
            }
        } else {
            for (int i = t; i < n; i += kClipThreads) {
                const float v = h2f(p[i]);
                s[0] = __builtin_fma((double)v, (double)v, s[0]);
            }
        }
    } else {
        const float* p = static_cast<const float*>(base) + off;
        if (n == kClipChunk && ((uintptr_t)p & 15) == 0) {
            float4 v[kPer / 4];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                v[u] = reinterpret_cast<const float4*>(p)[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                s[u & 3] = sumsq4(v[u], s[u & 3]);
        } else {
            for (int i = t; i < n; i += kClipThreads)
                s[0] = __builtin_fma((double)p[i], (double)p[i], s[0]);
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(kClipThreads) void k_clip_sumsq(const ClipArgs a, ClipEntry* table, double* partials)
{
    __shared__ double red[4];
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.count; i += kClipThreads) {
            ClipEntry e = a.e[i];
            e.chunk0 += a.chunk_base;
            table[a.table0 + i] = e;
        }
    const int64_t nb = gridDim.x, b = blockIdx.x;
    const int c0 = (int)(a.chunks * b / nb), c1 = (int)(a.chunks * (b + 1) / nb);
    int li = 0;  // the last tensor whose first chunk is at most c0 (empty tensors share it with their successor)
    for (int lo = 0, hi = a.count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (a.e[mid].chunk0 <= c0)
            lo = mid;
        else
            hi = mid;
        li = lo;
    }
    double s = 0.0;
    for (int c = c0; c < c1; c++) {
        while (li + 1 < a.count && a.e[li + 1].chunk0 <= c)
            li++;
        const ClipEntry& e = a.e[li];
        const int64_t off = (c - e.chunk0) * kClipChunk;
        const int64_t left = e.n - off;
        s += chunk_sumsq(e.g, off, (int)(left < kClipChunk ? left : kClipChunk), e.half != 0);
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = s;
}

__device__ __forceinline__ float scaled(float v, double c) { return (float)((double)v * c); }

__device__ __forceinline__ uint32_t scaled_h2(uint32_t v, double c)
{
    const uint32_t lo = f2h(scaled(h2f((uint16_t)(v & 0xffffu)), c));
    const uint32_t hi = f2h(scaled(h2f((uint16_t)(v >> 16)), c));
    return lo | (hi << 16);
}

// out = g * c, c == 1: an exact copy
__device__ __forceinline__ void chunk_scale(const ClipEntry& e, int64_t off, int n, double c)
{
    const int t = threadIdx.x;
    if (e.half) {
        const uint16_t* p = static_cast<const uint16_t*>(e.g) + off;
        uint16_t* o = static_cast<uint16_t*>(e.out) + off;
        if (n == kClipChunk && (((uintptr_t)p | (uintptr_t)o) & 15) == 0) {
            uint4 v[kPer / 8];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++)
                v[u] = reinterpret_cast<const uint4*>(p)[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++)
                reinterpret_cast<uint4*>(o)[t + kClipThreads * u] =
                    make_uint4(scaled_h2(v[u].x, c), scaled_h2(v[u].y, c), scaled_h2(v[u].z, c), scaled_h2(v[u].w, c));
        } else {
            for (int i = t; i < n; i += kClipThreads)
                o[i] = f2h(scaled(h2f(p[i]), c));
        }
    } else {
        const float* p = static_cast<const float*>(e.g) + off;
        float* o = static_cast<float*>(e.out) + off;
        if (n == kClipChunk && (((uintptr_t)p | (uintptr_t)o) & 15) == 0) {
            float4 v[kPer / 4];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                v[u] = reinterpret_cast<const float4*>(p)[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                reinterpret_cast<float4*>(o)[t + kClipThreads * u] =
                    make_float4(scaled(v[u].x, c), scaled(v[u].y, c), scaled(v[u].z, c), scaled(v[u].w, c));
        } else {
            for (int i = t; i < n; i += kClipThreads)
                o[i] = scaled(p[i], c);
        }
    }
}

__global__ __launch_bounds__(kClipThreads) void k_clip_scale(const ClipEntry* __restrict__ table, int count,
                                                             int64_t chunks, const double* __restrict__ partials,
                                                             int nparts, double max_norm, float* norm)
{
    __shared__ double red[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads)
        s += partials[i];
    const double total = sqrt(block_sum(s, red));
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *norm = (float)total;
    // NaN compares false, and an infinite norm leaves the tensors alone too
    const double c = total > max_norm && total < __builtin_inf() ? max_norm / total : 1.0;
    const int64_t nb = gridDim.x, b = blockIdx.x;
    const int64_t c0 = chunks * b / nb, c1 = chunks * (b + 1) / nb;
    if (c0 >= c1)
        return;
    int li = 0;
    for (int lo = 0, hi = count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (table[mid].chunk0 <= c0)
            lo = mid;
        else
            hi = mid;
        li = lo;
    }
    for (int64_t k = c0; k < c1; k++) {
        while (li + 1 < count && table[li + 1].chunk0 <= k)
            li++;
        const ClipEntry e = table[li];
        if (c == 1.0 && e.out == e.g)
            continue;
        const int64_t off = (k - e.chunk0) * kClipChunk;
        const int64_t left = e.n - off;
        chunk_scale(e, off, (int)(left < kClipChunk ? left : kClipChunk), c);
    }
}

int64_t chunks_of(int64_t n) { return (n + kClipChunk - 1) / kClipChunk; }

constexpr int kPartMax = 1024;   // blocks (and partials) per launch of pass 1
constexpr int kScaleMax = 2048;  // blocks of pass 2

}  // namespace

size_t clip_workspace_bytes(int count)
{
    const int launches = (count + kClipItems - 1) / kClipItems;
    return (size_t)launches * kPartMax * sizeof(double) + (size_t)count * sizeof(ClipEntry);
}

hipError_t launch_clip(const ClipEntry* items, int count, double max_norm, float* norm, void* ws, hipStream_t s)
{
    const int launches = (count + kClipItems - 1) / kClipItems;
    double* const partials = static_cast<double*>(ws);
    ClipEntry* const table = reinterpret_cast<ClipEntry*>(partials + (size_t)launches * kPartMax);
    int nparts = 0;
    int64_t base = 0;
    bool rewrite = max_norm < __builtin_inf();
    for (int i0 = 0; i0 < count; i0 += kClipItems) {
        ClipArgs a{};
        a.count = count - i0 < kClipItems ? count - i0 : kClipItems;
        a.table0 = i0;
        a.chunk_base = base;
        int64_t c = 0;
        for (int i = 0; i < a.count; i++) {
            a.e[i] = items[i0 + i];
            a.e[i].chunk0 = c;
            c += chunks_of(a.e[i].n);
            rewrite = rewrite || a.e[i].out != a.e[i].g;
        }
        if (c > INT32_MAX)
            return hipErrorInvalidValue;
        a.chunks = (int32_t)c;
        // an empty set of tensors still needs its table and one zero partial
        const int nb = c < 1 ? 1 : (c < kPartMax ? (int)c : kPartMax);
        hipLaunchKernelGGL(k_clip_sumsq, dim3(nb), dim3(kClipThreads), 0, s, a, table, partials + nparts);
        nparts += nb;
        base += c;
    }
    // with nothing to write (no limit, all in place) one block reports the norm
    const int nb = !rewrite || base < 1 ? 1 : (base < kScaleMax ? (int)base : kScaleMax);
    hipLaunchKernelGGL(k_clip_scale, dim3(nb), dim3(kClipThreads), 0, s, table, count, rewrite ? base : (int64_t)0,
                       partials, nparts, max_norm, norm);
    return hipGetLastError();
}

}  // namespace owq
