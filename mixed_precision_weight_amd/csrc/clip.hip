// clip.hip -- the global norm over many gradient tensors, and clipping by it (gfx950).
//
//   norm = sqrt(sum over every tensor and element of g^2)
//   out  = g * max_norm / norm  where norm > max_norm (and finite), else g
// both with the fp64 norm: the fp32 one that is reported is infinite also for finite
// gradients whose norm lies above fp32's range, and those are scaled.
//
// The weak columns of every linear are the parameters weak-column tuning trains,
// so a step has one small gradient per linear: hundreds of tensors of 10^5 - 10^6
// elements. Both passes therefore run over ONE sequence of 8192-element chunks that
// walks all tensors; a block owns a run of consecutive chunks, finds its first
// tensor by bisection and then only steps forward.
//
// Pass 1 (k_clip_sumsq, one launch per kClipItems tensors: their addresses and
// sizes travel in the kernel arguments, every block adds up the first chunks for
// itself, and one leaves the table in the workspace for pass 2) writes one fp64
// partial per block. Squares and sums are fp64: fp32 squares overflow from 1.8e19
// on, and the fp64 rate (two instructions per element) stays far below the memory
// time. Pass 2 (k_clip_scale, again one launch per kClipItems tensors, their outs in
// the arguments) adds the partials in a fixed order in every block (at most 2048
// per launch of pass 1, read from L2: cheaper than a launch that reduces them
// first), so the result does not depend on the launch's timing, and scales. The
// product is formed in fp64 and rounded to the tensor's type (fp16 by way of fp32).
// A tensor that stays as it is, in place, is neither read nor written by pass 2.
//
// Bound: memory, two reads and a write of every element; the second read comes from
// the 256 MB last-level cache where the tensors fit. Measured, 224 fp32 tensors of
// 5.1e7 elements: 57 us for pass 1 (3.5 TB/s) right after a call that wrote its outputs,
// which the caches write back meanwhile; 39 us (5.2 TB/s) after calls that wrote nothing
// or with 1 GiB read in between; 70 us for pass 2 (5.8 TB/s). With three launches of pass
// 1 in place of one it took 66 us.
#include "owq_device.h"
#include "owq_launch.h"

namespace owq {

namespace {

constexpr int kClipChunk = 8192;    // elements per chunk, both types
constexpr int kClipThreads = 256;
constexpr int kPer = kClipChunk / kClipThreads;  // elements per thread of a full chunk
constexpr int kPartMax = 2048;                   // blocks (and partials) per launch of pass 1: as many as the GPU holds at once
constexpr int kScaleMax = 2048;                  // blocks per launch of pass 2

// A run of tensors, 16 bytes each in the arguments of pass 1 (below 4 KB in all)
struct ClipArgs {
    const void* g[kClipItems];
    int64_t n2[kClipItems];  // 2 n + (1: fp16, 0: fp32)
    int32_t count;           // tensors of the run
    int32_t chunks;          // their chunks
};

struct ClipOuts {
    void* out[kClipItems];
    int32_t count, chunks;
};

// What pass 1 leaves for pass 2
struct ClipTable {
    const void* g;
    int64_t n2;
    int64_t chunk0;  // the tensor's first chunk in its run
};
static_assert(sizeof(ClipArgs) + 2 * sizeof(void*) <= 4096, "kernel arguments");

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

// 16 bytes at any element's address: the tensors may start anywhere, and unaligned
// pieces cost far less than single elements (37 fp16 tensors of 9e6 elements in all
// at odd addresses, pass 1: 13 us by elements, 7 by pieces)
typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));

// The tensors' addresses come from a table: the compiler has to be told that they
// are global memory, or it uses flat loads, which also wait on LDS
#define GLOBAL __attribute__((address_space(1)))
template <typename T>
__device__ __forceinline__ const GLOBAL T* global_at(const void* p, int64_t off)
{
    return (const GLOBAL T*)(uintptr_t)p + off;
}
template <typename T>
__device__ __forceinline__ GLOBAL T* global_at(void* p, int64_t off)
{
    return (GLOBAL T*)(uintptr_t)p + off;
}

__device__ __forceinline__ double sumsq4(f4_any v, double s)
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

// n elements at p (n <= kClipChunk). A whole chunk is read in 16-byte pieces, all in
// flight at once.
__device__ __forceinline__ double chunk_sumsq(const void* base, int64_t off, int n, bool half)
{
    const int t = threadIdx.x;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (half) {
        const GLOBAL uint16_t* p = global_at<uint16_t>(base, off);
        const GLOBAL u4_any* q = (const GLOBAL u4_any*)p;
        auto add = [&](u4_any v) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                s[e] = sumsq_h2(v[e], s[e]);
        };
        if (n == kClipChunk) {
            u4_any v[kPer / 8];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++)
                v[u] = q[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 8; u++)
                add(v[u]);
        } else {
            for (int i = t; i < n / 8; i += kClipThreads)
                add(q[i]);
            if (t < n % 8)
                s[0] = sumsq_h2(p[n - 1 - t], s[0]);
        }
    } else {
        const GLOBAL float* p = global_at<float>(base, off);
        const GLOBAL f4_any* q = (const GLOBAL f4_any*)p;
        if (n == kClipChunk) {
            f4_any v[kPer / 4];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                v[u] = q[t + kClipThreads * u];
#pragma unroll
            for (int u = 0; u < kPer / 4; u++)
                s[u & 3] = sumsq4(v[u], s[u & 3]);
        } else {
            for (int i = t; i < n / 4; i += kClipThreads)
                s[0] = sumsq4(q[i], s[0]);
            if (t < n % 4)
                s[1] = __builtin_fma((double)p[n - 1 - t], (double)p[n - 1 - t], s[1]);
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ int64_t chunks_of(int64_t n) { return (n + kClipChunk - 1) / kClipChunk; }

// Block b's first chunk where `most` blocks share them, or a block has one
template <int most>
__device__ __forceinline__ int first_chunk(int chunks, int b)
{
    return chunks <= most ? min(b, chunks) : (int)((int64_t)chunks * b / most);
}

// The last of count tensors whose first chunk is at most c (empty tensors share it
// with their successor)
template <typename F>
__device__ __forceinline__ int tensor_of(int count, int64_t c, F first)
{
    int li = 0;
    for (int lo = 0, hi = count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (first(mid) <= c)
            lo = mid;
        else
            hi = mid;
        li = lo;
    }
    return li;
}

__global__ __launch_bounds__(kClipThreads) __attribute__((amdgpu_waves_per_eu(8))) void k_clip_sumsq(const ClipArgs a, ClipTable* table, double* partials)
{
    static_assert(kClipItems <= kClipThreads, "one tensor of a run per thread");
    __shared__ double red[4];
    __shared__ int first[kClipItems], part[4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    // the tensors' first chunks (a run has fewer than 2^31 chunks)
    const int own = t < a.count ? (int)chunks_of(a.n2[t] >> 1) : 0;
    int upto = own;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int v = __shfl_up(upto, o, 64);
        upto += lane >= o ? v : 0;
    }
    if (lane == 63)
        part[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; w++)
        upto += part[w];
    if (t < a.count) {
        first[t] = upto - own;
        if (blockIdx.x == 0)
            table[t] = ClipTable{a.g[t], a.n2[t], upto - own};
    }
    __syncthreads();
    const int c0 = first_chunk<kPartMax>(a.chunks, blockIdx.x), c1 = first_chunk<kPartMax>(a.chunks, blockIdx.x + 1);
    int li = __builtin_amdgcn_readfirstlane(tensor_of(a.count, c0, [&](int i) { return first[i]; }));
    double s = 0.0;
    for (int c = c0; c < c1; c++) {
        while (li + 1 < a.count && __builtin_amdgcn_readfirstlane(first[li + 1]) <= c)
            li++;
        const int64_t off = (int64_t)(c - __builtin_amdgcn_readfirstlane(first[li])) * kClipChunk;
        const int64_t left = (a.n2[li] >> 1) - off;
        s += chunk_sumsq(a.g[li], off, (int)(left < kClipChunk ? left : kClipChunk), (a.n2[li] & 1) != 0);
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = s;
}

__device__ __forceinline__ float scaled(float v, double c) { return (float)((double)v * c); }

// To fp16 by way of fp32, a conversion of the hardware each (from fp64 the compiler
// would make some 40 instructions per value: 18 us against 9 for 9e6 values). The
// step in between adds 2^-13 of fp16's rounding error.
__device__ __forceinline__ uint16_t scaled_half(uint16_t v, double c)
{
    float f = scaled(h2f(v), c);
    asm volatile("" : "+v"(f));
    return f2h(f);
}

__device__ __forceinline__ uint32_t scaled_h2(uint32_t v, double c)
{
    return scaled_half((uint16_t)(v & 0xffffu), c) | ((uint32_t)scaled_half((uint16_t)(v >> 16), c) << 16);
}

// out = g * c, c == 1: an exact copy
template <typename V, typename E, typename MV, typename ME>
__device__ __forceinline__ void scale_pieces(const GLOBAL E* p, GLOBAL E* o, int n, MV mulv, ME mul)
{
    constexpr int VE = 16 / sizeof(E), U = kPer / VE;
    const int t = threadIdx.x;
    const GLOBAL V* q = (const GLOBAL V*)p;
    GLOBAL V* r = (GLOBAL V*)o;
    if (n == kClipChunk) {  // all loads in flight at once
        V v[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            v[u] = q[t + kClipThreads * u];
#pragma unroll
        for (int u = 0; u < U; u++)
            r[t + kClipThreads * u] = mulv(v[u]);
    } else {
        for (int i = t; i < n / VE; i += kClipThreads)
            r[i] = mulv(q[i]);
        if (t < n % VE)
            o[n - 1 - t] = mul(p[n - 1 - t]);
    }
}

__device__ __forceinline__ void chunk_scale(const void* g, void* out, bool half, int64_t off, int n, double c)
{
    if (half)
        scale_pieces<u4_any>(
            global_at<uint16_t>(g, off), global_at<uint16_t>(out, off), n,
            [&](u4_any v) {
                return u4_any{scaled_h2(v[0], c), scaled_h2(v[1], c), scaled_h2(v[2], c), scaled_h2(v[3], c)};
            },
            [&](uint16_t v) { return scaled_half(v, c); });
    else
        scale_pieces<f4_any>(
            global_at<float>(g, off), global_at<float>(out, off), n,
            [&](f4_any v) { return f4_any{scaled(v[0], c), scaled(v[1], c), scaled(v[2], c), scaled(v[3], c)}; },
            [&](float v) { return scaled(v, c); });
}

__global__ __launch_bounds__(kClipThreads) __attribute__((amdgpu_waves_per_eu(8))) void k_clip_scale(const ClipOuts a, const ClipTable* __restrict__ table,
                                                             const double* __restrict__ partials, int nparts,
                                                             double max_norm, float* norm)
{
    __shared__ double red[4];
    __shared__ ClipTable e[kClipItems];
    if ((int)threadIdx.x < a.count)
        e[threadIdx.x] = table[threadIdx.x];
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads)
        s += partials[i];
    const double total = sqrt(block_sum(s, red));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = (float)total;
    // NaN compares false, and an infinite norm leaves the tensors alone too
    const double c = total > max_norm && total < __builtin_inf() ? max_norm / total : 1.0;
    const int c0 = first_chunk<kScaleMax>(a.chunks, blockIdx.x), c1 = first_chunk<kScaleMax>(a.chunks, blockIdx.x + 1);
    if (c0 >= c1)
        return;
    // (block_sum's barriers lie between e's stores and its reads)
    int li = __builtin_amdgcn_readfirstlane(tensor_of(a.count, c0, [&](int i) { return e[i].chunk0; }));
    for (int k = c0; k < c1; k++) {
        while (li + 1 < a.count && e[li + 1].chunk0 <= k)
            li++;
        void* const out = a.out[li];
        if (c == 1.0 && out == e[li].g)
            continue;
        const int64_t off = (k - e[li].chunk0) * kClipChunk;
        const int64_t left = (e[li].n2 >> 1) - off;
        chunk_scale(e[li].g, out, (e[li].n2 & 1) != 0, off, (int)(left < kClipChunk ? left : kClipChunk), c);
    }
}

}  // namespace

size_t clip_workspace_bytes(int count)
{
    const int launches = (count + kClipItems - 1) / kClipItems;
    return (size_t)launches * kPartMax * sizeof(double) + (size_t)count * sizeof(ClipTable);
}

hipError_t launch_clip(const ClipEntry* items, int count, double max_norm, float* norm, void* ws, hipStream_t s)
{
    const int launches = (count + kClipItems - 1) / kClipItems;
    double* const partials = static_cast<double*>(ws);
    ClipTable* const table = reinterpret_cast<ClipTable*>(partials + (size_t)launches * kPartMax);
    auto chunks = [&](int i0) {  // of the run that starts at tensor i0
        int64_t c = 0;
        for (int i = i0; i < count && i < i0 + kClipItems; i++)
            c += (items[i].n + kClipChunk - 1) / kClipChunk;
        return c;
    };
    for (int i0 = 0; i0 < count; i0 += kClipItems)
        if (chunks(i0) > INT32_MAX)
            return hipErrorInvalidConfiguration;
    int nparts = 0;
    for (int i0 = 0; i0 < count; i0 += kClipItems) {
        ClipArgs a{};
        a.count = count - i0 < kClipItems ? count - i0 : kClipItems;
        a.chunks = (int32_t)chunks(i0);
        for (int i = 0; i < a.count; i++) {
            a.g[i] = items[i0 + i].g;
            a.n2[i] = 2 * items[i0 + i].n + (items[i0 + i].half ? 1 : 0);
        }
        // a run of empty tensors still needs one zero partial
        const int nb = a.chunks < 1 ? 1 : (a.chunks < kPartMax ? a.chunks : kPartMax);
        hipLaunchKernelGGL(k_clip_sumsq, dim3(nb), dim3(kClipThreads), 0, s, a, table + i0, partials + nparts);
        nparts += nb;
    }
    for (int i0 = 0; i0 < count; i0 += kClipItems) {
        ClipOuts a{};
        a.count = count - i0 < kClipItems ? count - i0 : kClipItems;
        bool rewrite = max_norm < __builtin_inf();
        for (int i = 0; i < a.count; i++) {
            a.out[i] = items[i0 + i].out;
            rewrite = rewrite || a.out[i] != items[i0 + i].g;
        }
        // with nothing to write (no limit, all in place) one block reports the norm
        a.chunks = rewrite ? (int32_t)chunks(i0) : 0;
        if (a.chunks == 0 && i0 > 0)
            continue;
        const int nb = a.chunks < 1 ? 1 : (a.chunks < kScaleMax ? a.chunks : kScaleMax);
        hipLaunchKernelGGL(k_clip_scale, dim3(nb), dim3(kClipThreads), 0, s, a, table + i0, partials, nparts, max_norm,
                           i0 == 0 ? norm : nullptr);
    }
    return hipGetLastError();
}

}  // namespace owq
