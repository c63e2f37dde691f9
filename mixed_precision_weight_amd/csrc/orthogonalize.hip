// orthogonalize.hip -- many matrices, each replaced by a nearly orthogonal factor of
// itself by Newton-Schulz products (gfx950).
//
//   X = G / (|G|_F + eps);  steps times: X <- a X + b (X X^T) X + c (X X^T)^2 X;  out = scale X
//
// With s the short side, S = X X^T (or X^T X) is s x s, and the steps act on it alone: for
// p(S) = a + b S + c S^2, X <- p(S) X and S <- S p(S)^2 (everything commutes). So a matrix
// with a short side of up to kNsShort (the weak columns' gradients, low-rank factors) is
// read twice and written once: its Gram matrix, the polynomial of it, the product. The
// Gram matrix squares the singular values, and the polynomial lifts the small ones by
// up to a^steps: both run in fp64 (in fp32 a direction at 1e-3 of the largest would come
// out 1 % off). Longer short sides run the steps as they stand, X in fp32.
#include "owq_device.h"
#include "owq_launch.h"

namespace owq {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float nf4 __attribute__((ext_vector_type(4)));
typedef float nf16 __attribute__((ext_vector_type(16)));

// One matrix as the kernels see it (device table, written by k_ns_table)
struct NsItem {
    const void* g;
    void* out;
    int64_t off;      // bytes into the workspace: its part
    int32_t rows, cols;
    float scale;
    int32_t half;     // 1: fp16, 0: fp32
    int32_t slices;   // of the long side (short form: Gram partials; long form: split sums)
    int32_t block0;   // first block of its class's Gram launch
    int32_t apply0;   // first block of its class's last launch
    int32_t pad;
};
static_assert(sizeof(NsItem) == 56, "table entry");

constexpr int kNsArg = 64;  // table entries per launch of k_ns_table (kernel arguments below 4 KB)
struct NsArgs {
    NsItem it[kNsArg];
    int32_t count;
};

__global__ __launch_bounds__(64) void k_ns_table(const NsArgs a, NsItem* table)
{
    if ((int)threadIdx.x < a.count)
        table[threadIdx.x] = a.it[threadIdx.x];
}

#define NS_GLOBAL __attribute__((address_space(1)))

__device__ __forceinline__ __amdgpu_buffer_rsrc_t ns_rsrc(const char* p, int64_t bytes)
{
    const uint64_t u = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    const int n = __builtin_amdgcn_readfirstlane((int)(bytes < 0x7fffffff ? (bytes > 0 ? bytes : 0) : 0x7fffffff));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uintptr_t)(((uint64_t)hi << 32) | lo)), (short)0, n,
                                             0x00020000);
}

// element at byte offset off (elements of 2 or 4 bytes); out of range: 0
__device__ __forceinline__ float ns_load(__amdgpu_buffer_rsrc_t r, int off, bool half)
{
    if (half)
        return h2f((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
    return __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

constexpr int kNsDead = 0x7ffffff0;  // an offset that is out of every buffer's range

// the item whose blocks hold block b: items are in block order
template <typename F>
__device__ __forceinline__ int ns_item(const NsItem* t, int count, int b, F first)
{
    int lo = 0;
    for (int hi = count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (first(t[mid]) <= b)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ------------------------------------------------------ short form: the Gram matrix --

constexpr int tri(int T) { return T * (T + 1) / 2; }

// A block sums one slice of the long side: v_mfma_f64_16x16x4_f64, the same register as
// both operands (lane l: short index l % 16 of a tile, long index l / 16). The partial
// sums are kept in lane order, a tile pair (ti <= tj) after the other.
template <int T>
__global__ __launch_bounds__(256) void k_ns_gram(const NsItem* __restrict__ table, int count, char* ws)
{
    __shared__ double red[4][256];
    const NsItem it = table[ns_item(table, count, blockIdx.x, [](const NsItem& i) { return i.block0; })];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slice = (int)blockIdx.x - it.block0;
    const bool half = it.half != 0, tall = it.rows > it.cols;
    const int sh = half ? 1 : 2;
    const int s = min(it.rows, it.cols), L = max(it.rows, it.cols);
    const int per = ((L + it.slices - 1) / it.slices + 3) & ~3;
    const int l0 = min(L, slice * per), len = min(L, l0 + per) - l0;
    const int i16 = lane & 15, kk = lane >> 4;
    f64x4 acc[tri(T)];
#pragma unroll
    for (int p = 0; p < tri(T); p++)
        acc[p] = f64x4{0.0, 0.0, 0.0, 0.0};
    constexpr int U = T <= 2 ? 16 : (T <= 4 ? 8 : 4);  // 4-row steps in flight
    const char* base = static_cast<const char*>(it.g);
    // element (short i, long l) of the slice
    const int64_t si = tall ? 1 : it.cols, sl = tall ? it.cols : 1;
    base += (l0 * sl) << sh;
    const __amdgpu_buffer_rsrc_t r =
        ns_rsrc(base, (tall ? (int64_t)len * it.cols : (int64_t)it.rows * it.cols - l0) << sh);
    int off[T];
#pragma unroll
    for (int t = 0; t < T; t++)
        off[t] = t * 16 + i16 < s ? (int)(((t * 16 + i16) * si + kk * sl) << sh) : kNsDead;
    const int step = (int)(sl * 4 << sh);
    for (int b = wave * U; b < (len + 3) >> 2; b += 4 * U) {
        float v[U][T];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = (b + u) * 4 + kk < len;
#pragma unroll
            for (int t = 0; t < T; t++)
                v[u][t] = ns_load(r, in && off[t] != kNsDead ? off[t] + (b + u) * step : kNsDead, half);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            double d[T];
#pragma unroll
            for (int t = 0; t < T; t++)
                d[t] = (double)v[u][t];
            int p = 0;
#pragma unroll
            for (int ti = 0; ti < T; ti++)
#pragma unroll
                for (int tj = ti; tj < T; tj++, p++)
                    acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[ti], d[tj], acc[p], 0, 0, 0);
        }
    }
    double* part = reinterpret_cast<double*>(ws + it.off) + (int64_t)slice * tri(T) * 256;
#pragma unroll
    for (int p = 0; p < tri(T); p++) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; q++)
            red[wave][q * 64 + lane] = acc[p][q];
        __syncthreads();
        part[p * 256 + tid] = ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid];
    }
}

// ------------------------------------------------------- short form: the polynomial --

// Element q of lane l of a 16 x 16 fp64 result: row 4 q + l / 16, column l % 16
__device__ __forceinline__ int ns_drow(int q, int lane) { return 4 * q + (lane >> 4); }

template <int T, int NW>
struct NsPoly {
    static constexpr int S = 16 * T;
    static constexpr int TILES = (tri(T) + NW - 1) / NW;  // result tiles per wave
};

// X Y for symmetric matrices that commute, the upper tiles of this wave
template <int T, int NW>
__device__ __forceinline__ void ns_mul(const double (*X)[16 * T], const double (*Y)[16 * T], f64x4 (&acc)[NsPoly<T, NW>::TILES],
                                       const int (&ti)[NsPoly<T, NW>::TILES], const int (&tj)[NsPoly<T, NW>::TILES], int lane)
{
    const int i16 = lane & 15, kk = lane >> 4;
#pragma unroll
    for (int p = 0; p < NsPoly<T, NW>::TILES; p++)
        acc[p] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
    for (int k0 = 0; k0 < 16 * T; k0 += 4)
#pragma unroll
        for (int p = 0; p < NsPoly<T, NW>::TILES; p++)
            acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(X[k0 + kk][ti[p] * 16 + i16], Y[k0 + kk][tj[p] * 16 + i16], acc[p],
                                                          0, 0, 0);
}

template <int T, int NW>
__device__ __forceinline__ void ns_store(double (*X)[16 * T], const f64x4 (&v)[NsPoly<T, NW>::TILES],
                                         const int (&ti)[NsPoly<T, NW>::TILES], const int (&tj)[NsPoly<T, NW>::TILES], int lane)
{
#pragma unroll
    for (int p = 0; p < NsPoly<T, NW>::TILES; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            // (below the diagonal of a tile on it: the mirror image, whose sum may round otherwise)
            const int r = ti[p] * 16 + ns_drow(q, lane), c = tj[p] * 16 + (lane & 15);
            if (r <= c) {
                X[r][c] = v[p][q];
                X[c][r] = v[p][q];
            }
        }
}

struct NsCoef {
    double a, b, c, eps;
    int32_t steps;
};

// One block per matrix: sums the partials, |G|^2 is their trace; then the steps. Waves
// past the tiles repeat the last tile (the same values to the same places).
template <int T, int NW>
__global__ __launch_bounds__(64 * NW) void k_ns_poly(const NsItem* __restrict__ table, char* ws, const NsCoef k)
{
    constexpr int S = 16 * T, TL = NsPoly<T, NW>::TILES;
    __shared__ double A[S][S];
    __shared__ double Q[S][S];
    const NsItem it = table[blockIdx.x];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int ti[TL], tj[TL], tp[TL];
#pragma unroll
    for (int p = 0; p < TL; p++) {
        int n = min(wave * TL + p, tri(T) - 1);
        tp[p] = n;
        int i = 0;
        while (n >= T - i) {
            n -= T - i;
            i++;
        }
        ti[p] = i;
        tj[p] = i + n;
    }
    const double* part = reinterpret_cast<const double*>(ws + it.off);
    f64x4 v[TL], P[TL], N[TL];
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            double x = 0.0;
            for (int sl = 0; sl < it.slices; sl++)
                x += part[((int64_t)sl * tri(T) + tp[p]) * 256 + q * 64 + lane];
            v[p][q] = x;
        }
    ns_store<T, NW>(A, v, ti, tj, lane);
    __syncthreads();
    double tr = 0.0;
    for (int i = 0; i < S; i++)
        tr += A[i][i];
    const double inv = 1.0 / (sqrt(tr) + k.eps);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < TL; p++)
        v[p] = v[p] * inv * inv;
    ns_store<T, NW>(A, v, ti, tj, lane);
    __syncthreads();
    for (int t = 0; t < k.steps; t++) {
        // v: A's tiles. N = A^2, then Q = a + b A + c A^2
        ns_mul<T, NW>(A, A, N, ti, tj, lane);
#pragma unroll
        for (int p = 0; p < TL; p++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const bool diag = ti[p] == tj[p] && ns_drow(q, lane) == (lane & 15);
                N[p][q] = k.c * N[p][q] + k.b * v[p][q] + (diag ? k.a : 0.0);
            }
        ns_store<T, NW>(Q, N, ti, tj, lane);
        __syncthreads();
        const bool last = t + 1 == k.steps;
        if (!last) {  // A <- (A Q) Q
            ns_mul<T, NW>(A, Q, v, ti, tj, lane);
            __syncthreads();
            ns_store<T, NW>(A, v, ti, tj, lane);
            __syncthreads();
            ns_mul<T, NW>(A, Q, v, ti, tj, lane);
            __syncthreads();
        }
        if (t == 0) {
#pragma unroll
            for (int p = 0; p < TL; p++)
                P[p] = N[p];
        } else {  // P <- P Q, through A's place
            ns_store<T, NW>(A, P, ti, tj, lane);
            __syncthreads();
            ns_mul<T, NW>(A, Q, P, ti, tj, lane);
            __syncthreads();
        }
        if (!last) {
            ns_store<T, NW>(A, v, ti, tj, lane);
            __syncthreads();
        }
    }
    // the matrix's factor, with the norm and the scale, over the first partials
    float* out = reinterpret_cast<float*>(ws + it.off);
    const double f = inv * (double)it.scale;
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = ti[p] * 16 + ns_drow(q, lane), c = tj[p] * 16 + (lane & 15);
            const float x = (float)(P[p][q] * f);
            if (r <= c) {
                out[r * S + c] = x;
                out[c * S + r] = x;
            }
        }
}

// --------------------------------------------------------- short form: the product --

constexpr int kNsRun = 8;  // 16-element runs of the long side per wave

// out = G F (tall) or F G (wide), F the symmetric factor: v_mfma_f32_16x16x4_f32 with F's
// rows as A and G as B; a wave holds a run of 16 of the long side in registers before it
// writes any of it, so out may be G. The contraction index 16 st + 4 (l / 16) + u is taken
// by product u of step st, so that a lane's four are consecutive.
template <int T>
__global__ __launch_bounds__(256) void k_ns_apply(const NsItem* __restrict__ table, int count, const char* ws)
{
    constexpr int S = 16 * T, LD = S + 4;
    __shared__ float F[S][LD];
    const NsItem it = table[ns_item(table, count, blockIdx.x, [](const NsItem& i) { return i.apply0; })];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float* f = reinterpret_cast<const float*>(ws + it.off);
    for (int e = tid; e < S * S; e += 256)
        F[e / S][e % S] = f[e];
    __syncthreads();
    const bool half = it.half != 0, tall = it.rows > it.cols;
    const int sh = half ? 1 : 2;
    const int s = min(it.rows, it.cols), L = max(it.rows, it.cols);
    const int n16 = lane & 15, kk = lane >> 4;
    const int64_t si = tall ? 1 : it.cols, sl = tall ? it.cols : 1;
    const int l0 = ((int)blockIdx.x - it.apply0) * 64 * kNsRun + wave * 16 * kNsRun;
    for (int run = 0; run < kNsRun; run++) {
        const int lb = l0 + run * 16;
        if (lb >= L)
            return;
        const int len = min(16, L - lb);
        const char* base = static_cast<const char*>(it.g) + ((lb * sl) << sh);
        const __amdgpu_buffer_rsrc_t r = ns_rsrc(base, (tall ? (int64_t)len * it.cols : (int64_t)it.rows * it.cols - lb) << sh);
        float v[T][4];
#pragma unroll
        for (int st = 0; st < T; st++)
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int i = 16 * st + 4 * kk + u;
                v[st][u] = ns_load(r, i < s && n16 < len ? (int)((i * si + n16 * sl) << sh) : kNsDead, half);
            }
        nf4 acc[T];
#pragma unroll
        for (int t = 0; t < T; t++)
            acc[t] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < T; st++)
#pragma unroll
            for (int t = 0; t < T; t++) {
                const nf4 a = *reinterpret_cast<const nf4*>(&F[t * 16 + n16][16 * st + 4 * kk]);
#pragma unroll
                for (int u = 0; u < 4; u++)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[u], v[st][u], acc[t], 0, 0, 0);
            }
        if (n16 < len) {
            char* ob = static_cast<char*>(it.out) + ((lb * sl) << sh);
#pragma unroll
            for (int t = 0; t < T; t++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int i = t * 16 + 4 * kk + q;
                    if (i < s) {
                        const int64_t at = i * si + n16 * sl;
                        if (half)
                            ((NS_GLOBAL uint16_t*)(uintptr_t)ob)[at] = f2h(acc[t][q]);
                        else
                            ((NS_GLOBAL float*)(uintptr_t)ob)[at] = acc[t][q];
                    }
                }
        }
    }
}

// ----------------------------------------------------------------- long form --

// Workspace of one matrix of the long form, fp32, X with the long side contiguous and
// both sides padded to 64 with zeros (the products need no edges): X, X', A, B, then
// the split sums of A, then the partial sums of squares.
struct NsLong {
    int64_t sp, lp;
    int64_t x0, x1, A, B, parts, sq, total;  // byte offsets
    int32_t splits, sqn;
};

__host__ __device__ inline NsLong ns_long(int64_t rows, int64_t cols)
{
    NsLong n{};
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    n.sp = (s + 63) / 64 * 64;
    n.lp = (l + 63) / 64 * 64;
    const int64_t tiles = (n.sp / 64) * (n.sp / 64 + 1) / 2;
    // 256 CUs want two blocks each; a split takes at least 256 of the long side
    int64_t sp = (512 + tiles - 1) / tiles;
    sp = sp < n.lp / 256 ? sp : n.lp / 256;
    n.splits = (int32_t)(sp < 1 ? 1 : sp);
    n.sqn = (int32_t)((rows * cols + 16383) / 16384 < 1024 ? (rows * cols + 16383) / 16384 : 1024);
    int64_t off = 0;
    n.x0 = off, off += 4 * n.sp * n.lp;
    n.x1 = off, off += 4 * n.sp * n.lp;
    n.A = off, off += 4 * n.sp * n.sp;
    n.B = off, off += 4 * n.sp * n.sp;
    n.parts = off, off += n.splits > 1 ? 4 * n.splits * n.sp * n.sp : 0;
    n.sq = off, off += 8 * n.sqn;
    n.total = (off + 255) / 256 * 256;
    return n;
}

__device__ __forceinline__ double ns_block_sum(double v, double* red)
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

// blockIdx.y: the matrix, in all kernels of the long form
__global__ __launch_bounds__(256) void k_nsl_sumsq(const NsItem* __restrict__ table, char* ws)
{
    __shared__ double red[4];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    if ((int)blockIdx.x >= n.sqn)
        return;
    const int64_t total = (int64_t)it.rows * it.cols;
    double s = 0.0;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)n.sqn * 256) {
        const float v = it.half ? h2f(static_cast<const uint16_t*>(it.g)[e]) : static_cast<const float*>(it.g)[e];
        s = __builtin_fma((double)v, (double)v, s);
    }
    s = ns_block_sum(s, red);
    if (threadIdx.x == 0)
        reinterpret_cast<double*>(ws + it.off + n.sq)[blockIdx.x] = s;
}

// X = G / (|G| + eps), the long side contiguous, padded with zeros. 64 x 64 tiles.
__global__ __launch_bounds__(256) void k_nsl_init(const NsItem* __restrict__ table, char* ws, double eps)
{
    __shared__ double red[4];
    __shared__ float tile[64][65];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t tl = n.lp / 64;
    if (blockIdx.x >= (n.sp / 64) * tl)
        return;
    const double* sq = reinterpret_cast<const double*>(ws + it.off + n.sq);
    double s = 0.0;
    for (int i = threadIdx.x; i < n.sqn; i += 256)
        s += sq[i];
    const double inv = 1.0 / (sqrt(ns_block_sum(s, red)) + eps);
    const bool tall = it.rows > it.cols;
    const int64_t i0 = blockIdx.x / tl * 64, l0 = blockIdx.x % tl * 64;
    const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    for (int r = r0; r < 64; r += 4) {
        const int64_t row = (tall ? l0 : i0) + r, col = (tall ? i0 : l0) + c;
        float v = 0.0f;
        if (row < it.rows && col < it.cols) {
            const int64_t e = row * it.cols + col;
            v = it.half ? h2f(static_cast<const uint16_t*>(it.g)[e]) : static_cast<const float*>(it.g)[e];
            v = (float)((double)v * inv);
        }
        tile[r][c] = v;
    }
    __syncthreads();
    float* x = reinterpret_cast<float*>(ws + it.off + n.x0);
    for (int r = r0; r < 64; r += 4)
        x[(i0 + r) * n.lp + l0 + c] = tall ? tile[c][r] : tile[r][c];
}

// out = scale X
__global__ __launch_bounds__(256) void k_nsl_out(const NsItem* __restrict__ table, const char* ws, int from1)
{
    __shared__ float tile[64][65];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t tl = n.lp / 64;
    if (blockIdx.x >= (n.sp / 64) * tl)
        return;
    const bool tall = it.rows > it.cols;
    const int64_t i0 = blockIdx.x / tl * 64, l0 = blockIdx.x % tl * 64;
    const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    const float* x = reinterpret_cast<const float*>(ws + it.off + (from1 ? n.x1 : n.x0));
    for (int r = r0; r < 64; r += 4)
        tile[r][c] = x[(i0 + r) * n.lp + l0 + c] * it.scale;
    __syncthreads();
    for (int r = r0; r < 64; r += 4) {
        const int64_t row = (tall ? l0 : i0) + r, col = (tall ? i0 : l0) + c;
        if (row < it.rows && col < it.cols) {
            const float v = tall ? tile[c][r] : tile[r][c];
            const int64_t e = row * it.cols + col;
            if (it.half)
                static_cast<uint16_t*>(it.out)[e] = f2h(v);
            else
                static_cast<float*>(it.out)[e] = v;
        }
    }
}

// acc[4] += 64 x 64 tile of Xrows Yrows^T over columns k0 .. k1 (NT: both with the
// contraction contiguous), or of Xrows Y (NN: Y [k][ldy]). 4 waves of 32 x 32, v_mfma_f32_32x32x2.
template <bool NT>
__device__ __forceinline__ void ns_tile(const float* X, int64_t ldx, const float* Y, int64_t ldy, int64_t k0, int64_t k1,
                                        nf16& acc)
{
    constexpr int KC = 32;
    __shared__ float xs[64][KC + 1];
    __shared__ float ys[NT ? 64 : KC][NT ? KC + 1 : 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l32 = lane & 31, h = lane >> 5, wm = wave & 1, wn = wave >> 1;
    for (int64_t k = k0; k < k1; k += KC) {
        nf4 xv[2], yv[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int u = t * 256 + tid;
            xv[t] = *reinterpret_cast<const nf4*>(X + (u >> 3) * ldx + k + (u & 7) * 4);
            yv[t] = NT ? *reinterpret_cast<const nf4*>(Y + (u >> 3) * ldy + k + (u & 7) * 4)
                       : *reinterpret_cast<const nf4*>(Y + (k + (u >> 4)) * ldy + (u & 15) * 4);
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int u = t * 256 + tid;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                xs[u >> 3][(u & 7) * 4 + e] = xv[t][e];
                if (NT)
                    ys[u >> 3][(u & 7) * 4 + e] = yv[t][e];
                else
                    ys[u >> 4][(u & 15) * 4 + e] = yv[t][e];
            }
        }
        __syncthreads();
#pragma unroll
        for (int st = 0; st < KC / 2; st++) {
            const float a = xs[wm * 32 + l32][2 * st + h];
            const float b = NT ? ys[wn * 32 + l32][2 * st + h] : ys[2 * st + h][wn * 32 + l32];
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc, 0, 0, 0);
        }
    }
}

__device__ __forceinline__ void ns_upper(int64_t n, int64_t T, int64_t& ti, int64_t& tj)
{
    int64_t i = 0;
    while (n >= T - i) {
        n -= T - i;
        i++;
    }
    ti = i;
    tj = i + n;
}

// row and column of element r of a lane in the block's 64 x 64 tile
__device__ __forceinline__ int ns_row(int r)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    return (wave & 1) * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
}
__device__ __forceinline__ int ns_col() { return (threadIdx.x >> 7) * 32 + (threadIdx.x & 31); }

// A = X X^T: upper tiles, `splits` parts of the long side each
__global__ __launch_bounds__(256) void k_nsl_gram(const NsItem* __restrict__ table, char* ws, int from1)
{
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t T = n.sp / 64, tiles = T * (T + 1) / 2;
    if (blockIdx.x >= tiles * n.splits)
        return;
    int64_t ti, tj;
    ns_upper(blockIdx.x / n.splits, T, ti, tj);
    const int64_t sl = blockIdx.x % n.splits, per = (n.lp / 64 + n.splits - 1) / n.splits * 64;
    const int64_t k0 = sl * per, k1 = k0 + per < n.lp ? k0 + per : n.lp;
    const float* x = reinterpret_cast<const float*>(ws + it.off + (from1 ? n.x1 : n.x0));
    nf16 acc;
#pragma unroll
    for (int r = 0; r < 16; r++)
        acc[r] = 0.0f;
    ns_tile<true>(x + ti * 64 * n.lp, n.lp, x + tj * 64 * n.lp, n.lp, k0, k1, acc);
    float* out = reinterpret_cast<float*>(ws + it.off + (n.splits > 1 ? n.parts : n.A)) + (n.splits > 1 ? sl * n.sp * n.sp : 0);
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const int64_t row = ti * 64 + ns_row(r), col = tj * 64 + ns_col();
        if (row <= col) {
            out[row * n.sp + col] = acc[r];
            if (n.splits == 1)
                out[col * n.sp + row] = acc[r];
        }
    }
}

// the parts' sums, and their mirror image
__global__ __launch_bounds__(256) void k_nsl_sum(const NsItem* __restrict__ table, char* ws)
{
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t T = n.sp / 64, tiles = T * (T + 1) / 2;
    if (n.splits == 1 || blockIdx.x >= tiles * 16)
        return;
    int64_t ti, tj;
    ns_upper(blockIdx.x >> 4, T, ti, tj);
    const int64_t row = ti * 64 + ((blockIdx.x & 15) * 4 + (threadIdx.x >> 6)), col = tj * 64 + (threadIdx.x & 63);
    if (row > col)
        return;
    const float* p = reinterpret_cast<const float*>(ws + it.off + n.parts) + row * n.sp + col;
    float s = 0.0f;
    for (int i = 0; i < n.splits; i++)
        s += p[i * n.sp * n.sp];
    float* A = reinterpret_cast<float*>(ws + it.off + n.A);
    A[row * n.sp + col] = s;
    A[col * n.sp + row] = s;
}

// B = b A + c A^2
__global__ __launch_bounds__(256) void k_nsl_poly(const NsItem* __restrict__ table, char* ws, float b, float c)
{
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t T = n.sp / 64;
    if (blockIdx.x >= T * (T + 1) / 2)
        return;
    int64_t ti, tj;
    ns_upper(blockIdx.x, T, ti, tj);
    const float* A = reinterpret_cast<const float*>(ws + it.off + n.A);
    nf16 acc;
#pragma unroll
    for (int r = 0; r < 16; r++)
        acc[r] = 0.0f;
    ns_tile<true>(A + ti * 64 * n.sp, n.sp, A + tj * 64 * n.sp, n.sp, 0, n.sp, acc);
    float* B = reinterpret_cast<float*>(ws + it.off + n.B);
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const int64_t row = ti * 64 + ns_row(r), col = tj * 64 + ns_col();
        const float v = __builtin_fmaf(c, acc[r], b * A[row * n.sp + col]);
        if (row <= col) {
            B[row * n.sp + col] = v;
            B[col * n.sp + row] = v;
        }
    }
}

// X' = a X + B X
__global__ __launch_bounds__(256) void k_nsl_step(const NsItem* __restrict__ table, char* ws, float a, int from1)
{
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t T = n.sp / 64;
    if (blockIdx.x >= T * (n.lp / 64))
        return;
    const int64_t ti = blockIdx.x % T, tl = blockIdx.x / T;
    const float* x = reinterpret_cast<const float*>(ws + it.off + (from1 ? n.x1 : n.x0));
    float* y = reinterpret_cast<float*>(ws + it.off + (from1 ? n.x0 : n.x1));
    const float* B = reinterpret_cast<const float*>(ws + it.off + n.B);
    nf16 acc;
#pragma unroll
    for (int r = 0; r < 16; r++)
        acc[r] = 0.0f;
    ns_tile<false>(B + ti * 64 * n.sp, n.sp, x + tl * 64, n.lp, 0, n.sp, acc);
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const int64_t at = (ti * 64 + ns_row(r)) * n.lp + tl * 64 + ns_col();
        y[at] = __builtin_fmaf(a, x[at], acc[r]);
    }
}

// ------------------------------------------------------------------ the plan --

constexpr int kNsShort = 96;  // short sides of the short form
int ns_class(int64_t s) { return s > kNsShort ? 3 : (s > 64 ? 2 : (s > 32 ? 1 : 0)); }
constexpr int kNsTiles[3] = {2, 4, 6};

// slices of the long side in the short form: at least 256 long, 64 at most (their
// partials are added by one block)
int ns_slices(int64_t l)
{
    const int64_t n = (l + 255) / 256;
    return (int)(n < 64 ? n : 64);
}

int64_t ns_bytes(int64_t rows, int64_t cols)
{
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    if (s == 0)
        return 0;
    const int c = ns_class(s);
    if (c == 3)
        return ns_long(rows, cols).total;
    const int64_t part = (int64_t)ns_slices(l) * tri(kNsTiles[c]) * 2048, f = 4LL * 256 * kNsTiles[c] * kNsTiles[c];
    return ((part > f ? part : f) + 255) / 256 * 256;
}

}  // namespace

size_t orthogonalize_workspace_bytes(const OrthoEntry* items, int count)
{
    int64_t total = ((int64_t)count * sizeof(NsItem) + 255) / 256 * 256;
    for (int i = 0; i < count; i++)
        total += ns_bytes(items[i].rows, items[i].cols);
    return (size_t)total;
}

bool orthogonalize_fits(int64_t rows, int64_t cols)
{
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    return l <= kOrthoMaxLong && s <= kOrthoMaxShort;
}

hipError_t launch_orthogonalize(const OrthoEntry* items, int count, double a, double b, double c, double eps, int steps,
                                void* ws, hipStream_t s)
{
    char* const w = static_cast<char*>(ws);
    NsItem* const table = reinterpret_cast<NsItem*>(w);
    int64_t off = ((int64_t)count * sizeof(NsItem) + 255) / 256 * 256;
    // the table in the order of the classes, the widest first
    int first[4], n[4] = {0, 0, 0, 0};
    int64_t grams[3] = {0, 0, 0}, applies[3] = {0, 0, 0};
    int64_t lsq = 0, ltile = 0, lgram = 0, lsum = 0, lpoly = 0, lstep = 0;
    NsArgs args{};
    int done = 0;
    for (int cl = 3; cl >= 0; cl--) {
        first[cl] = done + args.count;
        for (int i = 0; i < count; i++) {
            const OrthoEntry& e = items[i];
            const int64_t sd = e.rows < e.cols ? e.rows : e.cols, ld = e.rows < e.cols ? e.cols : e.rows;
            if (sd == 0 || ns_class(sd) != cl)
                continue;
            NsItem it{e.g, e.out, off, (int32_t)e.rows, (int32_t)e.cols, e.scale, e.half, 0, 0, 0, 0};
            off += ns_bytes(e.rows, e.cols);
            n[cl]++;
            if (cl < 3) {
                it.slices = ns_slices(ld);
                it.block0 = (int32_t)grams[cl];
                it.apply0 = (int32_t)applies[cl];
                grams[cl] += it.slices;
                applies[cl] += (ld + 64 * kNsRun - 1) / (64 * kNsRun);
            } else {
                const NsLong p = ns_long(e.rows, e.cols);
                const int64_t T = p.sp / 64, up = T * (T + 1) / 2;
                auto most = [](int64_t& v, int64_t x) { v = v > x ? v : x; };
                most(lsq, p.sqn);
                most(ltile, T * (p.lp / 64));
                most(lgram, up * p.splits);
                most(lsum, p.splits > 1 ? up * 16 : 0);
                most(lpoly, up);
                most(lstep, T * (p.lp / 64));
            }
            args.it[args.count++] = it;
            if (args.count == kNsArg) {
                hipLaunchKernelGGL(k_ns_table, dim3(1), dim3(64), 0, s, args, table + done);
                done += kNsArg;
                args.count = 0;
            }
        }
    }
    if (args.count > 0)
        hipLaunchKernelGGL(k_ns_table, dim3(1), dim3(64), 0, s, args, table + done);
    const NsCoef k{a, b, c, eps, steps};
    if (n[2] > 0)
        hipLaunchKernelGGL(k_ns_gram<6>, dim3((unsigned)grams[2]), dim3(256), 0, s, table + first[2], n[2], w);
    if (n[1] > 0)
        hipLaunchKernelGGL(k_ns_gram<4>, dim3((unsigned)grams[1]), dim3(256), 0, s, table + first[1], n[1], w);
    if (n[0] > 0)
        hipLaunchKernelGGL(k_ns_gram<2>, dim3((unsigned)grams[0]), dim3(256), 0, s, table + first[0], n[0], w);
    if (n[2] > 0)
        hipLaunchKernelGGL((k_ns_poly<6, 8>), dim3((unsigned)n[2]), dim3(512), 0, s, table + first[2], w, k);
    if (n[1] > 0)
        hipLaunchKernelGGL((k_ns_poly<4, 4>), dim3((unsigned)n[1]), dim3(256), 0, s, table + first[1], w, k);
    if (n[0] > 0)
        hipLaunchKernelGGL((k_ns_poly<2, 4>), dim3((unsigned)n[0]), dim3(256), 0, s, table + first[0], w, k);
    if (n[2] > 0)
        hipLaunchKernelGGL(k_ns_apply<6>, dim3((unsigned)applies[2]), dim3(256), 0, s, table + first[2], n[2], w);
    if (n[1] > 0)
        hipLaunchKernelGGL(k_ns_apply<4>, dim3((unsigned)applies[1]), dim3(256), 0, s, table + first[1], n[1], w);
    if (n[0] > 0)
        hipLaunchKernelGGL(k_ns_apply<2>, dim3((unsigned)applies[0]), dim3(256), 0, s, table + first[0], n[0], w);
    if (n[3] > 0) {
        const NsItem* const t = table + first[3];
        const unsigned y = (unsigned)n[3];
        hipLaunchKernelGGL(k_nsl_sumsq, dim3((unsigned)lsq, y), dim3(256), 0, s, t, w);
        hipLaunchKernelGGL(k_nsl_init, dim3((unsigned)ltile, y), dim3(256), 0, s, t, w, eps);
        for (int st = 0; st < steps; st++) {
            hipLaunchKernelGGL(k_nsl_gram, dim3((unsigned)lgram, y), dim3(256), 0, s, t, w, st & 1);
            if (lsum > 0)
                hipLaunchKernelGGL(k_nsl_sum, dim3((unsigned)lsum, y), dim3(256), 0, s, t, w);
            hipLaunchKernelGGL(k_nsl_poly, dim3((unsigned)lpoly, y), dim3(256), 0, s, t, w, (float)b, (float)c);
            hipLaunchKernelGGL(k_nsl_step, dim3((unsigned)lstep, y), dim3(256), 0, s, t, w, (float)a, st & 1);
        }
        hipLaunchKernelGGL(k_nsl_out, dim3((unsigned)ltile, y), dim3(256), 0, s, t, w, steps & 1);
    }
    return hipGetLastError();
}

}  // namespace owq
