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
#include <cmath>

#include "owq_device.h"
#include "owq_launch.h"
#include "owq_stage.h"

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
    int32_t tiles;    // short form: 16-wide tiles of the short side (2, 4 or 6)
    int32_t slices;   // of the long side, a block of k_ns_gram each
    int32_t gram0, apply0;  // first blocks of k_ns_gram and k_ns_apply
};
static_assert(sizeof(NsItem) == 56, "table entry");

constexpr int kNsArg = 64;  // table entries per launch of k_ns_table (kernel arguments below 4 KB)
struct NsArgs {
    NsItem it[kNsArg];
    int32_t count, first;  // first: place of the first one in the table
};

// 16-element runs of the long side per wave of k_ns_apply, and elements per block
constexpr int ns_runs(int T) { return T == 2 ? 4 : 2; }
constexpr int ns_apply_len(int T) { return 4 * 16 * ns_runs(T); }

// A block per matrix: its table entry, and which matrix each block of k_ns_gram and
// k_ns_apply works on.
__global__ __launch_bounds__(256) void k_ns_table(const NsArgs a, NsItem* table, int32_t* gram_item, int32_t* apply_item)
{
    const NsItem it = a.it[blockIdx.x];
    const int at = a.first + blockIdx.x;
    if (threadIdx.x == 0)
        table[at] = it;
    if (it.tiles == 0)
        return;
    for (int b = threadIdx.x; b < it.slices; b += 256)
        gram_item[it.gram0 + b] = at;
    const int blocks = (max(it.rows, it.cols) + ns_apply_len(it.tiles) - 1) / ns_apply_len(it.tiles);
    for (int b = threadIdx.x; b < blocks; b += 256)
        apply_item[it.apply0 + b] = at;
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

constexpr int kNsDead = 0x7fffff00;  // an offset that is out of every buffer's range (zeros)

// N consecutive elements at byte offset off; those out of range are 0
template <int N, bool HALF>
__device__ __forceinline__ void ns_load(float (&v)[N], __amdgpu_buffer_rsrc_t r, int off)
{
    if (HALF) {
#pragma unroll
        for (int e = 0; e < N; e++)
            v[e] = h2f((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off + 2 * e, 0, 0));
        return;
    }
    int e = 0;
#pragma unroll
    for (; e + 4 <= N; e += 4) {
        const nf4 q = __builtin_bit_cast(nf4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * e, 0, 0));
        v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
    }
    if (N % 4) {
        typedef float nf2 __attribute__((ext_vector_type(2)));
        static_assert(N % 2 == 0, "pairs");
        const nf2 q = __builtin_bit_cast(nf2, __builtin_amdgcn_raw_buffer_load_b64(r, off + 4 * e, 0, 0));
        v[e] = q.x, v[e + 1] = q.y;
    }
}

// ------------------------------------------------------ short form: the Gram matrix --

constexpr int tri(int T) { return T * (T + 1) / 2; }

// Index of the matrix's short side that entry r of its 16 T wide Gram matrix stands for: a
// lane of k_ns_gram loads T consecutive ones of a tall matrix, one for each tile.
template <int T>
__device__ __forceinline__ int ns_short(int r, bool tall) { return tall ? (r & 15) * T + (r >> 4) : r; }

// Sums over 4 long indices per instruction, v_mfma_f64_16x16x4_f64 with the same register
// as both operands (lane l: short index l % 16 of a tile, long index l / 16). The tile
// pairs ti <= tj are dealt out to WP waves, the long side to the other 4 / WP.
template <int T, bool HALF>
__device__ __forceinline__ void ns_gram(const NsItem& it, int slice, double* part, double (*red)[256])
{
    constexpr int WP = T == 6 ? 4 : 1;                  // waves that share the pairs
    constexpr int PAIRS = (tri(T) + WP - 1) / WP;       // of one wave
    constexpr int U = T == 2 ? 8 : 4;                   // steps of 4 long indices in flight
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int SH = HALF ? 1 : 2;
    const bool tall = it.rows > it.cols;
    const int s = min(it.rows, it.cols), L = max(it.rows, it.cols);
    const int per = ((L + it.slices - 1) / it.slices + 3) & ~3;
    const int l0 = min(L, slice * per), len = min(L, l0 + per) - l0;
    const int i16 = lane & 15, kk = lane >> 4;
    f64x4 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; p++)
        acc[p] = f64x4{0.0, 0.0, 0.0, 0.0};
    const int64_t sl = tall ? it.cols : 1;  // elements from one long index to the next
    const __amdgpu_buffer_rsrc_t r = ns_rsrc(static_cast<const char*>(it.g) + ((l0 * sl) << SH),
                                             (tall ? (int64_t)len * it.cols : (int64_t)it.rows * it.cols - l0) << SH);
    auto products = [&](const float (&v)[T]) {
        double d[T];
#pragma unroll
        for (int t = 0; t < T; t++)
            d[t] = (double)v[t];
        int n = 0;
#pragma unroll
        for (int ti = 0; ti < T; ti++)
#pragma unroll
            for (int tj = ti; tj < T; tj++, n++)
                if (WP == 1 || n / PAIRS == wave)  // (uniform)
                    acc[n % PAIRS] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[ti], d[tj], acc[n % PAIRS], 0, 0, 0);
    };
    const int steps = (len + 3) >> 2;
    if (tall) {
        // T consecutive values of one row; those past the row's end belong to the next and
        // are dropped
        const int at = i16 * T < s ? (kk * it.cols + i16 * T) << SH : kNsDead;
        for (int b = (WP == 1 ? wave * U : 0); b < steps; b += (WP == 1 ? 4 : 1) * U) {
            float v[U][T];
#pragma unroll
            for (int u = 0; u < U; u++)
                ns_load<T, HALF>(v[u], r, at != kNsDead && (b + u) * 4 + kk < len ? at + (((b + u) * 4 * it.cols) << SH) : kNsDead);
#pragma unroll
            for (int u = 0; u < U; u++) {
#pragma unroll
                for (int t = 0; t < T; t++)
                    v[u][t] = i16 * T + t < s ? v[u][t] : 0.0f;
                products(v[u]);
            }
        }
    } else {
        int at[T];
#pragma unroll
        for (int t = 0; t < T; t++)
            at[t] = t * 16 + i16 < s ? (int)(((int64_t)(t * 16 + i16) * it.cols + kk) << SH) : kNsDead;
        for (int b = (WP == 1 ? wave * U : 0); b < steps; b += (WP == 1 ? 4 : 1) * U) {
            float v[U][T];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const bool in = (b + u) * 4 + kk < len;
#pragma unroll
                for (int t = 0; t < T; t++) {
                    float one[1];
                    const int off = in && at[t] != kNsDead ? at[t] + (((b + u) * 4) << SH) : kNsDead;
                    if (HALF)
                        one[0] = h2f((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
                    else
                        one[0] = __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
                    v[u][t] = one[0];
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++)
                products(v[u]);
        }
    }
    // in lane order, a tile pair after the other
    if (WP == 1) {
#pragma unroll
        for (int p = 0; p < PAIRS; p++) {
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; q++)
                red[wave][q * 64 + lane] = acc[p][q];
            __syncthreads();
            part[p * 256 + tid] = ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid];
        }
    } else {
#pragma unroll
        for (int p = 0; p < PAIRS; p++)
            if (wave * PAIRS + p < tri(T))
#pragma unroll
                for (int q = 0; q < 4; q++)
                    part[(wave * PAIRS + p) * 256 + q * 64 + lane] = acc[p][q];
    }
}

// A block sums one slice of one matrix's long side; blocks first ... of the short form's.
// NARROW: the matrices of two tiles, which need few registers and many waves in flight.
template <bool NARROW>
__global__ __launch_bounds__(256) void k_ns_gram(const NsItem* __restrict__ table, const int32_t* __restrict__ item, char* ws,
                                                 int first)
{
    __shared__ double red[4][256];
    const int block = first + (int)blockIdx.x;
    const NsItem it = table[__builtin_amdgcn_readfirstlane(item[block])];
    const int slice = block - it.gram0;
    double* part = reinterpret_cast<double*>(ws + it.off) + (int64_t)slice * tri(it.tiles) * 256;
    if (NARROW)
        it.half ? ns_gram<2, true>(it, slice, part, red) : ns_gram<2, false>(it, slice, part, red);
    else if (it.tiles == 4)
        it.half ? ns_gram<4, true>(it, slice, part, red) : ns_gram<4, false>(it, slice, part, red);
    else
        it.half ? ns_gram<6, true>(it, slice, part, red) : ns_gram<6, false>(it, slice, part, red);
}

// The slices' sums, to the first slice's place: a block per tile pair (blockIdx.x) and
// matrix (blockIdx.y).
__global__ __launch_bounds__(256) void k_ns_gram_sum(const NsItem* __restrict__ table, char* ws)
{
    const NsItem& it = table[blockIdx.y];
    const int pairs = tri(it.tiles), slices = it.slices;
    if ((int)blockIdx.x >= pairs || slices == 1)
        return;
    double* p = reinterpret_cast<double*>(ws + it.off) + (int)blockIdx.x * 256 + threadIdx.x;
    double s = 0.0;
    int sl = 0;
    for (; sl + 8 <= slices; sl += 8) {
        double v[8];
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = p[(int64_t)(sl + e) * pairs * 256];
#pragma unroll
        for (int e = 0; e < 8; e++)
            s += v[e];
    }
    for (; sl < slices; sl++)
        s += p[(int64_t)sl * pairs * 256];
    p[0] = s;
}

// ------------------------------------------------------- short form: the polynomial --

constexpr int kNsWaves = 8;

// Element q of lane l of a 16 x 16 fp64 result: row 4 q + l / 16, column l % 16
__device__ __forceinline__ int ns_drow(int q, int lane) { return 4 * q + (lane >> 4); }

template <int T>
struct NsPoly {
    static constexpr int S = 16 * T;
    static constexpr int TILES = (tri(T) + kNsWaves - 1) / kNsWaves;  // result tiles per wave
    // place of entry (r, c): rows four entries longer, so that the four rows of an operand
    // read, and the sixteen of a mirrored write, spread over the banks
    static constexpr int LD = S + 4;
    static __device__ __forceinline__ int at(int r, int c) { return r * LD + c; }
};

// X Y for symmetric matrices that commute, the upper tiles of this wave
template <int T>
__device__ __forceinline__ void ns_mul(const double* X, const double* Y, f64x4 (&acc)[NsPoly<T>::TILES],
                                       const int (&ti)[NsPoly<T>::TILES], const int (&tj)[NsPoly<T>::TILES], int lane)
{
    using P = NsPoly<T>;
    const int i16 = lane & 15, kk = lane >> 4;
    int xa[P::TILES], ya[P::TILES];
#pragma unroll
    for (int p = 0; p < P::TILES; p++) {
        acc[p] = f64x4{0.0, 0.0, 0.0, 0.0};
        xa[p] = P::at(kk, ti[p] * 16 + i16);
        ya[p] = P::at(kk, tj[p] * 16 + i16);
    }
#pragma unroll 6
    for (int k0 = 0; k0 < P::S; k0 += 4)
#pragma unroll
        for (int p = 0; p < P::TILES; p++)
            acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(X[xa[p] + k0 * P::LD], Y[ya[p] + k0 * P::LD], acc[p], 0, 0, 0);
}

template <int T>
__device__ __forceinline__ void ns_store(double* X, const f64x4 (&v)[NsPoly<T>::TILES], const int (&ti)[NsPoly<T>::TILES],
                                         const int (&tj)[NsPoly<T>::TILES], int lane)
{
#pragma unroll
    for (int p = 0; p < NsPoly<T>::TILES; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            // (below the diagonal of a tile on it: the mirror image, whose sum may round otherwise)
            const int r = ti[p] * 16 + ns_drow(q, lane), c = tj[p] * 16 + (lane & 15);
            if (r <= c) {
                X[NsPoly<T>::at(r, c)] = v[p][q];
                X[NsPoly<T>::at(c, r)] = v[p][q];
            }
        }
}

struct NsCoef {
    double a, b, c, eps;
    int32_t steps;
};

// |G|^2 is the Gram matrix's trace; then the steps, on the S x S matrices A, Q in LDS and
// the waves' result tiles. Waves past the tiles repeat the last tile (the same values to
// the same places).
template <int T>
__device__ __forceinline__ void ns_poly(const NsItem& it, char* ws, const NsCoef& k, double* A, double* Q)
{
    using PL = NsPoly<T>;
    constexpr int S = PL::S, TL = PL::TILES;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int ti[TL], tj[TL];
    f64x4 v[TL], P[TL], N[TL];
    const double* part = reinterpret_cast<const double*>(ws + it.off);
#pragma unroll
    for (int p = 0; p < TL; p++) {
        int n = min(wave * TL + p, tri(T) - 1);
#pragma unroll
        for (int q = 0; q < 4; q++)
            v[p][q] = part[n * 256 + q * 64 + lane];
        int i = 0;
        while (n >= T - i) {
            n -= T - i;
            i++;
        }
        ti[p] = i;
        tj[p] = i + n;
    }
    ns_store<T>(A, v, ti, tj, lane);
    __syncthreads();
    double tr = 0.0;
    for (int i = 0; i < S; i++)
        tr += A[PL::at(i, i)];
    const double inv = 1.0 / (sqrt(tr) + k.eps);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < TL; p++)
        v[p] = v[p] * inv * inv;
    ns_store<T>(A, v, ti, tj, lane);
    __syncthreads();
    for (int t = 0; t < k.steps; t++) {
        // v: A's tiles. N = A^2, then Q = a + b A + c A^2
        ns_mul<T>(A, A, N, ti, tj, lane);
#pragma unroll
        for (int p = 0; p < TL; p++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const bool diag = ti[p] == tj[p] && ns_drow(q, lane) == (lane & 15);
                N[p][q] = k.c * N[p][q] + k.b * v[p][q] + (diag ? k.a : 0.0);
            }
        ns_store<T>(Q, N, ti, tj, lane);
        __syncthreads();
        const bool last = t + 1 == k.steps;
        if (!last) {  // A <- (A Q) Q
            ns_mul<T>(A, Q, v, ti, tj, lane);
            __syncthreads();
            ns_store<T>(A, v, ti, tj, lane);
            __syncthreads();
            ns_mul<T>(A, Q, v, ti, tj, lane);
            __syncthreads();
        }
        if (t == 0) {
#pragma unroll
            for (int p = 0; p < TL; p++)
                P[p] = N[p];
        } else {  // P <- P Q, through A's place
            ns_store<T>(A, P, ti, tj, lane);
            __syncthreads();
            ns_mul<T>(A, Q, P, ti, tj, lane);
            __syncthreads();
        }
        if (!last) {
            ns_store<T>(A, v, ti, tj, lane);
            __syncthreads();
        }
    }
    // the matrix's factor, with the norm and the scale, over the partials
    float* out = reinterpret_cast<float*>(ws + it.off);
    const double f = inv * (double)it.scale;
    const bool tall = it.rows > it.cols;
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = ti[p] * 16 + ns_drow(q, lane), c = tj[p] * 16 + (lane & 15);
            const float x = (float)(P[p][q] * f);
            if (r <= c) {
                out[ns_short<T>(r, tall) * S + ns_short<T>(c, tall)] = x;
                out[ns_short<T>(c, tall) * S + ns_short<T>(r, tall)] = x;
            }
        }
}

// One block per matrix.
__global__ __launch_bounds__(64 * kNsWaves) void k_ns_poly(const NsItem* __restrict__ table, char* ws, const NsCoef k)
{
    __shared__ double lds[2][96 * NsPoly<6>::LD];
    const NsItem it = table[blockIdx.x];
    if (it.tiles == 2)
        ns_poly<2>(it, ws, k, lds[0], lds[1]);
    else if (it.tiles == 4)
        ns_poly<4>(it, ws, k, lds[0], lds[1]);
    else
        ns_poly<6>(it, ws, k, lds[0], lds[1]);
}

// --------------------------------------------------------- short form: the product --

// out = G F (tall) or F G (wide), F the symmetric factor: v_mfma_f32_16x16x4_f32 with F's
// rows as A and G as B; a wave holds a run of 16 of the long side in registers before it
// writes any of it, so out may be G. The contraction index 16 st + 4 (l / 16) + u is taken
// by product u of step st, so that a lane's four are consecutive in a tall matrix's row, as
// are the four results it ends with.
template <int T, bool HALF>
__device__ __forceinline__ void ns_apply(const NsItem& it, int block, const float* f, float* F)
{
    constexpr int S = 16 * T, LD = S + 4, SH = HALF ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = tid; e < S * S / 4; e += 256)
        *reinterpret_cast<nf4*>(&F[e / (S / 4) * LD + e % (S / 4) * 4]) = reinterpret_cast<const nf4*>(f)[e];
    __syncthreads();
    const bool tall = it.rows > it.cols;
    const int s = min(it.rows, it.cols), L = max(it.rows, it.cols);
    const int n16 = lane & 15, kk = lane >> 4;
    const int64_t si = tall ? 1 : it.cols, sl = tall ? it.cols : 1;
    for (int run = 0; run < ns_runs(T); run++) {
        const int lb = block * ns_apply_len(T) + (run * 4 + wave) * 16;
        if (lb >= L)
            return;
        const int len = min(16, L - lb);
        const __amdgpu_buffer_rsrc_t r = ns_rsrc(static_cast<const char*>(it.g) + ((lb * sl) << SH),
                                                 (tall ? (int64_t)len * it.cols : (int64_t)it.rows * it.cols - lb) << SH);
        float v[T][4];
#pragma unroll
        for (int st = 0; st < T; st++) {
            const int i = 16 * st + 4 * kk;
            if (tall) {
                // (values past the row's end meet F's zeros; where one of them is not
                // finite, neither is the result anywhere)
                ns_load<4, HALF>(v[st], r, i < s && n16 < len ? (n16 * it.cols + i) << SH : kNsDead);
            } else {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int off = i + u < s && n16 < len ? (int)(((int64_t)(i + u) * it.cols + n16) << SH) : kNsDead;
                    v[st][u] = HALF ? h2f((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0))
                                    : __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
                }
            }
        }
        nf4 acc[T];
#pragma unroll
        for (int t = 0; t < T; t++)
            acc[t] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < T; st++)
#pragma unroll
            for (int t = 0; t < T; t++) {
                const nf4 a = *reinterpret_cast<const nf4*>(&F[(t * 16 + n16) * LD + 16 * st + 4 * kk]);
#pragma unroll
                for (int u = 0; u < 4; u++)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[u], v[st][u], acc[t], 0, 0, 0);
            }
        if (n16 < len) {
            char* ob = static_cast<char*>(it.out) + ((lb * sl) << SH);
#pragma unroll
            for (int t = 0; t < T; t++) {
                const int i = t * 16 + 4 * kk;
                if (tall && i + 4 <= s) {
                    typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
                    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
                    const int64_t at = n16 * (int64_t)it.cols + i;
                    if (HALF)
                        *(NS_GLOBAL u2_any*)(uintptr_t)(ob + 2 * at) =
                            u2_any{f2h(acc[t][0]) | ((uint32_t)f2h(acc[t][1]) << 16), f2h(acc[t][2]) | ((uint32_t)f2h(acc[t][3]) << 16)};
                    else
                        *(NS_GLOBAL f4_any*)(uintptr_t)(ob + 4 * at) = f4_any{acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
                    continue;
                }
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (i + q < s) {
                        const int64_t at = (i + q) * si + n16 * sl;
                        if (HALF)
                            ((NS_GLOBAL uint16_t*)(uintptr_t)ob)[at] = f2h(acc[t][q]);
                        else
                            ((NS_GLOBAL float*)(uintptr_t)ob)[at] = acc[t][q];
                    }
            }
        }
    }
}

__global__ __launch_bounds__(256) void k_ns_apply(const NsItem* __restrict__ table, const int32_t* __restrict__ item,
                                                  const char* ws)
{
    __shared__ float F[96 * 100];
    const NsItem it = table[__builtin_amdgcn_readfirstlane(item[blockIdx.x])];
    const int block = (int)blockIdx.x - it.apply0;
    const float* f = reinterpret_cast<const float*>(ws + it.off);
    if (it.tiles == 2)
        it.half ? ns_apply<2, true>(it, block, f, F) : ns_apply<2, false>(it, block, f, F);
    else if (it.tiles == 4)
        it.half ? ns_apply<4, true>(it, block, f, F) : ns_apply<4, false>(it, block, f, F);
    else
        it.half ? ns_apply<6, true>(it, block, f, F) : ns_apply<6, false>(it, block, f, F);
}

// ----------------------------------------------------------------- long form --

// X, A = X X^T and B = b A + c A^2 are kept as pairs of fp16 values, a number times 2^m and
// what its rounding left: 22 bits, and 2^-25 of the scaled number absolutely, which is as
// good as fp32 here (relative error of the result 2.33e-6 against 2.29e-6 with fp32 for a
// Gaussian 300 x 1200 matrix, 5.1e-6 against 4.8e-6 with singular values down to 1e-4 of
// the largest). So each product is three on the fp16 matrix cores (high by high, high by
// low twice; low by low lies below the pairs' precision), with fp32 sums: 5 times the rate
// of the fp32 matrix instructions. m comes from a bound of the singular values after each
// step, which the caller of the kernels works out from the coefficients, so nothing
// overflows.
//
// X lies with the long side contiguous, both sides padded to 128 with zeros.
struct NsLong {
    int64_t sp, lp, tiles;
    int64_t x, x_next, A, B, parts, sq, total;  // byte offsets; high planes first, low behind
    int32_t splits, sqn;
};

constexpr int kNsTile = 128, kNsDepth = 32;  // of the products: tile, contraction per stage

__host__ __device__ inline NsLong ns_long(int64_t rows, int64_t cols)
{
    NsLong n{};
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    n.sp = (s + kNsTile - 1) / kNsTile * kNsTile;
    n.lp = (l + kNsTile - 1) / kNsTile * kNsTile;
    const int64_t t = n.sp / kNsTile;
    n.tiles = t * (t + 1) / 2;  // on and above A's diagonal
    // the long side in as many parts as give every CU a block, each of at least 8 stages
    int64_t sp = 256 / n.tiles;
    sp = sp < n.lp / (8 * kNsDepth) ? sp : n.lp / (8 * kNsDepth);
    n.splits = (int32_t)(sp < 1 ? 1 : sp);
    const int64_t sq = (rows * cols + 16383) / 16384;
    n.sqn = (int32_t)(sq < 1024 ? sq : 1024);
    int64_t off = 0;
    n.x = off, off += 4 * n.sp * n.lp;
    n.x_next = off, off += 4 * n.sp * n.lp;
    n.A = off, off += 4 * n.sp * n.sp;
    n.B = off, off += 4 * n.sp * n.sp;
    n.parts = off, off += 4 * n.splits * n.tiles * kNsTile * kNsTile;
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
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    auto add = [&](float v, int e) { s[e] = __builtin_fma((double)v, (double)v, s[e]); };
    // four consecutive elements per thread, at any element's address
    typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint16_t h4_any __attribute__((ext_vector_type(4), aligned(2)));
    const int64_t step = (int64_t)n.sqn * 256, quads = total >> 2;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < quads; q += step) {
        if (it.half) {
            const h4_any v = ((const NS_GLOBAL h4_any*)(uintptr_t)it.g)[q];
#pragma unroll
            for (int e = 0; e < 4; e++)
                add(h2f(v[e]), e);
        } else {
            const f4_any v = ((const NS_GLOBAL f4_any*)(uintptr_t)it.g)[q];
#pragma unroll
            for (int e = 0; e < 4; e++)
                add(v[e], e);
        }
    }
    if (blockIdx.x == 0 && (int)threadIdx.x < (int)(total & 3)) {
        const int64_t e = (quads << 2) + threadIdx.x;
        add(it.half ? h2f(static_cast<const uint16_t*>(it.g)[e]) : static_cast<const float*>(it.g)[e], 0);
    }
    const double sum = ns_block_sum((s[0] + s[1]) + (s[2] + s[3]), red);
    if (threadIdx.x == 0)
        reinterpret_cast<double*>(ws + it.off + n.sq)[blockIdx.x] = sum;
}

// The pair of a number that is scaled already
struct NsPair {
    uint16_t hi, lo;
};
__device__ __forceinline__ NsPair ns_pair(float v)
{
    NsPair p;
    p.hi = f2h(v);
    p.lo = f2h(v - h2f(p.hi));
    return p;
}

// X = G / (|G| + eps), padded with zeros. 64 x 64 tiles.
__global__ __launch_bounds__(256) void k_nsl_init(const NsItem* __restrict__ table, char* ws, double eps, float scale)
{
    __shared__ double red[4];
    __shared__ float tile[64][65];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int64_t tl = n.lp / 64;
    if (blockIdx.x >= (n.sp / 64) * tl)
        return;
    const bool tall = it.rows > it.cols;
    const int64_t i0 = blockIdx.x / tl * 64, l0 = blockIdx.x % tl * 64;
    const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    const int64_t row0 = (tall ? l0 : i0) + r0, col = (tall ? i0 : l0) + c, e0 = row0 * it.cols + col;
    float v[16];
    auto load = [&](auto* p) {
        const int rows = col < it.cols ? (int)min((int64_t)64, it.rows - row0) : 0;
#pragma unroll
        for (int q = 0; q < 16; q++, p += 4 * (int64_t)it.cols) {
            v[q] = 0.0f;
            if (4 * q < rows) {
                if constexpr (sizeof(*p) == 2)
                    v[q] = h2f(*p);
                else
                    v[q] = *p;
            }
        }
    };
    if (it.half)
        load(static_cast<const uint16_t*>(it.g) + e0);
    else
        load(static_cast<const float*>(it.g) + e0);
    const double* sq = reinterpret_cast<const double*>(ws + it.off + n.sq);
    double part[4];
#pragma unroll
    for (int q = 0; q < 4; q++)
        part[q] = (int)threadIdx.x + 256 * q < n.sqn ? sq[threadIdx.x + 256 * q] : 0.0;
    const double inv = 1.0 / (sqrt(ns_block_sum((part[0] + part[1]) + (part[2] + part[3]), red)) + eps);
    for (int r = r0; r < 64; r += 4)
        tile[r][c] = (float)((double)v[(r - r0) / 4] * inv) * scale;
    __syncthreads();
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + it.off + n.x);
    for (int r = r0; r < 64; r += 4) {
        const NsPair p = ns_pair(tall ? tile[c][r] : tile[r][c]);
        const int64_t at = (i0 + r) * n.lp + l0 + c;
        x[at] = p.hi;
        x[n.sp * n.lp + at] = p.lo;
    }
}

// out = scale X, X times 2^m taken back by `unscale`
__global__ __launch_bounds__(256) void k_nsl_out(const NsItem* __restrict__ table, const char* ws, int from, float unscale)
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
    const uint16_t* x = reinterpret_cast<const uint16_t*>(ws + it.off + (from ? n.x_next : n.x));
    uint16_t hi[16], lo[16];
    const int64_t at0 = (i0 + r0) * n.lp + l0 + c;
#pragma unroll
    for (int q = 0; q < 16; q++) {
        hi[q] = x[at0 + 4 * q * n.lp];
        lo[q] = x[at0 + 4 * q * n.lp + n.sp * n.lp];
    }
#pragma unroll
    for (int q = 0; q < 16; q++)
        tile[r0 + 4 * q][c] = (h2f(hi[q]) + h2f(lo[q])) * unscale * it.scale;
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

// A 128 x 128 tile of P Q^T over stages c0 .. c1 - 1 of the contraction, 8 waves of 32 (P) x
// 64 (Q), in a ring of four stages as in the integer form's product. (128 x 256 tiles, six
// stages half as deep: 112 against 119 us for X' of a 2048 x 4096 matrix, but 27 against 18
// with a short side of 221; two blocks per CU of half as deep stages: 139.) P: rows with the
// contraction contiguous (pitch p_pitch). Q: likewise, or (TURN) rows along the contraction,
// 128 columns of each, which ds_read_tr turns round. Both as high and low planes, p_low and
// q_low bytes apart. Result element r of a lane: Q's row or column l % 32 (of 32 f), P's row
// 8 (r / 4) + 4 (l / 32) + r % 4, or the other way round (TURN: four consecutive columns).
constexpr int kNsPlane = kNsTile * 64, kNsStage = 4 * kNsPlane;
typedef short ns_s4 __attribute__((ext_vector_type(4)));

template <bool TURN>
__device__ __forceinline__ void ns_product(const char* p, int64_t p_pitch, int64_t p_low, const char* q, int64_t q_pitch,
                                           int64_t q_low, int c0, int c1, char* s0, char* s1, char* s2, char* s3,
                                           nf16 (&acc)[2])
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave & 3, wq = wave >> 2;
    const int l32 = lane & 31, h = lane >> 5;
    // a wave loads half a plane: planes P high, P low, Q high, Q low
    const int plane = wave >> 1;
    const bool turned = TURN && plane >= 2;
    const int64_t pitch = plane < 2 ? p_pitch : q_pitch;
    const char* const from = (plane < 2 ? p + (plane & 1) * p_low : q + (plane & 1) * q_low);
    int src[4];
#pragma unroll
    for (int t = 0; t < 4; t++) {
        const int u = (wave & 1) * 256 + t * 64 + lane;
        // turned: row u / 16 of the stage; piece c of it in slot c ^ 4 (row % 4), so that the
        // 64 bytes that a read takes of each of four rows lie in different banks
        src[t] = turned ? (u >> 4) * (int)pitch + ((u & 15) ^ (((u >> 4) & 3) << 2)) * 16
                        : stage_row(u) * (int)pitch + stage_piece(u) * 16;
    }
    const __amdgpu_buffer_rsrc_t whole =
        uniform_rsrc(from, turned ? (int64_t)c1 * kNsDepth * pitch : (int64_t)kNsTile * pitch);
    auto dma = [&](int c, char* stage) {
        const int dead = c < c1 ? 0 : kDeadLoad, cc = min(c, c1 - 1);
        // (turned: the rows may reach far, so the descriptor moves)
        const __amdgpu_buffer_rsrc_t r =
            turned ? uniform_rsrc(from + (int64_t)cc * kNsDepth * pitch, (int64_t)kNsDepth * pitch) : whole;
        const int o = turned ? 0 : cc * 64;
#pragma unroll
        for (int t = 0; t < 4; t++)
            dma16_lds(r, stage + plane * kNsPlane + ((wave & 1) * 4 + t) * 1024, (src[t] + o) | dead);
    };
    // operand reads of 16-deep step st: P's 32 rows, Q's two times 32
    const int pa[2] = {wp * 2048 + stage_at(l32, h), wp * 2048 + stage_at(l32, 2 + h)};
    int qa[2][2];
#pragma unroll
    for (int st = 0; st < 2; st++)
#pragma unroll
        for (int f = 0; f < 2; f++) {
            if (TURN) {
                // in a group of 16 lanes, lane i names 4 columns of row i / 4 and gets
                // column i of the 4 rows; the rows 4 further on by a second read
                const int row = 16 * st + 8 * h + ((lane & 15) >> 2);
                const int col = wq * 64 + 32 * f + 16 * ((lane >> 4) & 1) + (lane & 3) * 4;
                qa[st][f] = 2 * kNsPlane + row * 256 + (((col >> 3) ^ ((row & 3) << 2)) * 16) + (col & 4) * 2;
            } else
                qa[st][f] = 2 * kNsPlane + (wq * 2 + f) * 2048 + stage_at(l32, 2 * st + h);
        }
    half8_t pv[2][2], qv[2][2][2];  // [set][high, low], [set][high, low][f]
    auto read = [&](const char* stage, int st) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
            pv[st][e] = *reinterpret_cast<const half8_t*>(stage + e * kNsPlane + pa[st]);
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const char* at = stage + e * kNsPlane + qa[st][f];
                if (TURN) {
                    const ns_s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) ns_s4*)at);
                    const ns_s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) ns_s4*)(at + 4 * 256));
                    qv[st][e][f] = __builtin_bit_cast(half8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
                } else
                    qv[st][e][f] = *reinterpret_cast<const half8_t*>(at);
            }
        }
    };
    auto mul = [&](int st) {
#pragma unroll
        for (int e = 0; e < 3; e++)  // high high, high low, low high
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const half8_t a = pv[st][e == 2 ? 1 : 0], b = qv[st][e == 1 ? 1 : 0][f];
                acc[f] = TURN ? __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, acc[f], 0, 0, 0)
                              : __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc[f], 0, 0, 0);
            }
#pragma unroll
        for (int e = 0; e < 6; e++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
    };
    auto step = [&](int c, const char* cur, const char* next, char* fill) {
        stage_barrier<4, 15>();
        dma(c + 3, fill);
        if (c < c1) {
            read(cur, 1);
            mul(0);
            read(next, 0);
            mul(1);
            // the reads of cur are done before this wave lets it be overwritten
#pragma unroll
            for (int e = 0; e < 2; e++)
                asm volatile("" ::"v"(pv[1][e]), "v"(qv[1][e][0]), "v"(qv[1][e][1]));
        }
    };
    dma(c0, s0);
    dma(c0 + 1, s1);
    dma(c0 + 2, s2);
    stage_barrier<8>();
    read(s0, 0);
    for (int c = c0; c < c1; c += 4) {
        step(c, s0, s1, s3);
        step(c + 1, s1, s2, s0);
        step(c + 2, s2, s3, s1);
        step(c + 3, s3, s0, s2);
    }
#pragma unroll
    for (int e = 0; e < 2; e++)
        asm volatile("" ::"v"(pv[0][e]), "v"(qv[0][e][0]), "v"(qv[0][e][1]));
    stage_barrier<0>();  // the loads past the end have written their zeros
}

#define NS_STAGES                                                        \
    __shared__ __attribute__((aligned(1024))) char s0[kNsStage];         \
    __shared__ __attribute__((aligned(1024))) char s1[kNsStage];         \
    __shared__ __attribute__((aligned(1024))) char s2[kNsStage];         \
    __shared__ __attribute__((aligned(1024))) char s3[kNsStage];         \
    nf16 acc[2];                                                         \
    for (int f = 0; f < 2; f++)                                          \
        for (int r = 0; r < 16; r++)                                     \
            acc[f][r] = 0.0f

__device__ __forceinline__ void ns_upper(int n, int T, int& ti, int& tj)
{
    int i = 0;
    while (n >= T - i) {
        n -= T - i;
        i++;
    }
    ti = i;
    tj = i + n;
}

// A = X X^T: tiles on and above the diagonal, `splits` parts of the long side each, in lane order
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_gram(const NsItem* __restrict__ table,
                                                                                             char* ws, int from)
{
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    if (blockIdx.x >= n.tiles * n.splits)
        return;
    int ti, tj;
    ns_upper((int)blockIdx.x / n.splits, (int)(n.sp / kNsTile), ti, tj);
    const int sl = (int)blockIdx.x % n.splits, all = (int)(n.lp / kNsDepth);
    const char* x = ws + it.off + (from ? n.x_next : n.x);
    const int64_t pitch = 2 * n.lp, low = 2 * n.sp * n.lp;
    ns_product<false>(x + ti * kNsTile * pitch, pitch, low, x + tj * kNsTile * pitch, pitch, low, (int)((int64_t)all * sl / n.splits),
                      (int)((int64_t)all * (sl + 1) / n.splits), s0, s1, s2, s3, acc);
    nf4* part = reinterpret_cast<nf4*>(ws + it.off + n.parts) + (int64_t)blockIdx.x * (kNsTile * kNsTile / 4) +
                (threadIdx.x >> 6) * 512 + (threadIdx.x & 63);
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int e = 0; e < 4; e++)
            part[(f * 4 + e) * 64] = nf4{acc[f][4 * e], acc[f][4 * e + 1], acc[f][4 * e + 2], acc[f][4 * e + 3]};
}

// Four numbers of a symmetric matrix, rows i .. i + 3 of column j, to both their places
__device__ __forceinline__ void ns_put(uint16_t* m, int64_t pitch, int64_t low, int i, int j, nf4 v)
{
    NsPair p[4];
#pragma unroll
    for (int e = 0; e < 4; e++)
        p[e] = ns_pair(v[e]);
    if (i + 3 <= j) {
        *reinterpret_cast<uint2*>(m + j * pitch + i) = make_uint2(p[0].hi | ((uint32_t)p[1].hi << 16), p[2].hi | ((uint32_t)p[3].hi << 16));
        *reinterpret_cast<uint2*>(m + low + j * pitch + i) =
            make_uint2(p[0].lo | ((uint32_t)p[1].lo << 16), p[2].lo | ((uint32_t)p[3].lo << 16));
#pragma unroll
        for (int e = 0; e < 4; e++) {
            m[(i + e) * pitch + j] = p[e].hi;
            m[low + (i + e) * pitch + j] = p[e].lo;
        }
    } else if (i <= j) {  // the diagonal runs through the four
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (i + e <= j) {
                m[(i + e) * pitch + j] = m[j * pitch + i + e] = p[e].hi;
                m[low + (i + e) * pitch + j] = m[low + j * pitch + i + e] = p[e].lo;
            }
    }
}

// The four numbers of two words of a high and of a low plane
__device__ __forceinline__ nf4 ns_join(uint2 hi, uint2 lo)
{
    const uint32_t ph[2] = {hi.x, hi.y}, pl[2] = {lo.x, lo.y};
    nf4 v;
#pragma unroll
    for (int k = 0; k < 4; k++)
        v[k] = h2f((uint16_t)(ph[k >> 1] >> (16 * (k & 1)))) + h2f((uint16_t)(pl[k >> 1] >> (16 * (k & 1))));
    return v;
}

// The parts' sums: a wave per 32 x 32 piece's quarter. scale: 2^(m of A - 2 m of X)
__global__ __launch_bounds__(256) void k_nsl_sum(const NsItem* __restrict__ table, char* ws, float scale)
{
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int tile = (int)blockIdx.x >> 4;
    if (tile >= n.tiles)
        return;
    int ti, tj;
    ns_upper(tile, (int)(n.sp / kNsTile), ti, tj);
    const int at = ((int)blockIdx.x & 15) * 256 + threadIdx.x;  // vector of four of the tile
    const nf4* p = reinterpret_cast<const nf4*>(ws + it.off + n.parts) + (int64_t)tile * n.splits * (kNsTile * kNsTile / 4) + at;
    nf4 s = p[0];
    int sl = 1;
    for (; sl + 4 <= n.splits; sl += 4) {
        nf4 v[4];
#pragma unroll
        for (int e = 0; e < 4; e++)
            v[e] = p[(int64_t)(sl + e) * (kNsTile * kNsTile / 4)];
#pragma unroll
        for (int e = 0; e < 4; e++)
            s += v[e];
    }
    for (; sl < n.splits; sl++)
        s += p[(int64_t)sl * (kNsTile * kNsTile / 4)];
    const int wave = at >> 9, f = (at >> 8) & 1, e = (at >> 6) & 3, lane = at & 63;
    ns_put(reinterpret_cast<uint16_t*>(ws + it.off + n.A), n.sp, n.sp * n.sp, ti * kNsTile + (wave & 3) * 32 + 8 * e + 4 * (lane >> 5),
           tj * kNsTile + (wave >> 2) * 64 + 32 * f + (lane & 31), s * scale);
}

// B = b A + c A^2; b and c with the powers of two of A and B
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_poly(const NsItem* __restrict__ table,
                                                                                             char* ws, float b, float c)
{
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    if (blockIdx.x >= n.tiles)
        return;
    int ti, tj;
    ns_upper((int)blockIdx.x, (int)(n.sp / kNsTile), ti, tj);
    const char* A = ws + it.off + n.A;
    const int64_t pitch = 2 * n.sp, low = 2 * n.sp * n.sp;
    ns_product<false>(A + ti * kNsTile * pitch, pitch, low, A + tj * kNsTile * pitch, pitch, low, 0, (int)(n.sp / kNsDepth), s0, s1,
                      s2, s3, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t* a = reinterpret_cast<const uint16_t*>(A);
    const int i0 = ti * kNsTile + (wave & 3) * 32 + 4 * (lane >> 5), j0 = tj * kNsTile + (wave >> 2) * 64 + (lane & 31);
    uint2 hi[8], lo[8];  // all loads before the first store
#pragma unroll
    for (int q = 0; q < 8; q++) {
        const uint16_t* at = a + (j0 + 32 * (q >> 2)) * n.sp + i0 + 8 * (q & 3);
        hi[q] = *reinterpret_cast<const uint2*>(at);
        lo[q] = *reinterpret_cast<const uint2*>(at + n.sp * n.sp);
    }
#pragma unroll
    for (int q = 0; q < 8; q++) {
        const nf4 x = ns_join(hi[q], lo[q]);
        nf4 v;
#pragma unroll
        for (int k = 0; k < 4; k++)
            v[k] = __builtin_fmaf(c, acc[q >> 2][4 * (q & 3) + k], b * x[k]);
        ns_put(reinterpret_cast<uint16_t*>(ws + it.off + n.B), n.sp, n.sp * n.sp, i0 + 8 * (q & 3), j0 + 32 * (q >> 2), v);
    }
}

// X' = a X + B X; a and the product with the powers of two of X, B and X'
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_step(const NsItem* __restrict__ table,
                                                                                             char* ws, float a, float scale, int from)
{
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols);
    const int T = (int)(n.sp / kNsTile);
    if (blockIdx.x >= T * (n.lp / kNsTile))
        return;
    const int place = xcd_place((int)blockIdx.x, (int)(T * (n.lp / kNsTile)));
    const int ti = place % T;
    const int64_t l0 = (int64_t)(place / T) * kNsTile;
    const char* x = ws + it.off + (from ? n.x_next : n.x);
    const char* B = ws + it.off + n.B;
    const int64_t low = n.sp * n.lp;
    ns_product<true>(B + ti * kNsTile * (2 * n.sp), 2 * n.sp, 2 * n.sp * n.sp, x + 2 * l0, 2 * n.lp, 2 * low, 0, (int)(n.sp / kNsDepth),
                     s0, s1, s2, s3, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t* xo = reinterpret_cast<const uint16_t*>(x);
    uint16_t* y = reinterpret_cast<uint16_t*>(ws + it.off + (from ? n.x : n.x_next));
    const int64_t at0 = (ti * kNsTile + (wave & 3) * 32 + (lane & 31)) * n.lp + l0 + (wave >> 2) * 64 + 4 * (lane >> 5);
    uint2 hi[8], lo[8];  // all loads before the first store
#pragma unroll
    for (int q = 0; q < 8; q++) {
        hi[q] = *reinterpret_cast<const uint2*>(xo + at0 + 8 * q);
        lo[q] = *reinterpret_cast<const uint2*>(xo + low + at0 + 8 * q);
    }
#pragma unroll
    for (int q = 0; q < 8; q++) {
        const nf4 v = ns_join(hi[q], lo[q]);
        NsPair p[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            p[k] = ns_pair(__builtin_fmaf(a, v[k], acc[q >> 2][4 * (q & 3) + k] * scale));
        *reinterpret_cast<uint2*>(y + at0 + 8 * q) = make_uint2(p[0].hi | ((uint32_t)p[1].hi << 16), p[2].hi | ((uint32_t)p[3].hi << 16));
        *reinterpret_cast<uint2*>(y + low + at0 + 8 * q) = make_uint2(p[0].lo | ((uint32_t)p[1].lo << 16), p[2].lo | ((uint32_t)p[3].lo << 16));
    }
}

// Powers of two that bring numbers of at most `bound` below 2^14, as exponents
int ns_exponent(double bound)
{
    int e = 0;
    std::frexp(bound > 1e-30 ? (bound < 1e30 ? bound : 1e30) : 1e-30, &e);  // bound <= 2^e
    return 14 - e;
}

// Bounds of what a step holds: the elements of A and of B (no element of a symmetric matrix
// passes its largest |eigenvalue|) and the singular values that it leaves, from those it
// finds (at most x) and its polynomial on a grid over [0, x]. 1e-3 is for what lies between
// the grid's points and for roundings; much more would grow from step to step where the
// polynomial leaves its range (with 3.4445, -4.775, 2.0315, 1.2025 maps into itself and 1.27
// does not). Above 2^14 the pairs have a factor of 4 left.
struct NsBound {
    double a, b, next;
};
NsBound ns_bound(double x, double a, double b, double c)
{
    NsBound n{x * x, 0.0, 0.0};
    for (int i = 0; i <= 1024; i++) {
        const double v = x * i / 1024.0, l = v * v;
        n.b = std::fmax(n.b, std::fabs(b * l + c * l * l));
        n.next = std::fmax(n.next, std::fabs(v * (a + b * l + c * l * l)));
    }
    n.b *= 1.001;
    n.next *= 1.001;
    return n;
}

// ------------------------------------------------------------------ the plan --

constexpr int kNsShort = 96;  // short sides of the short form
int ns_tiles(int64_t s) { return s > kNsShort ? 0 : (s > 64 ? 6 : (s > 32 ? 4 : 2)); }

// slices of the long side in the short form: at least 256 long (128 for wide Gram
// matrices, whose products take longer), at most 128
int ns_slices(int64_t l, int T)
{
    const int64_t len = T == 2 ? 256 : 128, n = (l + len - 1) / len;
    return (int)(n < 128 ? n : 128);
}

int64_t ns_bytes(int64_t rows, int64_t cols)
{
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    if (s == 0)
        return 0;
    const int T = ns_tiles(s);
    if (T == 0)
        return ns_long(rows, cols).total;
    const int64_t part = (int64_t)ns_slices(l, T) * tri(T) * 2048, f = 4LL * 256 * T * T;
    return ((part > f ? part : f) + 255) / 256 * 256;
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Blocks of k_ns_gram and k_ns_apply of one matrix
int64_t ns_gram_blocks(int64_t s, int64_t l) { return s > 0 && ns_tiles(s) ? ns_slices(l, ns_tiles(s)) : 0; }
int64_t ns_apply_blocks(int64_t s, int64_t l)
{
    const int T = ns_tiles(s);
    return s > 0 && T ? (l + ns_apply_len(T) - 1) / ns_apply_len(T) : 0;
}

}  // namespace

size_t orthogonalize_workspace_bytes(const OrthoEntry* items, int count)
{
    int64_t total = up256((int64_t)count * sizeof(NsItem)), grams = 0, applies = 0;
    for (int i = 0; i < count; i++) {
        const int64_t s = items[i].rows < items[i].cols ? items[i].rows : items[i].cols, l = items[i].rows + items[i].cols - s;
        total += ns_bytes(items[i].rows, items[i].cols);
        grams += ns_gram_blocks(s, l);
        applies += ns_apply_blocks(s, l);
    }
    return (size_t)(total + up256(4 * grams) + up256(4 * applies));
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
    int64_t grams = 0, applies = 0;
    for (int i = 0; i < count; i++) {
        const int64_t sd = items[i].rows < items[i].cols ? items[i].rows : items[i].cols, ld = items[i].rows + items[i].cols - sd;
        grams += ns_gram_blocks(sd, ld);
        applies += ns_apply_blocks(sd, ld);
    }
    int64_t off = up256((int64_t)count * sizeof(NsItem));
    int32_t* const gram_item = reinterpret_cast<int32_t*>(w + off);
    off += up256(4 * grams);
    int32_t* const apply_item = reinterpret_cast<int32_t*>(w + off);
    off += up256(4 * applies);
    // the table: the long form, then the short one, the widest first (they take longest)
    grams = applies = 0;
    int longs = 0, shorts = 0;
    unsigned pairs = 0;
    int64_t lsq = 0, ltile = 0, lgram = 0, lpoly = 0, lstep = 0;
    auto most = [](auto& v, auto x) { v = v > x ? v : x; };
    NsArgs args{};
    auto flush = [&] {
        if (args.count > 0)
            hipLaunchKernelGGL(k_ns_table, dim3((unsigned)args.count), dim3(256), 0, s, args, table, gram_item, apply_item);
        args.first += args.count;
        args.count = 0;
    };
    int64_t wide = 0;  // blocks of k_ns_gram for more than two tiles
    for (const int T : {0, 6, 4, 2}) {
        if (T == 2)
            wide = grams;
        for (int i = 0; i < count; i++) {
            const OrthoEntry& e = items[i];
            const int64_t sd = e.rows < e.cols ? e.rows : e.cols, ld = e.rows + e.cols - sd;
            if (sd == 0 || ns_tiles(sd) != T)
                continue;
            NsItem it{e.g, e.out, off, (int32_t)e.rows, (int32_t)e.cols, e.scale, e.half, T, 0, (int32_t)grams, (int32_t)applies};
            off += ns_bytes(e.rows, e.cols);
            if (T > 0) {
                it.slices = ns_slices(ld, T);
                grams += ns_gram_blocks(sd, ld);
                applies += ns_apply_blocks(sd, ld);
                most(pairs, (unsigned)tri(T));
                shorts++;
            } else {
                const NsLong p = ns_long(e.rows, e.cols);
                most(lsq, (int64_t)p.sqn);
                most(ltile, (p.sp / 64) * (p.lp / 64));
                most(lgram, p.tiles * p.splits);
                most(lpoly, p.tiles);
                most(lstep, (p.sp / kNsTile) * (p.lp / kNsTile));
                longs++;
            }
            args.it[args.count++] = it;
            if (args.count == kNsArg)
                flush();
        }
    }
    flush();
    if (shorts > 0) {
        const NsItem* const t = table + longs;
        if (wide > 0)
            hipLaunchKernelGGL(k_ns_gram<false>, dim3((unsigned)wide), dim3(256), 0, s, table, gram_item, w, 0);
        if (grams > wide)
            hipLaunchKernelGGL(k_ns_gram<true>, dim3((unsigned)(grams - wide)), dim3(256), 0, s, table, gram_item, w, (int)wide);
        hipLaunchKernelGGL(k_ns_gram_sum, dim3(pairs, (unsigned)shorts), dim3(256), 0, s, t, w);
        hipLaunchKernelGGL(k_ns_poly, dim3((unsigned)shorts), dim3(64 * kNsWaves), 0, s, t, w, NsCoef{a, b, c, eps, steps});
        hipLaunchKernelGGL(k_ns_apply, dim3((unsigned)applies), dim3(256), 0, s, table, apply_item, w);
    }
    if (longs > 0) {
        const unsigned y = (unsigned)longs;
        hipLaunchKernelGGL(k_nsl_sumsq, dim3((unsigned)lsq, y), dim3(256), 0, s, table, w);
        auto two = [](int e) { return (float)std::ldexp(1.0, e); };
        double bound = 1.0;
        int mx = ns_exponent(bound);
        hipLaunchKernelGGL(k_nsl_init, dim3((unsigned)ltile, y), dim3(256), 0, s, table, w, eps, two(mx));
        for (int st = 0; st < steps; st++) {
            const NsBound n = ns_bound(bound, a, b, c);
            const int ma = ns_exponent(n.a), mb = ns_exponent(n.b);
            bound = n.next;
            const int next = ns_exponent(bound);
            hipLaunchKernelGGL(k_nsl_gram, dim3((unsigned)lgram, y), dim3(512), 0, s, table, w, st & 1);
            hipLaunchKernelGGL(k_nsl_sum, dim3((unsigned)(16 * lpoly), y), dim3(256), 0, s, table, w, two(ma - 2 * mx));
            hipLaunchKernelGGL(k_nsl_poly, dim3((unsigned)lpoly, y), dim3(512), 0, s, table, w, (float)(b * two(mb - ma)),
                               (float)(c * two(mb - 2 * ma)));
            hipLaunchKernelGGL(k_nsl_step, dim3((unsigned)lstep, y), dim3(512), 0, s, table, w, (float)(a * two(next - mx)),
                               two(next - mb - mx), st & 1);
            mx = next;
        }
        hipLaunchKernelGGL(k_nsl_out, dim3((unsigned)ltile, y), dim3(256), 0, s, table, w, steps & 1, two(-mx));
    }
    return hipGetLastError();
}

}  // namespace owq
