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
    int64_t lsq = 0, ltile = 0, lgram = 0, lsum = 0, lpoly = 0, lstep = 0;
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
                const int64_t n = p.sp / 64, upper = n * (n + 1) / 2;
                most(lsq, (int64_t)p.sqn);
                most(ltile, n * (p.lp / 64));
                most(lgram, upper * p.splits);
                most(lsum, p.splits > 1 ? upper * 16 : 0);
                most(lpoly, upper);
                most(lstep, n * (p.lp / 64));
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
        hipLaunchKernelGGL(k_nsl_init, dim3((unsigned)ltile, y), dim3(256), 0, s, table, w, eps);
        for (int st = 0; st < steps; st++) {
            hipLaunchKernelGGL(k_nsl_gram, dim3((unsigned)lgram, y), dim3(256), 0, s, table, w, st & 1);
            if (lsum > 0)
                hipLaunchKernelGGL(k_nsl_sum, dim3((unsigned)lsum, y), dim3(256), 0, s, table, w);
            hipLaunchKernelGGL(k_nsl_poly, dim3((unsigned)lpoly, y), dim3(256), 0, s, table, w, (float)b, (float)c);
            hipLaunchKernelGGL(k_nsl_step, dim3((unsigned)lstep, y), dim3(256), 0, s, table, w, (float)a, st & 1);
        }
        hipLaunchKernelGGL(k_nsl_out, dim3((unsigned)ltile, y), dim3(256), 0, s, table, w, steps & 1);
    }
    return hipGetLastError();
}

}  // namespace owq
