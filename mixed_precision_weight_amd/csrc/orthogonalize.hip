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
// up to a^steps: the first is summed in fp64, the second runs on 40-bit fixed point (in fp32
// a direction at 1e-3 of the largest would come out 1 % off), or on fp64 where the steps lift
// so far that 40 bits are not enough (ns_fixed). Longer short sides run the steps as they
// stand, on pairs of fp16.
#include <cmath>

#include "owq_device.h"
#include "owq_launch.h"
#include "owq_stage.h"

namespace owq {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float nf4 __attribute__((ext_vector_type(4)));
typedef int ns_i4 __attribute__((ext_vector_type(4)));
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
    int32_t slices;   // of the long side, a block of k_ns_gram each (long form: parts, a block each per tile)
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
// k_ns_apply works on. The entries come as kernel arguments, so a captured call keeps its own
// and no copy from the host is recorded; 4.6 us per 64 matrices.
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
// Narrow ones are bound by memory and the fp64 matrix cores (busy 61 %): 192 matrices of 32
// columns, 157 MB in 44 us (3.6 TB/s, and 30 MB of partial sums). Wide ones by the matrix
// cores and the loads before them: 32 matrices 4096 x 86, 45 us, where the products alone
// take 20.
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
// matrix (blockIdx.y). 224 matrices: 15 us, 75 MB at 5 TB/s; a few: one latency, 4.6 us.
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

// The polynomial works on numbers of 40 bits in fixed point: x = u I with |I| <= 2^38 and a
// power of two u per matrix, found from its largest entry, and I in five digits base 256
// from -128 to 127. A product of two matrices is then 19 products of digit matrices on the
// 8-bit matrix cores, whose sums are exact: digits i and j of place i + j <= 5. What is left
// out lies below 2^-40 of the product of the largest entries, and rounding to 40 bits is
// 2^-39 of the largest entry. Such an error grows by up to a^2 = 12 per step along directions
// far below the largest: some 1e-7 of the result after five steps; ns_fixed says how far that
// goes. (Without place 5, 15
// products and 2^-35, a direction at 1e-4 of the largest came out 4 % off; fp32 products,
// 2^-24, do that at 1e-3; fp64 matrix instructions take 102 us against 60 for a short side
// of 86. One matrix is one CU's work, so a card full of matrices does not help.)
template <int T>
struct NsPoly {
    static constexpr int S = 16 * T;
    static constexpr int TILES = (tri(T) + kNsWaves - 1) / kNsWaves;  // result tiles per wave
    static constexpr int WAVES = T == 6 ? 8 : T == 4 ? 5 : 3;         // waves with tiles
    static constexpr int KS = S > 64 ? 2 : 1;                         // 64-deep products
    // digit matrices in LDS: rows of S bytes, 16 apart, so that 16 rows' pieces of 16 bytes
    // fall on all 64 banks
    static constexpr int PITCH = S + 16, PLANE = S * PITCH, MATRIX = 5 * PLANE;
};
constexpr int kNsLds = 3 * NsPoly<6>::MATRIX + 64;  // (the last rows' reads reach 16 bytes further)

// The tiles of a wave: of tile row `ctr`, columns `par`; a symmetric matrix's tile (i, j) is
// any wave's that has i and j. Nibbles by wave.
template <int T>
__device__ __forceinline__ void ns_tiles_of(int wave, int& ctr, int (&par)[NsPoly<T>::TILES])
{
    auto nibble = [&](uint32_t v) { return (int)((v >> (4 * wave)) & 15); };
    if constexpr (T == 6) {
        ctr = nibble(0x42354100);
        par[0] = nibble(0x52354130);
        par[1] = nibble(0x53411241);
        par[2] = nibble(0x53522352);
    } else if constexpr (T == 4) {
        ctr = nibble(0x23100);
        par[0] = nibble(0x23120);
        par[1] = nibble(0x31231);
    } else {
        ctr = nibble(0x100);
        par[0] = nibble(0x110);
    }
}

// unit X Y for symmetric matrices that commute, this wave's tiles: element q of lane l is row
// 4 (l / 16) + q of tile row ctr, column l % 16 of tile column par[p]
template <int T>
__device__ __forceinline__ void ns_mul(const char* X, const char* Y, double unit, f64x4 (&v)[NsPoly<T>::TILES], int ctr,
                                       const int (&par)[NsPoly<T>::TILES], int lane)
{
    using P = NsPoly<T>;
    const int at = (lane & 15) * P::PITCH + (lane >> 4) * 16;
    ns_i4 x[P::KS][5];
#pragma unroll
    for (int ks = 0; ks < P::KS; ks++)
#pragma unroll
        for (int i = 0; i < 5; i++) {
            x[ks][i] = *reinterpret_cast<const ns_i4*>(X + i * P::PLANE + ctr * 16 * P::PITCH + at + ks * 64);
            // past the matrix's columns: zeros (whatever Y's bytes are there)
            if (P::S - ks * 64 < 64 && lane >= 32)
                x[ks][i] = ns_i4{0, 0, 0, 0};
        }
#pragma unroll
    for (int p = 0; p < P::TILES; p++) {
        ns_i4 d[6] = {};
#pragma unroll
        for (int ks = 0; ks < P::KS; ks++) {
            ns_i4 y[5];
#pragma unroll
            for (int j = 0; j < 5; j++)
                y[j] = *reinterpret_cast<const ns_i4*>(Y + j * P::PLANE + par[p] * 16 * P::PITCH + at + ks * 64);
#pragma unroll
            for (int i = 0; i < 5; i++)
#pragma unroll
                for (int j = 0; j < 5 && i + j < 6; j++)
                    d[i + j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[ks][i], y[j], d[i + j], 0, 0, 0);
        }
        // |d[n]| <= 5 * 96 * 2^14, so two places fit 32 bits together
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const double hi = (double)(d[0][q] * 256 + d[1][q]), mid = (double)(d[2][q] * 256 + d[3][q]), lo = (double)(d[4][q] * 256 + d[5][q]);
            v[p][q] = unit * __builtin_fma(hi, 0x1p56, __builtin_fma(mid, 0x1p40, lo * 0x1p24));
        }
    }
}

// The scale of a matrix: E (biased exponent) with every entry below 2^(E - 1022)
__device__ __forceinline__ double ns_two(int biased)
{
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)biased << 52);
}
__device__ __forceinline__ double ns_up(int E) { return ns_two(2083 - E); }    // 2^38 over it
__device__ __forceinline__ double ns_unit(int E) { return ns_two(E - 37); }    // and back

// Largest of the wave's entries, as the upper half of a double in a float's bits (their order
// is the same); infinite where one is not finite or leaves the range
template <int TL>
__device__ __forceinline__ float ns_top(const f64x4 (&v)[TL])
{
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const double x = v[p][q];  // (the cast of a vector's element itself reads element 0)
            const uint32_t h = (uint32_t)(__builtin_bit_cast(uint64_t, x) >> 32) & 0x7fffffffu;
            m = h > m ? h : m;
        }
    return wave_max_dpp(__builtin_bit_cast(float, m < 0x7f000000u ? m : 0x7f800000u));
}
// over the waves; bad: not finite
template <int WAVES>
__device__ __forceinline__ int ns_exponent_of(const float* red, bool& bad)
{
    float m = red[0];
#pragma unroll
    for (int w = 1; w < WAVES; w++)
        m = fmaxf(m, red[w]);
    const uint32_t b = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, m));
    bad = bad || b >= 0x7f000000u;
    const int E = (int)(b >> 20);
    return E < 64 ? 64 : E > 0x7f0 ? 0x7f0 : E;
}

// The digits of this wave's tiles to X, up = 2^38 over their bound. A byte of the low 40 bits
// of I + 0x8080808080 is a digit + 128; the sum is in the constant that rounds to integers.
template <int T>
__device__ __forceinline__ void ns_store(char* X, const f64x4 (&v)[NsPoly<T>::TILES], double up, int ctr,
                                         const int (&par)[NsPoly<T>::TILES], int lane)
{
    using P = NsPoly<T>;
    const double magic = __builtin_bit_cast(double, (uint64_t)0x4338008080808080ull);
    const uint32_t one = lane & 1 ? 0x03070105u : 0x06020400u, two = lane & 2 ? 0x03020706u : 0x05040100u;
#pragma unroll
    for (int p = 0; p < P::TILES; p++) {
        uint32_t lo[4], hi[4], d[5];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint64_t t = __builtin_bit_cast(uint64_t, __builtin_fma(v[p][q], up, magic));
            lo[q] = (uint32_t)t;
            hi[q] = (uint32_t)(t >> 32);
        }
        // d[i]: digit i of the lane's four rows
        const uint32_t a01 = __builtin_amdgcn_perm(lo[1], lo[0], 0x05010400u), b01 = __builtin_amdgcn_perm(lo[1], lo[0], 0x07030602u);
        const uint32_t a23 = __builtin_amdgcn_perm(lo[3], lo[2], 0x05010400u), b23 = __builtin_amdgcn_perm(lo[3], lo[2], 0x07030602u);
        d[4] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
        d[3] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
        d[2] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
        d[1] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
        d[0] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(hi[3], hi[2], 0x0c0c0400u), __builtin_amdgcn_perm(hi[1], hi[0], 0x0c0c0400u),
                                     0x05040100u);
        char* const down = X + (par[p] * 16 + (lane & 15)) * P::PITCH + ctr * 16 + (lane >> 4) * 4;
        char* const across = X + (ctr * 16 + (lane >> 4) * 4 + (lane & 3)) * P::PITCH + par[p] * 16 + (lane & 12);
#pragma unroll
        for (int i = 0; i < 5; i++) {
            d[i] ^= 0x80808080u;
            *reinterpret_cast<uint32_t*>(down + i * P::PLANE) = d[i];
        }
        if (par[p] != ctr) {
            // four lanes' columns turned into rows: bytes exchanged with lane ^ 1, then ^ 2
#pragma unroll
            for (int i = 0; i < 5; i++) {
                const uint32_t e = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)d[i], 0xb1, 0xf, 0xf, false);
                const uint32_t w = __builtin_amdgcn_perm(e, d[i], one);
                const uint32_t f = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x4e, 0xf, 0xf, false);
                *reinterpret_cast<uint32_t*>(across + i * P::PLANE) = __builtin_amdgcn_perm(f, w, two);
            }
        }
    }
}

struct NsCoef {
    double a, b, c, eps;
    int32_t steps;
};

// |G| + eps = m 2^e, m in [1/2, 1): 1 / m, and e. So numbers stay in range whatever |G| and eps
// are: G enters the product times 2^-e, the Gram matrix here times 2^-2e, and a matrix of
// zeros stays one.
struct NsNorm {
    double inv;
    int e;
};
__device__ __forceinline__ NsNorm ns_norm(double trace, double eps)
{
    const double n = sqrt(trace) + eps;
    return NsNorm{1.0 / __builtin_amdgcn_frexp_mant(n), __builtin_amdgcn_frexp_exp(n)};
}

// out = 2^(p + es) (P 2^-p / m ms) (G 2^-e), with scale = ms 2^es and every entry of P below 2^p:
// what an entry of P becomes, and, behind the factor, the exponents for G and for out.
struct NsFactor {
    double f;
    int p;
};
template <int S>
__device__ __forceinline__ NsFactor ns_factor(const NsItem& it, const NsNorm& n, int p, bool bad, float* out)
{
    if (threadIdx.x == 0) {
        reinterpret_cast<int*>(out)[S * S] = -n.e;
        reinterpret_cast<int*>(out)[S * S + 1] = p + __builtin_amdgcn_frexp_expf(it.scale);
    }
    return NsFactor{bad ? __builtin_nan("") : n.inv * (double)__builtin_amdgcn_frexp_mantf(it.scale), p};
}
__device__ __forceinline__ float ns_entry(const NsFactor& f, double v) { return (float)__builtin_amdgcn_ldexp(v * f.f, -f.p); }

// |G|^2 is the Gram matrix's trace; then the steps, on A, Q = p(A) and the product P of the
// Qs, whose digits lie in LDS and whose tiles v, N, pv the waves hold as well.
template <int T>
__device__ __forceinline__ void ns_poly(const NsItem& it, char* ws, const NsCoef& k, char* lds, double* sums, float (*red)[kNsWaves])
{
    using PL = NsPoly<T>;
    constexpr int S = PL::S, TL = PL::TILES;
    char *const A = lds, *const Q = lds + PL::MATRIX, *const P = lds + 2 * PL::MATRIX;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool on = wave < PL::WAVES;
    int ctr = 0, par[TL] = {};
    if (on)
        ns_tiles_of<T>(wave, ctr, par);
    f64x4 v[TL], N[TL], pv[TL];
    bool diag[4], one[4];  // one: on the diagonal of the matrix's own part, so that padding sets no unit
    const bool tall = it.rows > it.cols;
    const double* part = reinterpret_cast<const double*>(ws + it.off);
    double tr = 0.0;
#pragma unroll
    for (int p = 0; p < TL; p++) {
        const bool turn = ctr > par[p];
        const int i = turn ? par[p] : ctr, j = turn ? ctr : par[p], n = i * T - i * (i - 1) / 2 + j - i;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = 4 * (lane >> 4) + q, c = lane & 15;
            diag[q] = r == c;
            one[q] = r == c && ns_short<T>(ctr * 16 + r, tall) < min(it.rows, it.cols);
            v[p][q] = part[n * 256 + (turn ? c * 16 + r : r * 16 + c)];
            if (diag[q] && ctr == par[p] && p == 0)  // (a diagonal tile is its wave's first)
                tr += v[p][q];
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        tr += shfl_xor_f64(tr, o);
    if (lane == 0)
        sums[wave] = on ? tr : 0.0;
    __syncthreads();
    tr = 0.0;
#pragma unroll
    for (int w = 0; w < kNsWaves; w++)
        tr += sums[w];
    const NsNorm norm = ns_norm(tr, k.eps);
    bool bad = !(tr < 0x1p1000);
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            v[p][q] = __builtin_amdgcn_ldexp(v[p][q] * norm.inv * norm.inv, -2 * norm.e);
    int eA = 1023, eQ, eR, eP = 0;  // (no entry passes the trace, 1)
    if (on)
        ns_store<T>(A, v, ns_up(eA), ctr, par, lane);
    __syncthreads();
    for (int t = 0; t < k.steps; t++) {
        const bool last = t + 1 == k.steps;
        // Q = a + b A + c A^2
        if (on) {
            ns_mul<T>(A, A, ns_unit(eA) * ns_unit(eA), N, ctr, par, lane);
#pragma unroll
            for (int p = 0; p < TL; p++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    N[p][q] = k.c * N[p][q] + k.b * v[p][q] + (one[q] && par[p] == ctr ? k.a : 0.0);
            const float m = ns_top<TL>(N);
            if (lane == 0)
                red[0][wave] = m;
        }
        __syncthreads();
        eQ = ns_exponent_of<PL::WAVES>(red[0], bad);
        if (on) {
            if (!last || t > 0)
                ns_store<T>(Q, N, ns_up(eQ), ctr, par, lane);
            if (t == 0) {
                ns_store<T>(P, N, ns_up(eQ), ctr, par, lane);
#pragma unroll
                for (int p = 0; p < TL; p++)
                    pv[p] = N[p];
            }
        }
        eP = t == 0 ? eQ : eP;
        __syncthreads();
        // A Q, and P <- P Q
        if (on) {
            if (t > 0) {
                ns_mul<T>(P, Q, ns_unit(eP) * ns_unit(eQ), pv, ctr, par, lane);
                const float m = ns_top<TL>(pv);
                if (lane == 0)
                    red[1][wave] = m;
            }
            if (!last) {
                ns_mul<T>(A, Q, ns_unit(eA) * ns_unit(eQ), v, ctr, par, lane);
                const float m = ns_top<TL>(v);
                if (lane == 0)
                    red[0][wave] = m;
            }
        }
        if (last)
            break;
        __syncthreads();
        eR = ns_exponent_of<PL::WAVES>(red[0], bad);
        eP = t > 0 ? ns_exponent_of<PL::WAVES>(red[1], bad) : eP;
        if (on) {
            ns_store<T>(A, v, ns_up(eR), ctr, par, lane);
            if (t > 0)
                ns_store<T>(P, pv, ns_up(eP), ctr, par, lane);
        }
        __syncthreads();
        // A <- (A Q) Q
        if (on) {
            ns_mul<T>(A, Q, ns_unit(eR) * ns_unit(eQ), v, ctr, par, lane);
            const float m = ns_top<TL>(v);
            if (lane == 0)
                red[0][wave] = m;
        }
        __syncthreads();
        eA = ns_exponent_of<PL::WAVES>(red[0], bad);
        if (on)
            ns_store<T>(A, v, ns_up(eA), ctr, par, lane);
        __syncthreads();
    }
    __syncthreads();
    if (!on)
        return;
    eP = k.steps > 1 ? ns_exponent_of<PL::WAVES>(red[1], bad) : eP;
    // the matrix's factor, with the norm and the scale, over the partials
    float* out = reinterpret_cast<float*>(ws + it.off);
    const NsFactor f = ns_factor<S>(it, norm, eP - 1022, bad, out);
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = ctr * 16 + 4 * (lane >> 4) + q, c = par[p] * 16 + (lane & 15);
            const float x = ns_entry(f, pv[p][q]);
            out[ns_short<T>(c, tall) * S + ns_short<T>(r, tall)] = x;
            if (par[p] != ctr)
                out[ns_short<T>(r, tall) * S + ns_short<T>(c, tall)] = x;
        }
}

// One block per matrix. Short sides up to 96 / 64: 61 / 30 us for five steps: 14 phases
// of products (28 of the 61 us at the 8-bit rate of one CU), rounding to digits, two barriers.
__global__ __launch_bounds__(64 * kNsWaves) void k_ns_poly(const NsItem* __restrict__ table, char* ws, const NsCoef k)
{
    __shared__ __attribute__((aligned(16))) char lds[kNsLds];
    __shared__ double sums[kNsWaves];
    __shared__ float red[2][kNsWaves];
    const NsItem it = table[blockIdx.x];
    if (it.tiles == 2)
        ns_poly<2>(it, ws, k, lds, sums, red);
    else if (it.tiles == 4)
        ns_poly<4>(it, ws, k, lds, sums, red);
    else
        ns_poly<6>(it, ws, k, lds, sums, red);
}

// The same in fp64, for steps that lift the smallest directions further than 40 bits reach.
// A direction that G lacks has an eigenvalue 0 in S, where rounding leaves one of either sign;
// a negative one never turns back (p(S) = a + |b| |S| + c S^2 only grows), so S starts with
// 2^-47 of its trace added to its diagonal: some eight times what the sums over 2^20 leave, and
// along a direction that G has, no more than fp32 products lose (a singular value of 1e-6 of the
// largest after 16 steps: 4.2e-3, where fp32 products give 2.8e-3). v_mfma_f64_16x16x4_f64, the
// matrices in LDS with rows four entries longer, so that the four rows of an operand read, and
// the sixteen of a mirrored write, spread over the banks. 22 us per step for a
// short side of 86, where 40 bits take 12.
constexpr double kNsShift = 0x1p-47;

template <int T>
struct NsPoly64 {
    static constexpr int S = 16 * T, LD = S + 4;
    static constexpr int TILES = (tri(T) + kNsWaves - 1) / kNsWaves;  // result tiles per wave
    // Element q of lane l of a 16 x 16 result: row 4 q + l / 16, column l % 16
    static __device__ __forceinline__ int row(int q, int lane) { return 4 * q + (lane >> 4); }
};

// X Y for symmetric matrices that commute, the upper tiles of this wave
template <int T>
__device__ __forceinline__ void ns_mul64(const double* X, const double* Y, f64x4 (&acc)[NsPoly64<T>::TILES],
                                         const int (&ti)[NsPoly64<T>::TILES], const int (&tj)[NsPoly64<T>::TILES], int lane)
{
    using P = NsPoly64<T>;
    const int i16 = lane & 15, kk = lane >> 4;
    int xa[P::TILES], ya[P::TILES];
#pragma unroll
    for (int p = 0; p < P::TILES; p++) {
        acc[p] = f64x4{0.0, 0.0, 0.0, 0.0};
        xa[p] = kk * P::LD + ti[p] * 16 + i16;
        ya[p] = kk * P::LD + tj[p] * 16 + i16;
    }
#pragma unroll 4
    for (int k0 = 0; k0 < P::S; k0 += 4)
#pragma unroll
        for (int p = 0; p < P::TILES; p++)
            acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(X[xa[p] + k0 * P::LD], Y[ya[p] + k0 * P::LD], acc[p], 0, 0, 0);
}

template <int T>
__device__ __forceinline__ void ns_store64(double* X, const f64x4 (&v)[NsPoly64<T>::TILES], const int (&ti)[NsPoly64<T>::TILES],
                                           const int (&tj)[NsPoly64<T>::TILES], int lane)
{
    using P = NsPoly64<T>;
#pragma unroll
    for (int p = 0; p < P::TILES; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            // (below the diagonal of a tile on it: the mirror image, whose sum may round otherwise)
            const int r = ti[p] * 16 + P::row(q, lane), c = tj[p] * 16 + (lane & 15);
            if (r <= c) {
                X[r * P::LD + c] = v[p][q];
                X[c * P::LD + r] = v[p][q];
            }
        }
}

// The steps on A, Q in LDS and the waves' result tiles, the product P of the Qs through A's
// place. Waves past the tiles repeat the last tile (the same values to the same places).
template <int T>
__device__ __forceinline__ void ns_poly64(const NsItem& it, char* ws, const NsCoef& k, double* A, double* Q, float* red)
{
    using PL = NsPoly64<T>;
    constexpr int S = PL::S, TL = PL::TILES;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool tall = it.rows > it.cols;
    const int s = min(it.rows, it.cols);
    int ti[TL], tj[TL];
    bool diag[TL][4];  // on the diagonal of the matrix's own part
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
#pragma unroll
        for (int q = 0; q < 4; q++)
            diag[p][q] = n == 0 && PL::row(q, lane) == (lane & 15) && ns_short<T>(i * 16 + (lane & 15), tall) < s;
    }
    ns_store64<T>(A, v, ti, tj, lane);
    __syncthreads();
    double tr = 0.0;
    for (int i = 0; i < S; i++)
        tr += A[i * PL::LD + i];
    const NsNorm norm = ns_norm(tr, k.eps);
    bool bad = !(tr < 0x1p1000);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            v[p][q] = __builtin_amdgcn_ldexp(v[p][q] * norm.inv * norm.inv, -2 * norm.e) + (diag[p][q] ? kNsShift : 0.0);
    ns_store64<T>(A, v, ti, tj, lane);
    __syncthreads();
    for (int t = 0; t < k.steps; t++) {
        const bool last = t + 1 == k.steps;
        // v: A's tiles. N = A^2, then Q = a + b A + c A^2
        ns_mul64<T>(A, A, N, ti, tj, lane);
#pragma unroll
        for (int p = 0; p < TL; p++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                N[p][q] = k.c * N[p][q] + k.b * v[p][q] + (diag[p][q] ? k.a : 0.0);
        ns_store64<T>(Q, N, ti, tj, lane);
        __syncthreads();
        if (!last) {  // A <- (A Q) Q
            ns_mul64<T>(A, Q, v, ti, tj, lane);
            __syncthreads();
            ns_store64<T>(A, v, ti, tj, lane);
            __syncthreads();
            ns_mul64<T>(A, Q, v, ti, tj, lane);
            __syncthreads();
        }
        if (t == 0) {
#pragma unroll
            for (int p = 0; p < TL; p++)
                P[p] = N[p];
        } else {  // P <- P Q, through A's place
            ns_store64<T>(A, P, ti, tj, lane);
            __syncthreads();
            ns_mul64<T>(A, Q, P, ti, tj, lane);
            __syncthreads();
        }
        if (!last) {
            ns_store64<T>(A, v, ti, tj, lane);
            __syncthreads();
        }
    }
    // the matrix's factor, with the norm and the scale, over the partials
    const float m = ns_top<TL>(P);
    if (lane == 0)
        red[wave] = m;
    __syncthreads();
    const int eP = ns_exponent_of<kNsWaves>(red, bad);
    float* out = reinterpret_cast<float*>(ws + it.off);
    const NsFactor f = ns_factor<S>(it, norm, eP - 1022, bad, out);
#pragma unroll
    for (int p = 0; p < TL; p++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = ti[p] * 16 + PL::row(q, lane), c = tj[p] * 16 + (lane & 15);
            const float x = ns_entry(f, P[p][q]);
            if (r <= c) {
                out[ns_short<T>(r, tall) * S + ns_short<T>(c, tall)] = x;
                out[ns_short<T>(c, tall) * S + ns_short<T>(r, tall)] = x;
            }
        }
}

// One block per matrix
__global__ __launch_bounds__(64 * kNsWaves) void k_ns_poly64(const NsItem* __restrict__ table, char* ws, const NsCoef k)
{
    __shared__ double lds[2][NsPoly64<6>::S * NsPoly64<6>::LD];
    __shared__ float red[kNsWaves];
    const NsItem it = table[blockIdx.x];
    if (it.tiles == 2)
        ns_poly64<2>(it, ws, k, lds[0], lds[1], red);
    else if (it.tiles == 4)
        ns_poly64<4>(it, ws, k, lds[0], lds[1], red);
    else
        ns_poly64<6>(it, ws, k, lds[0], lds[1], red);
}

// --------------------------------------------------------- short form: the product --

// out = G F (tall) or F G (wide), F the symmetric factor: v_mfma_f32_16x16x4_f32 with F's
// rows as A and G as B; a wave holds a run of 16 of the long side in registers before it
// writes any of it, so out may be G. The contraction index 16 st + 4 (l / 16) + u is taken
// by product u of step st, so that a lane's four are consecutive in a tall matrix's row, as
// are the four results it ends with. Bound by memory: 224 matrices, 406 MB in 95 us (4.3
// TB/s; a copy reaches 5.15); 7 matrices: 12 us.
template <int T, bool HALF>
__device__ __forceinline__ void ns_apply(const NsItem& it, int block, const float* f, float* F)
{
    constexpr int S = 16 * T, LD = S + 4, SH = HALF ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = tid; e < S * S / 4; e += 256)
        *reinterpret_cast<nf4*>(&F[e / (S / 4) * LD + e % (S / 4) * 4]) = reinterpret_cast<const nf4*>(f)[e];
    __syncthreads();
    const int eg = reinterpret_cast<const int*>(f)[S * S], eo = reinterpret_cast<const int*>(f)[S * S + 1];  // (ns_factor)
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
                for (int u = 0; u < 4; u++) {  // (rows past the last are out of range)
                    const int off = n16 < len ? (int)(((int64_t)(i + u) * it.cols + n16) << SH) : kNsDead;
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
        for (int st = 0; st < T; st++) {
#pragma unroll
            for (int u = 0; u < 4; u++)
                v[st][u] = __builtin_amdgcn_ldexpf(v[st][u], eg);
#pragma unroll
            for (int t = 0; t < T; t++) {
                const nf4 a = *reinterpret_cast<const nf4*>(&F[(t * 16 + n16) * LD + 16 * st + 4 * kk]);
#pragma unroll
                for (int u = 0; u < 4; u++)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[u], v[st][u], acc[t], 0, 0, 0);
            }
        }
        if (n16 < len) {
            char* ob = static_cast<char*>(it.out) + ((lb * sl) << SH);
#pragma unroll
            for (int t = 0; t < T; t++) {
                const int i = t * 16 + 4 * kk;
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[t][q] = __builtin_amdgcn_ldexpf(acc[t][q], eo);
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
                                                  const char* ws, int first)
{
    __shared__ float F[96 * 100];
    const int at = first + (int)blockIdx.x;
    const NsItem it = table[__builtin_amdgcn_readfirstlane(item[at])];
    const int block = at - it.apply0;
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
// low twice; low by low lies below the pairs' precision), with fp32 sums: 3 times the rate
// of the fp32 matrix instructions. m comes from a bound of the singular values after each
// step, which the caller of the kernels works out from the coefficients, so nothing
// overflows.
//
// A number's high and low halves lie 32 bytes apart: 16 highs, 16 lows, 16 highs, ... along
// a row, so that 16 of a row are one run of 64 bytes, which is what a stage of the products
// takes. X lies with the long side contiguous, padded with zeros: the short side to 128, the
// long side to 256.
struct NsLong {
    int64_t sp, lp;
    int64_t sq, x, x_next, A, B, parts;  // byte offsets
    int32_t sqn;
    int32_t high;         // tiles of 128 down the short side
    int32_t wide;         // tiles of A and of X' are 128 x 256, else 128 x 128
    int32_t tiles, gram;  // tiles of A on and above the diagonal, parts of the long side
    int32_t squares;      // the same of A^2, 128 x 128
};

constexpr int kNsTile = 128, kNsDepth = 16;  // of the products: rows of a tile, contraction per stage
constexpr int kNsMaxParts = 64;

// gram: the parts, ns_parts' choice
__host__ __device__ inline NsLong ns_long(int64_t rows, int64_t cols, int32_t gram)
{
    NsLong n;
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    n.sp = (s + 127) & ~(int64_t)127;
    n.lp = (l + 255) & ~(int64_t)255;
    n.high = (int)(n.sp >> 7);
    n.squares = n.high * (n.high + 1) / 2;
    // 128 x 256 where they fill the 256 CUs (X' of 2048 x 4096: 100 against 112 us), else
    // twice as many that half as many bytes feed
    n.wide = n.high * (n.lp >> 8) >= 256;
    const int half = (n.high + 1) / 2;
    n.tiles = n.wide ? half * (half + 1) - (n.high & 1) : n.squares;
    n.gram = gram;
    const int64_t sq = (s * l + 16383) >> 14;
    n.sqn = (int32_t)(sq < 1024 ? sq : 1024);
    n.sq = 0;
    n.x = 8192;
    n.x_next = n.x + 4 * n.sp * n.lp;
    n.A = n.x_next + 4 * n.sp * n.lp;
    n.B = n.A + 4 * n.sp * n.sp;
    n.parts = n.B + 4 * n.sp * n.sp;
    return n;
}

int64_t ns_long_bytes(const NsLong& n) { return n.parts + (int64_t)n.gram * n.tiles * (n.wide ? 2 : 1) * (4 * 128 * 128); }

// The long side in parts: the rounds of 256 blocks that they take (0.35 us per 128 x 128 and
// stage) against the partial tiles that are written and read (64 KB each, at 4 TB/s); a part
// has at least 16 stages.
int ns_parts(int64_t rows, int64_t cols)
{
    const NsLong n = ns_long(rows, cols, 1);
    const int stages = (int)(n.lp / kNsDepth);
    double best = 0.0;
    int parts = 1;
    for (int p = 1; p <= kNsMaxParts && (p == 1 || p * 16 <= stages); p++) {
        const int rounds = (n.tiles * p + 255) / 256;
        const double t = (n.wide ? 2 : 1) * rounds * ((stages + p - 1) / p) * 0.35 + (double)(p * n.squares) * 0.033;
        if (p == 1 || t < best) {
            best = t;
            parts = p;
        }
    }
    return parts;
}

// place of element (r, c) of a matrix of pairs in 16-bit units; its low half lies 16 further on
__host__ __device__ inline int64_t ns_place(int64_t r, int64_t c, int64_t pitch)
{
    return 2 * r * pitch + ((c >> 4) << 5) + (c & 15);
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

// blockIdx.y: the matrix, in all kernels of the long form. 2048 x 4096 fp32: 8.8 us, 34 MB at
// 3.8 TB/s.
__global__ __launch_bounds__(256) void k_nsl_sumsq(const NsItem* __restrict__ table, char* ws)
{
    __shared__ double red[4];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
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

// X = G / (|G| + eps), padded with zeros. 64 x 64 tiles. 2048 x 4096 fp32: 14.5 us, 67 MB at 4.6
// TB/s.
__global__ __launch_bounds__(256) void k_nsl_init(const NsItem* __restrict__ table, char* ws, double eps, float scale)
{
    __shared__ double red[4];
    __shared__ float tile[64][65];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
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
    const double sum = ns_block_sum((part[0] + part[1]) + (part[2] + part[3]), red);
    const double inv = sum == 0.0 ? 0.0 : 1.0 / (sqrt(sum) + eps);  // (1 / eps may be infinite)
    for (int r = r0; r < 64; r += 4)
        tile[r][c] = (float)((double)v[(r - r0) / 4] * inv) * scale;
    __syncthreads();
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + it.off + n.x);
    for (int r = r0; r < 64; r += 4) {
        const NsPair p = ns_pair(tall ? tile[c][r] : tile[r][c]);
        const int64_t at = ns_place(i0 + r, l0 + c, n.lp);
        x[at] = p.hi;
        x[at + 16] = p.lo;
    }
}

// out = scale X, X times 2^m taken back by `unscale`. 2048 x 4096 fp32: 11.7 us, 5.7 TB/s.
__global__ __launch_bounds__(256) void k_nsl_out(const NsItem* __restrict__ table, const char* ws, int from, float unscale)
{
    __shared__ float tile[64][65];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
    const int64_t tl = n.lp / 64;
    if (blockIdx.x >= (n.sp / 64) * tl)
        return;
    const bool tall = it.rows > it.cols;
    const int64_t i0 = blockIdx.x / tl * 64, l0 = blockIdx.x % tl * 64;
    const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    const uint16_t* x = reinterpret_cast<const uint16_t*>(ws + it.off + (from ? n.x_next : n.x));
    uint16_t hi[16], lo[16];
    const int64_t at0 = ns_place(i0 + r0, l0 + c, n.lp);
#pragma unroll
    for (int q = 0; q < 16; q++) {
        hi[q] = x[at0 + 8 * q * n.lp];
        lo[q] = x[at0 + 8 * q * n.lp + 16];
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

// A tile of P Q^T over stages c0 .. c1 - 1 of the contraction, 128 rows of P by 128 FP of Q,
// 8 waves of 32 FP x 64, operands read one stage ahead, in a ring of six stages (FP = 2) or of
// eight with a barrier for every second one (FP = 1: its stages are half as long). P: rows
// with the contraction contiguous (pitch in bytes), Q: likewise, q_rows of them, or (TURN)
// rows along the contraction, 128 FP columns of each, which ds_read_tr turns round. Result
// element r of a lane in acc[g][f]: Q's row (of 32 (2 wq + f)) l % 32, P's row
// 8 (r / 4) + 4 (l / 32) + r % 4 (of 32 (FP wp + g)), or the other way round (TURN: four
// consecutive columns).
//
// X' of 2048 x 4096, 103 GFLOP in three products: 100 us, 1.03 PFLOP/s (the library's fp16 product
// of 8192^3: 1.4). Products alone take 75 us of it, loads alone 61; the matrix cores are busy
// 60 % of the cycles at 1.9 GHz and no LDS access meets a conflict. FP = 1 there: 112.
// Two blocks per CU (FP = 1, rings of four): 139. Rows padded off powers of two: no change.
constexpr int kNsStageP = kNsTile * 64;
typedef short ns_s4 __attribute__((ext_vector_type(4)));

template <int FP, bool TURN>
__device__ __forceinline__ void ns_product(const char* p, int64_t p_pitch, const char* q, int64_t q_pitch, int q_rows, int c0,
                                           int c1, char* s0, char* s1, char* s2, char* s3, char* s4, char* s5, char* s6,
                                           char* s7, nf16 (&acc)[FP][2])
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = FP == 2 ? wave & 1 : wave & 3, wq = FP == 2 ? wave >> 1 : wave >> 2;
    const int l32 = lane & 31, h = lane >> 5;
    // turned: 64 FP-byte units per row; unit c of row r in slot c ^ (2 (r % 2) + 8 (r / 2 % 2)),
    // so that the two times 32 bytes that a read takes of each of four rows lie in different banks
    auto turn = [](int row) { return ((row & 1) << 1) | ((row & 2) << 2); };
    const int up = wave * 64 + lane;
    const int src_p = stage_row(up) * (int)p_pitch + stage_piece(up) * 16;
    int src_q[FP];
#pragma unroll
    for (int t = 0; t < FP; t++) {
        const int u = (wave * FP + t) * 64 + lane, row = u / (32 * FP);
        src_q[t] = TURN ? row * (int)q_pitch + ((u & (32 * FP - 1)) ^ turn(row)) * 16
                        : stage_row(u) * (int)q_pitch + stage_piece(u) * 16;
    }
    const __amdgpu_buffer_rsrc_t rp = uniform_rsrc(p, (int64_t)kNsTile * p_pitch);
    const __amdgpu_buffer_rsrc_t rq = uniform_rsrc(q, (int64_t)(TURN ? kNsDepth : q_rows) * q_pitch);
    auto dma = [&](int c, char* stage) {
        const int dead = c < c1 ? 0 : kDeadLoad, cc = min(c, c1 - 1);
        dma16_lds(rp, stage + wave * 1024, (src_p + cc * 64) | dead);
        // (turned: the rows may reach far, so the descriptor moves)
        const __amdgpu_buffer_rsrc_t r =
            TURN ? uniform_rsrc(q + (int64_t)cc * kNsDepth * q_pitch, (int64_t)kNsDepth * q_pitch) : rq;
#pragma unroll
        for (int t = 0; t < FP; t++)
            dma16_lds(r, stage + kNsStageP + (wave * FP + t) * 1024, (src_q[t] + (TURN ? 0 : cc * 64)) | dead);
    };
    int pa[2], qa[2][2];  // [high, low]
#pragma unroll
    for (int e = 0; e < 2; e++) {
        pa[e] = wp * FP * 2048 + stage_at(l32, 2 * e + h);
#pragma unroll
        for (int f = 0; f < 2; f++) {
            if (TURN) {
                // in a group of 16 lanes, lane i names 4 columns of row i / 4 and gets column
                // i of the 4 rows; the rows 4 further on by a second read
                const int row = 8 * h + ((lane & 15) >> 2);
                const int unit = (wq * 4 + 2 * f + ((lane >> 4) & 1)) * 4 + 2 * e + ((lane & 3) >> 1);
                qa[e][f] = kNsStageP + row * (512 * FP) + (unit ^ turn(row)) * 16 + (lane & 1) * 8;
            } else
                qa[e][f] = kNsStageP + (wq * 2 + f) * 2048 + stage_at(l32, 2 * e + h);
        }
    }
    half8_t pv[2][2][FP], qv[2][2][2];  // [set][high, low][g or f]
    auto read = [&](const char* stage, int st) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
#pragma unroll
            for (int g = 0; g < FP; g++)
                pv[st][e][g] = *reinterpret_cast<const half8_t*>(stage + pa[e] + g * 2048);
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const char* at = stage + qa[e][f];
                if (TURN) {
                    const ns_s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) ns_s4*)at);
                    const ns_s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) ns_s4*)(at + 4 * 512 * FP));
                    qv[st][e][f] = __builtin_bit_cast(half8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
                } else
                    qv[st][e][f] = *reinterpret_cast<const half8_t*>(at);
            }
        }
    };
    auto hold = [&](int st) {  // the reads of this set are done here
#pragma unroll
        for (int e = 0; e < 2; e++)
            asm volatile("" ::"v"(pv[st][e][0]), "v"(pv[st][e][FP - 1]), "v"(qv[st][e][0]), "v"(qv[st][e][1]));
    };
    auto mul = [&](int c, int st, const char* next) {
        if (c >= c1)
            return;
        read(next, st ^ 1);
#pragma unroll
        for (int e = 0; e < 3; e++)  // high high, high low, low high
#pragma unroll
            for (int g = 0; g < FP; g++)
#pragma unroll
                for (int f = 0; f < 2; f++) {
                    const half8_t a = pv[st][e == 2 ? 1 : 0][g], b = qv[st][e == 1 ? 1 : 0][f];
                    acc[g][f] = TURN ? __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, acc[g][f], 0, 0, 0)
                                     : __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc[g][f], 0, 0, 0);
                }
#pragma unroll
        for (int e = 0; e < 6 * FP; e++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, FP == 2 ? 1 : 2, 0);
        }
        hold(st);
    };
    dma(c0, s0);
    dma(c0 + 1, s1);
    dma(c0 + 2, s2);
    dma(c0 + 3, s3);
    dma(c0 + 4, s4);
    if constexpr (FP == 2) {
        auto step = [&](int c, int st, const char* next, char* fill) {
            stage_barrier<9, 15>();  // stage c + 1 has arrived, everyone has read stage c - 1
            dma(c + 5, fill);
            mul(c, st, next);
        };
        stage_barrier<12>();
        read(s0, 0);
        for (int c = c0; c < c1; c += 6) {
            step(c, 0, s1, s5);
            step(c + 1, 1, s2, s0);
            step(c + 2, 0, s3, s1);
            step(c + 3, 1, s4, s2);
            step(c + 4, 0, s5, s3);
            step(c + 5, 1, s0, s4);
        }
    } else {
        auto step = [&](int c, const char* n1, const char* n2, char* f1, char* f2) {
            stage_barrier<6, 15>();  // stage c + 2 has arrived, everyone has read stage c - 1
            dma(c + 6, f1);
            dma(c + 7, f2);
            mul(c, 0, n1);
            mul(c + 1, 1, n2);
        };
        dma(c0 + 5, s5);
        stage_barrier<10>();
        read(s0, 0);
        for (int c = c0; c < c1; c += 8) {
            step(c, s1, s2, s6, s7);
            step(c + 2, s3, s4, s0, s1);
            step(c + 4, s5, s6, s2, s3);
            step(c + 6, s7, s0, s4, s5);
        }
    }
    hold(0);
    hold(1);
    stage_barrier<0>();  // the loads past the end have written their zeros
}

#define NS_STAGES                                                                              \
    constexpr int kStage = kNsStageP * (FP + 1), kSpare = FP == 1 ? kStage : 16;               \
    __shared__ __attribute__((aligned(1024))) char s0[kStage], s1[kStage], s2[kStage], s3[kStage], s4[kStage], s5[kStage], \
        s6[kSpare], s7[kSpare]

template <int FP>
__device__ __forceinline__ void ns_clear(nf16 (&acc)[FP][2])
{
#pragma unroll
    for (int g = 0; g < FP; g++)
#pragma unroll
        for (int f = 0; f < 2; f++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[g][f][r] = 0.0f;
}

// Tile n of those on and above the diagonal of a matrix T tiles high
template <int FP>
__device__ __forceinline__ void ns_upper(int n, int T, int& ti, int& tj)
{
    tj = 0;
    for (;;) {
        const int here = min(T, (tj + 1) * FP);
        if (n < here)
            break;
        n -= here;
        tj++;
    }
    ti = n;
}

// A = X X^T, the tiles on and above the diagonal, parts of the long side each, left in lane
// order. 2048 x 4096: 59 us, three parts on 216 CUs (one part of 128 x 128 tiles, 136 CUs: 75).
template <int FP>
__device__ __forceinline__ void ns_gram_tile(const NsLong& n, char* ws, int from, int block, char* s0, char* s1, char* s2, char* s3,
                                             char* s4, char* s5, char* s6, char* s7)
{
    nf16 acc[FP][2];
    ns_clear(acc);
    // an XCD takes consecutive places: the tiles of one part together
    const int place = xcd_place(block, n.tiles * n.gram);
    const int tile = place % n.tiles, part = place / n.tiles, all = (int)(n.lp / kNsDepth);
    int ti, tj;
    ns_upper<FP>(tile, n.high, ti, tj);
    const char* x = ws + (from ? n.x_next : n.x);
    const int64_t pitch = 4 * n.lp;
    ns_product<FP, false>(x + ti * kNsTile * pitch, pitch, x + (int64_t)tj * (128 * FP) * pitch, pitch,
                          (int)min((int64_t)(128 * FP), n.sp - tj * (128 * FP)), all * part / n.gram, all * (part + 1) / n.gram, s0,
                          s1, s2, s3, s4, s5, s6, s7, acc);
    nf4* to = reinterpret_cast<nf4*>(ws + n.parts) + (int64_t)(tile * n.gram + part) * (kNsTile * 32 * FP) +
              (threadIdx.x >> 6) * (512 * FP) + (threadIdx.x & 63);
#pragma unroll
    for (int g = 0; g < FP; g++)
#pragma unroll
        for (int f = 0; f < 2; f++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                to[((g * 2 + f) * 4 + e) * 64] =
                    nf4{acc[g][f][4 * e], acc[g][f][4 * e + 1], acc[g][f][4 * e + 2], acc[g][f][4 * e + 3]};
}

template <int FP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_gram(const NsItem* __restrict__ table,
                                                                                             char* ws, int from)
{
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
    if (n.wide != (FP == 2) || (int)blockIdx.x >= n.tiles * n.gram)
        return;
    ns_gram_tile<FP>(n, ws + it.off, from, (int)blockIdx.x, s0, s1, s2, s3, s4, s5, s6, s7);
}

// Results leave by way of LDS, a wave's 32 x 32 at a time, in runs of 16 numbers per lane (64
// bytes: highs and lows). kNsPiece: floats that a wave needs for it.
constexpr int kNsPitch = 33, kNsPiece = 32 * kNsPitch;

struct NsRun {
    uint4 q[4];  // 16 highs, 16 lows
};
__device__ __forceinline__ NsRun ns_get(const uint16_t* p)
{
    NsRun r;
#pragma unroll
    for (int i = 0; i < 4; i++)
        r.q[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
__device__ __forceinline__ float ns_value(const NsRun& r, int i)
{
    const uint4 h = r.q[i >> 3], l = r.q[2 + (i >> 3)];
    const uint32_t wh = (i & 6) == 0 ? h.x : (i & 6) == 2 ? h.y : (i & 6) == 4 ? h.z : h.w;
    const uint32_t wl = (i & 6) == 0 ? l.x : (i & 6) == 2 ? l.y : (i & 6) == 4 ? l.z : l.w;
    return h2f((uint16_t)(wh >> (16 * (i & 1)))) + h2f((uint16_t)(wl >> (16 * (i & 1))));
}
__device__ __forceinline__ void ns_put(uint16_t* p, const float (&v)[16])
{
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const NsPair a = ns_pair(v[2 * i]), b = ns_pair(v[2 * i + 1]);
        w[i] = a.hi | ((uint32_t)b.hi << 16);
        w[8 + i] = a.lo | ((uint32_t)b.lo << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// LDS of one wave: its writes before its reads (they run in order)
__device__ __forceinline__ void ns_wave_lds()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// A 32 x 32 piece of a symmetric matrix, at (ib, jb) on or above the diagonal, to both its
// places; v as the products leave it: row 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
__device__ __forceinline__ void ns_put_both(uint16_t* m, int64_t pitch, int ib, int jb, const nf16& v, float* T, int lane)
{
#pragma unroll
    for (int r = 0; r < 16; r++)
        T[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * kNsPitch + (lane & 31)] = v[r];
    ns_wave_lds();
    const int row = lane >> 1, c0 = (lane & 1) * 16;
    float up[16];
#pragma unroll
    for (int c = 0; c < 16; c++)  // on the diagonal the upper half serves both
        up[c] = ib == jb && c0 + c < row ? T[(c0 + c) * kNsPitch + row] : T[row * kNsPitch + c0 + c];
    ns_put(m + ns_place(ib + row, jb + c0, pitch), up);
    if (ib != jb) {
#pragma unroll
        for (int c = 0; c < 16; c++)
            up[c] = T[(c0 + c) * kNsPitch + row];
        ns_put(m + ns_place(jb + row, ib + c0, pitch), up);
    }
    ns_wave_lds();
}

// The parts' sums, a block per 32 x 32 piece: a wave adds every fourth part, the first adds
// theirs. scale: the power of two of A over that of X squared. 2048: 13 us, 45 MB.
template <int FP>
__device__ __forceinline__ void ns_sum(const NsLong& n, char* ws, int piece, float scale, float* lds)
{
    constexpr int V = kNsTile * 32 * FP;  // vectors of four in a tile
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = piece / (16 * FP), at = piece % (16 * FP);
    int ti, tj;
    ns_upper<FP>(tile, n.high, ti, tj);
    const int wave = at / (2 * FP), g = FP == 2 ? (at >> 1) & 1 : 0, f = at & 1;
    const int wp = FP == 2 ? wave & 1 : wave & 3, wq = FP == 2 ? wave >> 1 : wave >> 2;
    const int ib = ti * kNsTile + (wp * FP + g) * 32, jb = tj * (128 * FP) + (wq * 2 + f) * 32;
    if (jb >= n.sp || ib > jb)
        return;
    const nf4* p = reinterpret_cast<const nf4*>(ws + n.parts) + (int64_t)tile * n.gram * V + at * 256 + lane;
    nf16 s;
#pragma unroll
    for (int r = 0; r < 16; r++)
        s[r] = 0.0f;
    for (int part = w; part < n.gram; part += 8) {
        nf4 v[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[u][e] = part + 4 * u < n.gram ? p[(int64_t)(part + 4 * u) * V + e * 64] : nf4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                s[r] += v[u][r >> 2][r & 3];
    }
    nf4* mine = reinterpret_cast<nf4*>(lds) + (w - 1) * 256 + lane;
    if (w > 0) {
#pragma unroll
        for (int e = 0; e < 4; e++)
            mine[e * 64] = nf4{s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]};
    }
    __syncthreads();
    if (w > 0)
        return;
#pragma unroll
    for (int u = 1; u < 4; u++)
#pragma unroll
        for (int r = 0; r < 16; r++)
            s[r] += mine[u * 256 + (r >> 2) * 64][r & 3];
    ns_wave_lds();
    ns_put_both(reinterpret_cast<uint16_t*>(ws + n.A), n.sp, ib, jb, s * scale, lds, lane);
}

__global__ __launch_bounds__(256) void k_nsl_sum(const NsItem* __restrict__ table, char* ws, float scale)
{
    __shared__ __attribute__((aligned(16))) float lds[3 * 1024 > kNsPiece ? 3 * 1024 : kNsPiece];
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
    if ((int)blockIdx.x >= n.tiles * (n.wide ? 32 : 16))
        return;
    if (n.wide)
        ns_sum<2>(n, ws + it.off, (int)blockIdx.x, scale, lds);
    else
        ns_sum<1>(n, ws + it.off, (int)blockIdx.x, scale, lds);
}

// B = b A + c A^2; b and c with the powers of two of A and B. 2048: 58 us on 136 of the CUs (128 x
// 256 tiles in three parts and their sum: 45 + 12).
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_poly(const NsItem* __restrict__ table,
                                                                                             char* ws, float b, float c)
{
    constexpr int FP = 1;
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
    if ((int)blockIdx.x >= n.squares)
        return;
    nf16 acc[1][2];
    ns_clear(acc);
    int ti, tj;
    ns_upper<1>((int)blockIdx.x, n.high, ti, tj);
    const char* A = ws + it.off + n.A;
    const int64_t pitch = 4 * n.sp;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ib = ti * kNsTile + (wave & 3) * 32, jb = tj * kNsTile + (wave >> 2) * 64;
    // (from below the diagonal: four of a column lie side by side there)
    uint2 hi[8], lo[8];
#pragma unroll
    for (int q = 0; q < 8; q++) {
        const uint16_t* from = reinterpret_cast<const uint16_t*>(A) +
                               ns_place(jb + 32 * (q >> 2) + (lane & 31), ib + 8 * (q & 3) + 4 * (lane >> 5), n.sp);
        hi[q] = *reinterpret_cast<const uint2*>(from);
        lo[q] = *reinterpret_cast<const uint2*>(from + 16);
    }
    ns_product<1, false>(A + ti * kNsTile * pitch, pitch, A + tj * kNsTile * pitch, pitch, kNsTile, 0, (int)(n.sp / kNsDepth), s0, s1,
                         s2, s3, s4, s5, s6, s7, acc);
    float* T = reinterpret_cast<float*>(wave < 2 ? s0 : wave < 4 ? s1 : wave < 6 ? s2 : s3) + (wave & 1) * kNsPiece;
#pragma unroll
    for (int f = 0; f < 2; f++) {
        nf16 v;
#pragma unroll
        for (int r = 0; r < 16; r++) {
            const int q = f * 4 + (r >> 2);
            const uint32_t h = r & 2 ? hi[q].y : hi[q].x, l = r & 2 ? lo[q].y : lo[q].x;
            const float x = h2f((uint16_t)(h >> (16 * (r & 1)))) + h2f((uint16_t)(l >> (16 * (r & 1))));
            v[r] = __builtin_fmaf(c, acc[0][f][r], b * x);
        }
        if (ib <= jb + 32 * f)
            ns_put_both(reinterpret_cast<uint16_t*>(ws + it.off + n.B), n.sp, ib, jb + 32 * f, v, T, lane);
    }
}

// X' = a X + B X; a and the product with the powers of two of X, B and X'
template <int FP>
__device__ __forceinline__ void ns_step(const NsLong& n, char* ws, int block, float a, float scale, int from, char* s0, char* s1,
                                        char* s2, char* s3, char* s4, char* s5, char* s6, char* s7)
{
    nf16 acc[FP][2];
    ns_clear(acc);
    const int high = n.high, place = xcd_place(block, high * (int)(n.lp / (128 * FP)));
    const int ti = place % high;
    const int64_t l0 = (int64_t)(place / high) * (128 * FP);
    const char* x = ws + (from ? n.x_next : n.x);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wp = FP == 2 ? wave & 1 : wave & 3, wq = FP == 2 ? wave >> 1 : wave >> 2;
    // this lane's runs of X: 16 of row lane / 2 of every 32 x 32 piece, there before the
    // products are done
    const int64_t at0 = ns_place(ti * kNsTile + wp * FP * 32 + (lane >> 1), l0 + wq * 64 + (lane & 1) * 16, n.lp);
    NsRun old[FP][2];
#pragma unroll
    for (int g = 0; g < FP; g++)
#pragma unroll
        for (int f = 0; f < 2; f++)
            old[g][f] = ns_get(reinterpret_cast<const uint16_t*>(x) + at0 + 64 * g * n.lp + 64 * f);
    ns_product<FP, true>(ws + n.B + ti * kNsTile * (4 * n.sp), 4 * n.sp, x + 4 * l0, 4 * n.lp, 0, 0, (int)(n.sp / kNsDepth), s0, s1,
                         s2, s3, s4, s5, s6, s7, acc);
    uint16_t* y = reinterpret_cast<uint16_t*>(ws + (from ? n.x : n.x_next));
    float* T = reinterpret_cast<float*>(wave < 2 ? s0 : wave < 4 ? s1 : wave < 6 ? s2 : s3) + (wave & 1) * kNsPiece;
#pragma unroll
    for (int g = 0; g < FP; g++)
#pragma unroll
        for (int f = 0; f < 2; f++) {
#pragma unroll
            for (int r = 0; r < 16; r++)
                T[(lane & 31) * kNsPitch + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)] = acc[g][f][r];
            ns_wave_lds();
            float v[16];
#pragma unroll
            for (int c = 0; c < 16; c++)
                v[c] = __builtin_fmaf(a, ns_value(old[g][f], c), T[(lane >> 1) * kNsPitch + (lane & 1) * 16 + c] * scale);
            ns_put(y + at0 + 64 * g * n.lp + 64 * f, v);
            ns_wave_lds();
        }
}

template <int FP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_nsl_step(const NsItem* __restrict__ table,
                                                                                             char* ws, float a, float scale, int from)
{
    NS_STAGES;
    const NsItem it = table[blockIdx.y];
    const NsLong n = ns_long(it.rows, it.cols, it.slices);
    if (n.wide != (FP == 2) || (int)blockIdx.x >= n.high * (int)(n.lp / (128 * FP)))
        return;
    ns_step<FP>(n, ws + it.off, (int)blockIdx.x, a, scale, from, s0, s1, s2, s3, s4, s5, s6, s7);
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

// Whether 40 bits do for the short form's polynomial. What it leaves along a direction grows
// with every step by the square of the factor p(S) that the step lifts it by, and is as small
// as what fp32 products of X leave (2^-24, growing by p(S) itself) until those factors' largest
// have multiplied to some 2^11. Relative error of a 700 x 86 matrix of rank 8 | that of fp32
// products | with fp64 here, by that product: (3.4445, -4.775, 2.0315), 6 steps (1670) 6.9e-5 | 7.7e-5,
// 7 (5753) 6.2e-4 | 2.1e-4 | 1.9e-4, 8 2e-2 | 8.4e-4 | 7.8e-4; (1.875, -1.25, 0.375), 12 steps (1888)
// 7.2e-5 | 4.8e-5, 13 (3540) 2.4e-4 | 1e-4 | 1.2e-4, 14 1.3e-3 | 1.8e-4 | 2.2e-4; (3, -3.2, 1.2), 6
// steps (729) 2.4e-5 | 2.7e-5, 8 (6561) 9.8e-4 | 2.2e-4 | 2.1e-4. Up to 16 steps fp64 stays near fp32
// products; five steps of 4096 x 86 take 92 us with 40 bits, eight 128, and eight with fp64 204.
// The largest of |p| and of the singular values that a step leaves lie at the ends of its
// range or where the derivatives vanish.
bool ns_fixed(double a, double b, double c, int steps)
{
    double x2 = 1.0, growth = 1.0;  // the largest eigenvalue of S
    for (int t = 0; t < steps; t++) {
        auto p = [&](double l) { return std::fabs(a + b * l + c * l * l); };
        double most = std::fmax(p(0.0), p(x2)), next = x2 * p(x2) * p(x2);
        const double top = -b / (2.0 * c);
        if (top > 0.0 && top < x2)
            most = std::fmax(most, p(top));
        // d/dx x p(x^2) = a + 3 b l + 5 c l^2
        const double disc = 9.0 * b * b - 20.0 * a * c;
        for (const double sign : {-1.0, 1.0}) {
            const double l = c != 0.0 ? (-3.0 * b + sign * std::sqrt(disc)) / (10.0 * c) : -a / (3.0 * b);
            if (l > 0.0 && l < x2)
                next = std::fmax(next, l * p(l) * p(l));
        }
        growth *= most;
        x2 = next;
    }
    return growth <= 2048.0;  // (a NaN is not)
}

// ------------------------------------------------------------------ the plan --

// Short sides of the short form: the digits of three 96 x 96 matrices fill a CU's LDS. Five steps,
// short | long form, us: 96 x 96 95 | 164, 4096 x 96 94 | 172, 4096 x 64 50 | 172, 2^18 x 96 313 | 1205,
// 32 of 4096 x 86 149 | 500; 4096 x 97 takes the long form's 174.
constexpr int kNsShort = 96;
int ns_tiles(int64_t s) { return s > kNsShort ? 0 : (s > 64 ? 6 : (s > 32 ? 4 : 2)); }

// slices of the long side in the short form: at least 256 long (128 for wide Gram
// matrices, whose products take longer), at most 128
int ns_slices(int64_t l, int T)
{
    const int64_t len = T == 2 ? 256 : 128, n = (l + len - 1) / len;
    return (int)(n < 128 ? n : 128);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

int64_t ns_bytes(int64_t rows, int64_t cols)
{
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    if (s == 0)
        return 0;
    const int T = ns_tiles(s);
    if (T == 0)
        return up256(ns_long_bytes(ns_long(rows, cols, ns_parts(rows, cols))));
    const int64_t part = (int64_t)ns_slices(l, T) * tri(T) * 2048, f = 4LL * 256 * T * T + 8;  // (with two exponents)
    return ((part > f ? part : f) + 255) / 256 * 256;
}

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

// (every launch but k_ns_apply's, which goes in ranges, stays below 2^32 threads for the largest
// sides and list: k_ns_gram 4096 x 128 blocks of 256, the long form's kernels at most
// 2^22 of 256 per matrix)
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
    int64_t lsq = 0, ltile = 0, lsum = 0, lpoly = 0, lgram[2] = {0, 0}, lstep[2] = {0, 0};  // [narrow, wide]
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
                it.slices = ns_parts(e.rows, e.cols);
                const NsLong p = ns_long(e.rows, e.cols, it.slices);
                most(lsq, (int64_t)p.sqn);
                most(ltile, (p.sp / 64) * (p.lp / 64));
                most(lsum, (int64_t)p.tiles * (p.wide ? 32 : 16));
                most(lgram[p.wide], (int64_t)p.tiles * p.gram);
                most(lpoly, (int64_t)p.squares);
                most(lstep[p.wide], p.high * (p.lp / (p.wide ? 256 : 128)));
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
        const NsCoef coef{a, b, c, eps, steps};
        if (ns_fixed(a, b, c, steps))
            hipLaunchKernelGGL(k_ns_poly, dim3((unsigned)shorts), dim3(64 * kNsWaves), 0, s, t, w, coef);
        else
            hipLaunchKernelGGL(k_ns_poly64, dim3((unsigned)shorts), dim3(64 * kNsWaves), 0, s, t, w, coef);
        // (4096 matrices of 2^20 x 1 are 2^24 blocks, more than a grid's 2^32 threads)
        constexpr int64_t kMost = (int64_t)1 << 23;
        static_assert(grid_fits(kMost, 256), "blocks per launch");
        for (int64_t first = 0; first < applies; first += kMost)
            hipLaunchKernelGGL(k_ns_apply, dim3((unsigned)(applies - first < kMost ? applies - first : kMost)), dim3(256), 0, s,
                               table, apply_item, w, (int)first);
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
            if (lgram[0] > 0)
                hipLaunchKernelGGL(k_nsl_gram<1>, dim3((unsigned)lgram[0], y), dim3(512), 0, s, table, w, st & 1);
            if (lgram[1] > 0)
                hipLaunchKernelGGL(k_nsl_gram<2>, dim3((unsigned)lgram[1], y), dim3(512), 0, s, table, w, st & 1);
            hipLaunchKernelGGL(k_nsl_sum, dim3((unsigned)lsum, y), dim3(256), 0, s, table, w, two(ma - 2 * mx));
            hipLaunchKernelGGL(k_nsl_poly, dim3((unsigned)lpoly, y), dim3(512), 0, s, table, w, (float)(b * two(mb - ma)),
                               (float)(c * two(mb - 2 * ma)));
            const float fa = (float)(a * two(next - mx)), fs = two(next - mb - mx);
            if (lstep[0] > 0)
                hipLaunchKernelGGL(k_nsl_step<1>, dim3((unsigned)lstep[0], y), dim3(512), 0, s, table, w, fa, fs, st & 1);
            if (lstep[1] > 0)
                hipLaunchKernelGGL(k_nsl_step<2>, dim3((unsigned)lstep[1], y), dim3(512), 0, s, table, w, fa, fs, st & 1);
            mx = next;
        }
        hipLaunchKernelGGL(k_nsl_out, dim3((unsigned)ltile, y), dim3(256), 0, s, table, w, steps & 1, two(-mx));
    }
    return hipGetLastError();
}

}  // namespace owq
