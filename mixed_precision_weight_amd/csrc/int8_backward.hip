// int8_backward.hip -- backward of the 8-bit form's linear for weak-column tuning (gfx950).
//
//   dx[m][j]      = sum_i dy[m][i] W[i][j],  W = scale_i code_ij, the weak columns as they are
//   dw_weak[i][c] = sum_m dy[m][i] x[m][idx_c]
// (the rounding of the tokens to 8 bits passes gradients as the identity does).
//
// The dense part of dx runs on the fp16 matrix cores: dy_i scale_i is rounded to fp16
// after scaling each token by a power of two (11 bits of every term that is not below
// 2^-28 of the token's largest, and none overflows), the codes are exact in fp16. The
// weak parts multiply dy and x as they are.
#include "owq_int8.h"

namespace owq {

namespace {

typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f4_any8 __attribute__((ext_vector_type(4), aligned(4)));

struct BwdArgs8 {
    const int8_t* q;
    const float* s;
    const int32_t* idx;
    const uint16_t* ww;
    const uint16_t* x;
    const uint16_t* dy;
    uint16_t* dx;
    float* dw;
    uint16_t* g;     // [M][Np]
    float* unscale;  // [M]
    uint16_t* wwt;   // [kp][Np]
    uint16_t* xwt;   // [kp][Mp]
    float* part;     // [slices][M][kp]
    int32_t M, N, K, k, Np, Mp, kp, slices, mblocks;
};

// ------------------------------------------------------- the scaled gradients --

// One block per token: g = dy scale 2^e, the largest magnitude in [2^14, 2^15), zeros
// from N to Np.
__global__ __launch_bounds__(256) void k_int8_scale_dy(const BwdArgs8 a)
{
    __shared__ float red[4];
    const int tid = threadIdx.x, N = a.N;
    const int64_t m = blockIdx.x;
    const uint16_t* dy = a.dy + m * N;
    uint32_t top = 0;  // as bits: a NaN is the largest
    for (int p = tid * 8; p < N; p += 2048) {
        if (p + 8 <= N) {
            const u16x8_any v = *reinterpret_cast<const u16x8_any*>(dy + p);
            const f4_any8 s0 = *reinterpret_cast<const f4_any8*>(a.s + p), s1 = *reinterpret_cast<const f4_any8*>(a.s + p + 4);
#pragma unroll
            for (int e = 0; e < 8; e++)
                top = max(top, __builtin_bit_cast(uint32_t, h2f(v[e]) * (e < 4 ? s0[e] : s1[e - 4])) & 0x7fffffffu);
        } else {
            for (int e = p; e < N; e++)
                top = max(top, __builtin_bit_cast(uint32_t, h2f(dy[e]) * a.s[e]) & 0x7fffffffu);
        }
    }
    top = wave_max_u32(top);
    if ((tid & 63) == 0)
        red[tid >> 6] = __builtin_bit_cast(float, top);
    __syncthreads();
    for (int w = 0; w < 4; w++)
        top = max(top, __builtin_bit_cast(uint32_t, red[w]));
    // a row of zeros, and one that is not finite, stays as it is
    const int ex = (int)(top >> 23);
    const bool scaled = top != 0 && ex != 255;
    const float f = scaled ? __builtin_bit_cast(float, (uint32_t)min(max(268 - ex, 1), 254) << 23) : 1.0f;
    if (tid == 0)  // codes come as code 2^-9
        a.unscale[m] = 512.0f / f;
    uint16_t* g = a.g + m * a.Np;
    for (int p = tid * 8; p < a.Np; p += 2048) {  // Np is a multiple of 64
        uint32_t o[4];
        if (p + 8 <= N) {
            const u16x8_any v = *reinterpret_cast<const u16x8_any*>(dy + p);
            const f4_any8 s0 = *reinterpret_cast<const f4_any8*>(a.s + p), s1 = *reinterpret_cast<const f4_any8*>(a.s + p + 4);
#pragma unroll
            for (int e = 0; e < 4; e++)
                o[e] = f2h(h2f(v[2 * e]) * (e < 2 ? s0[2 * e] : s1[2 * e - 4]) * f) |
                       ((uint32_t)f2h(h2f(v[2 * e + 1]) * (e < 2 ? s0[2 * e + 1] : s1[2 * e - 3]) * f) << 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int n = p + 2 * e;
                o[e] = (n < N ? f2h(h2f(dy[n]) * a.s[n] * f) : 0u) |
                       ((uint32_t)(n + 1 < N ? f2h(h2f(dy[n + 1]) * a.s[n + 1] * f) : 0u) << 16);
            }
        }
        *reinterpret_cast<uint4*>(g + p) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The weak weights and the tokens' weak columns with the long side contiguous, padded
// with zeros: wwt[c][i], xwt[c][m].
__global__ __launch_bounds__(256) void k_int8_weak_t(const BwdArgs8 a)
{
    const int64_t nw = a.dx ? (int64_t)a.kp * a.Np : 0, nx = a.dw ? (int64_t)a.kp * a.Mp : 0;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < nw + nx; e += (int64_t)gridDim.x * 256) {
        if (e < nw) {
            const int c = (int)(e / a.Np), i = (int)(e % a.Np);
            a.wwt[e] = c < a.k && i < a.N ? a.ww[(int64_t)i * a.k + c] : (uint16_t)0;
        } else {
            const int c = (int)((e - nw) / a.Mp), m = (int)((e - nw) % a.Mp);
            const int j = c < a.k ? a.idx[c] : -1;
            a.xwt[e - nw] = m < a.M && j >= 0 && j < a.K ? a.x[(int64_t)m * a.K + j] : (uint16_t)0;
        }
    }
}

// ------------------------------------------------------------------ weak sums --

constexpr int kWeakWaves = 8;

// The waves' 32 x 32 sums added in LDS in a fixed order; element r of lane l afterwards
// in sum[r * 64 + l].
__device__ __forceinline__ void add_waves(float (*red)[16 * 64], const i8_f16v& acc, int wave, int lane)
{
#pragma unroll
    for (int r = 0; r < 16; r++)
        red[wave][r * 64 + lane] = acc[r];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * 64; e += 64 * kWeakWaves) {
        float v = red[0][e];
        for (int w = 1; w < kWeakWaves; w++)
            v += red[w][e];
        red[0][e] = v;
    }
    __syncthreads();
}

// dy w_weak: 32 tokens x 32 weak columns over a slice of the rows
__global__ __launch_bounds__(64 * kWeakWaves) void k_int8_weak_dx(const BwdArgs8 a)
{
    __shared__ float red[kWeakWaves][16 * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int m0 = (int)blockIdx.x * 32, c0 = (int)blockIdx.y * 32, sl = blockIdx.z;
    const int steps = a.Np >> 4, per = (steps + a.slices - 1) / a.slices;
    const int s0 = sl * per, s1 = min(steps, s0 + per);
    const uint16_t* dy = a.dy + (int64_t)min(m0 + l32, a.M - 1) * a.N;
    const uint16_t* w = a.wwt + (int64_t)(c0 + l32) * a.Np;
    i8_f16v acc;
#pragma unroll
    for (int r = 0; r < 16; r++)
        acc[r] = 0.0f;
    for (int st = s0 + wave; st < s1; st += kWeakWaves) {
        const int n = st * 16 + 8 * h;
        half8_t av;
        if (n + 8 <= a.N) {
            av = __builtin_bit_cast(half8_t, *reinterpret_cast<const u16x8_any*>(dy + n));
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                av[e] = __builtin_bit_cast(_Float16, n + e < a.N ? dy[n + e] : (uint16_t)0);
        }
        const half8_t bv = *reinterpret_cast<const half8_t*>(w + n);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(av, bv, acc, 0, 0, 0);
    }
    add_waves(red, acc, wave, lane);
    for (int e = threadIdx.x; e < 1024; e += 64 * kWeakWaves) {
        const int r = e >> 6, l = e & 63;
        const int m = m0 + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), c = c0 + (l & 31);
        if (m < a.M)
            a.part[((int64_t)sl * a.M + m) * a.kp + c] = red[0][e];
    }
}

// The slices' sums into dx's weak columns
__global__ __launch_bounds__(256) void k_int8_weak_put(const BwdArgs8 a)
{
    const int64_t n = (int64_t)a.M * a.k;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t m = e / a.k;
        const int c = (int)(e % a.k), j = a.idx[c];
        float v = 0.0f;
        for (int sl = 0; sl < a.slices; sl++)
            v += a.part[((int64_t)sl * a.M + m) * a.kp + c];
        if (j >= 0 && j < a.K)
            a.dx[m * a.K + j] = f2h(v);
    }
}

// dy^T x_weak: 32 rows x 32 weak columns over all tokens
__global__ __launch_bounds__(64 * kWeakWaves) void k_int8_weak_dw(const BwdArgs8 a)
{
    __shared__ float red[kWeakWaves][16 * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int i0 = (int)blockIdx.x * 32, c0 = (int)blockIdx.y * 32;
    const uint16_t* dy = a.dy + min(i0 + l32, a.N - 1);
    const uint16_t* xw = a.xwt + (int64_t)(c0 + l32) * a.Mp;
    i8_f16v acc;
#pragma unroll
    for (int r = 0; r < 16; r++)
        acc[r] = 0.0f;
    for (int st = wave; st < a.Mp >> 4; st += kWeakWaves) {
        const int m = st * 16 + 8 * h;
        half8_t av;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint16_t v = dy[(int64_t)min(m + e, a.M - 1) * a.N];
            av[e] = __builtin_bit_cast(_Float16, m + e < a.M ? v : (uint16_t)0);
        }
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(av, *reinterpret_cast<const half8_t*>(xw + m), acc, 0, 0, 0);
    }
    add_waves(red, acc, wave, lane);
    for (int e = threadIdx.x; e < 1024; e += 64 * kWeakWaves) {
        const int r = e >> 6, l = e & 63;
        const int i = i0 + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), c = c0 + (l & 31);
        if (i < a.N && c < a.k)
            a.dw[(int64_t)i * a.k + c] = red[0][e];
    }
}

// ------------------------------------------------------------- dense part of dx --

template <int FM, int FN, int WM, int WN>
struct TileDx {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BM = 32 * FM * WM, BJ = 32 * FN * WN;
    static constexpr int DA = BM * 128 / 16 / NT;
    static constexpr int QUADS = BJ / 4;           // 4-column groups
    static constexpr int GROUPS = QUADS * 8 / NT;  // (4 columns, 8 rows) pieces per thread and stage
    static_assert(DA * NT * 16 == BM * 128 && GROUPS * NT == QUADS * 8, "a stage must split evenly over the threads");
};

// slot of piece p (8 values of the contraction) of row r of a stage: reads take 32
// consecutive rows, the writes of codes every fourth row
__device__ __forceinline__ int dx_slot(int r, int p) { return p ^ ((r ^ (r >> 3)) & 7); }

// BM tokens x BJ columns per block; the contraction runs over the layer's rows, 64 at a
// time: g by direct-to-LDS loads, the codes through registers, where 8 rows of 4 columns
// are turned round and widened (a byte pair becomes two fp16 subnormals, one fused
// multiply-add makes them code 2^-9).
template <int FM, int FN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void k_int8_dx(const BwdArgs8 a)
{
    using T = TileDx<FM, FN, WM, WN>;
    constexpr int BM = T::BM, BJ = T::BJ;
    __shared__ __attribute__((aligned(1024))) char s0[(BM + BJ) * 128];
    __shared__ __attribute__((aligned(1024))) char s1[(BM + BJ) * 128];
    const int M = a.M, N = a.N, K = a.K, Np = a.Np;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int l32 = lane & 31, h = lane >> 5;
    const int m0 = ((int)blockIdx.x % a.mblocks) * BM, j0 = ((int)blockIdx.x / a.mblocks) * BJ;
    const int mv = min(BM, M - m0);
    const __amdgpu_buffer_rsrc_t gr = bytes_rsrc(a.g + (int64_t)m0 * Np, (int64_t)mv * Np * 2);
    int gsrc[T::DA];
#pragma unroll
    for (int t = 0; t < T::DA; t++) {
        const int u = (wave * T::DA + t) * 64 + lane, row = u >> 3;
        gsrc[t] = min(row, mv - 1) * Np * 2 + dx_slot(row, u & 7) * 16;
    }
    auto dma = [&](int c, char* stage) {
#pragma unroll
        for (int t = 0; t < T::DA; t++)
            dma16_lds(gr, stage + (wave * T::DA + t) * 1024, gsrc[t] + c * 128);
    };
    // this thread's pieces: 4 columns 4 q4, rows 8 o .. 8 o + 7 of the stage
    auto load = [&](int c, uint32_t (&v)[T::GROUPS][8]) {
        const int64_t i0 = (int64_t)c * 64;
        const __amdgpu_buffer_rsrc_t qr =
            bytes_rsrc(a.q + (i0 < N ? i0 * K + j0 : 0), i0 < N ? (int64_t)min(64, (int)(N - i0)) * K - j0 : 0);
#pragma unroll
        for (int t = 0; t < T::GROUPS; t++) {
            const int u = t * T::NT + tid, q4 = u % T::QUADS, o = u / T::QUADS;
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[t][e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(qr, (8 * o + e) * K + 4 * q4, 0, 0);
        }
    };
    auto put = [&](const uint32_t (&v)[T::GROUPS][8], char* stage) {
        const half2_t mul = {(_Float16)32768.0f, (_Float16)32768.0f}, add = {(_Float16)-0.25f, (_Float16)-0.25f};
#pragma unroll
        for (int t = 0; t < T::GROUPS; t++) {
            const int u = t * T::NT + tid, q4 = u % T::QUADS, o = u / T::QUADS;
            uint32_t d[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                d[e] = v[t][e] ^ 0x80808080u;  // code + 128
#pragma unroll
            for (int b = 0; b < 4; b++) {
                uint32_t w[4];
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    const uint32_t two = __builtin_amdgcn_perm(d[2 * p + 1], d[2 * p],
                                                               0x0c000c00u | (uint32_t)((4 + b) << 16) | (uint32_t)b);
                    w[p] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, two), mul, add));
                }
                const int row = 4 * q4 + b;
                *reinterpret_cast<uint4*>(stage + (BM + row) * 128 + dx_slot(row, o) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    i8_f16v acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[i][f][r] = 0.0f;
    const int chunks = Np >> 6;
    uint32_t cv[T::GROUPS][8];
    auto step = [&](int c, const char* cur, char* nxt) {
        stage_barrier<0>();
        if (c + 1 < chunks) {
            dma(c + 1, nxt);
            put(cv, nxt);
            load(c + 2, cv);
        }
        if (c < chunks) {
#pragma unroll
            for (int st = 0; st < 4; st++) {
                half8_t av[FM], bv[FN];
#pragma unroll
                for (int i = 0; i < FM; i++) {
                    const int row = wm * 32 * FM + 32 * i + l32;
                    av[i] = *reinterpret_cast<const half8_t*>(cur + row * 128 + dx_slot(row, st * 2 + h) * 16);
                }
#pragma unroll
                for (int f = 0; f < FN; f++) {
                    const int row = wn * 32 * FN + 32 * f + l32;
                    bv[f] = *reinterpret_cast<const half8_t*>(cur + (BM + row) * 128 + dx_slot(row, st * 2 + h) * 16);
                }
#pragma unroll
                for (int i = 0; i < FM; i++)
#pragma unroll
                    for (int f = 0; f < FN; f++)
                        acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[i], bv[f], acc[i][f], 0, 0, 0);
            }
        }
    };
    load(0, cv);
    dma(0, s0);
    put(cv, s0);
    load(1, cv);
    for (int c = 0; c < chunks; c += 2) {
        step(c, s0, s1);
        step(c + 1, s1, s0);
    }
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int mb = wm * 32 * FM + 32 * i;
        float un[16];
#pragma unroll
        for (int r = 0; r < 16; r++)
            un[r] = a.unscale[m0 + min(mb + 8 * (r >> 2) + 4 * h + (r & 3), mv - 1)];
#pragma unroll
        for (int f = 0; f < FN; f++) {
            const int j = j0 + wn * 32 * FN + 32 * f + l32;
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int m = m0 + mb + 8 * (r >> 2) + 4 * h + (r & 3);
                if (m < M && j < K)
                    a.dx[(int64_t)m * K + j] = f2h(acc[i][f][r] * un[r]);
            }
        }
    }
}

template <int FM, int FN, int WM, int WN>
hipError_t launch_dx(BwdArgs8 a, hipStream_t s)
{
    using T = TileDx<FM, FN, WM, WN>;
    a.mblocks = (a.M + T::BM - 1) / T::BM;
    const int64_t blocks = (int64_t)a.mblocks * ((a.K + T::BJ - 1) / T::BJ);
    hipLaunchKernelGGL((k_int8_dx<FM, FN, WM, WN>), dim3((unsigned)blocks), dim3(T::NT), 0, s, a);
    return hipGetLastError();
}

constexpr int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace

Int8BwdPlan int8_bwd_plan(int64_t N, int64_t K, int32_t k, int64_t M)
{
    (void)K;
    Int8BwdPlan p{};
    p.Np = up(N, 64);
    p.Mp = up(M, 16);
    p.kp = up(k, 32);
    // slices of the weak columns' sums: enough blocks, at least 512 rows each
    const int64_t tiles = (M + 31) / 32 * (p.kp / 32 > 0 ? p.kp / 32 : 1);
    int64_t sl = (512 + tiles - 1) / tiles;
    sl = sl < p.Np / 512 ? sl : p.Np / 512;
    p.slices = sl < 1 ? 1 : sl;
    size_t off = (size_t)up(2 * M * p.Np, 256);
    p.off_un = off;
    off += (size_t)up(4 * M, 256);
    p.off_wwt = off;
    off += (size_t)up(2 * p.kp * p.Np, 256);
    p.off_xwt = off;
    off += (size_t)up(2 * p.kp * p.Mp, 256);
    p.off_part = off;
    off += (size_t)up(4 * p.slices * M * p.kp, 256);
    p.total = off;
    return p;
}

hipError_t launch_linear_int8_backward(const Int8Desc& d, const uint16_t* dy, int64_t M, uint16_t* dx, float* dw,
                                       void* ws, const Int8BwdPlan& p, hipStream_t s)
{
    char* const w = static_cast<char*>(ws);
    const BwdArgs8 a{d.q, d.s, d.idx, d.ww, d.x, dy, dx, d.k > 0 ? dw : nullptr, reinterpret_cast<uint16_t*>(w),
                     reinterpret_cast<float*>(w + p.off_un), reinterpret_cast<uint16_t*>(w + p.off_wwt),
                     reinterpret_cast<uint16_t*>(w + p.off_xwt), reinterpret_cast<float*>(w + p.off_part), (int32_t)M,
                     (int32_t)d.N, (int32_t)d.K, d.k, (int32_t)p.Np, (int32_t)p.Mp, (int32_t)p.kp, (int32_t)p.slices, 1};
    if (d.k > 0) {
        const int64_t n = (a.dx ? p.kp * p.Np : 0) + (a.dw ? p.kp * p.Mp : 0);
        const int64_t blocks = (n + 255) / 256;
        hipLaunchKernelGGL(k_int8_weak_t, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s, a);
    }
    if (a.dw)
        hipLaunchKernelGGL(k_int8_weak_dw, dim3((unsigned)((d.N + 31) / 32), (unsigned)(p.kp / 32)), dim3(64 * kWeakWaves), 0,
                           s, a);
    if (dx) {
        if (d.k > 0)
            hipLaunchKernelGGL(k_int8_weak_dx, dim3((unsigned)((M + 31) / 32), (unsigned)(p.kp / 32), (unsigned)p.slices),
                               dim3(64 * kWeakWaves), 0, s, a);
        hipLaunchKernelGGL(k_int8_scale_dy, dim3((unsigned)M), dim3(256), 0, s, a);
        const hipError_t e = M > 128 ? launch_dx<4, 2, 2, 4>(a, s) : launch_dx<1, 1, 1, 4>(a, s);
        if (e != hipSuccess)
            return e;
        if (d.k > 0) {
            const int64_t blocks = (M * d.k + 255) / 256;
            hipLaunchKernelGGL(k_int8_weak_put, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s, a);
        }
    }
    return hipGetLastError();
}

}  // namespace owq
