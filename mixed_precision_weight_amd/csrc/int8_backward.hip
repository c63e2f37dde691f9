// int8_backward.hip -- backward of the integer form's linear for weak-column tuning (gfx950).
//
//   dx[m][j]      = sum_i dy[m][i] W[i][j],  W = scale_i code_ij, the weak columns as they are
//   dw_weak[i][c] = sum_m dy[m][i] x[m][idx_c]
// (the rounding of the tokens to 8 bits passes gradients as the identity does).
//
// The dense part of dx runs on the fp16 matrix cores: dy_i scale_i is kept as a pair of fp16
// values, itself rounded and what that left, after scaling each token by a power of two (22
// bits, and none overflows; what lies below 2^-17 of the token's largest is held to 2^-39 of
// it), the codes are exact in fp16: two products for one, so that dx is the fp32 sum rounded
// once: 2.1e-4 against 64 bits, the fp16 result's own rounding. (One product with eleven bits of
// dy_i scale_i takes 190 us instead of 340 for 2048 tokens, 11008 x 4096, and gives 2.9e-4.)
// The weak parts multiply dy and x as they are.
#include "owq_int8.h"

namespace owq {

namespace {

typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f4_any8 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kDxTokens = 128, kDxCols = 128;  // of a tile
constexpr int kDxRows = 32;                    // of the layer per stage
constexpr int kDxPlane = kDxTokens * 64;       // high halves of a stage's g; the low ones follow
constexpr int kDxStage = 2 * kDxPlane + kDxRows * kDxCols;
constexpr int kDxLoads = 4 + 1;  // per wave and stage, of g and of the codes

struct BwdArgs8 {
    const int8_t* q;
    const float* s;
    const int32_t* idx;
    const uint16_t* ww;
    const uint16_t* x;
    const uint16_t* dy;
    uint16_t* dx;
    float* dw;
    uint16_t* g;     // [M][Np] pairs in panels of kDxTokens: a stage's high halves, its low halves
    float* unscale;  // [M]
    uint16_t* wwt;   // [kp][Np]
    uint16_t* xwt;   // [kp][Mp]
    float* part;     // [slices][M][kp]
    i8_f4v* sums;    // [split][tile][wave][16][lane], where splits > 1
    int32_t M, N, K, k, Np, Mp, kp, slices, mblocks, splits;
};

// ------------------------------------------------------- the scaled gradients --

// Two values as a pair each: the words of the high and of the low halves
__device__ __forceinline__ void dx_pairs(float a, float b, uint32_t& hi, uint32_t& lo)
{
    const uint16_t ha = f2h(a), hb = f2h(b);
    hi = ha | ((uint32_t)hb << 16);
    lo = f2h(a - h2f(ha)) | ((uint32_t)f2h(b - h2f(hb)) << 16);
}

// The first blocks: one per token, g = dy scale 2^e, the largest magnitude in [2^14, 2^15),
// zeros from N to Np. The others: the weak weights and the tokens' weak columns with the
// long side contiguous, padded with zeros: wwt[c][i], xwt[c][m]. Bound by memory: 2048 tokens
// of 11008, 45 MB read twice, the second time from L2 or the memory's cache, and 90 MB written in 33
// us (4.1 TB/s).
__global__ __launch_bounds__(256) void k_int8_prepare(const BwdArgs8 a, int tokens)
{
    __shared__ float red[4];
    const int tid = threadIdx.x, N = a.N;
    if ((int)blockIdx.x >= tokens) {
        const int64_t nw = a.dx ? (int64_t)a.kp * a.Np : 0, nx = a.dw ? (int64_t)a.kp * a.Mp : 0;
        const int64_t step = (int64_t)((int)gridDim.x - tokens) * 256;
        for (int64_t e = (int64_t)((int)blockIdx.x - tokens) * 256 + tid; e < nw + nx; e += step) {
            if (e < nw) {
                const int c = (int)(e / a.Np), i = (int)(e % a.Np);
                a.wwt[e] = c < a.k && i < N ? a.ww[(int64_t)i * a.k + c] : (uint16_t)0;
            } else {
                const int c = (int)((e - nw) / a.Mp), m = (int)((e - nw) % a.Mp);
                const int j = c < a.k ? a.idx[c] : -1;
                a.xwt[e - nw] = m < a.M && j >= 0 && j < a.K ? a.x[(int64_t)m * a.K + j] : (uint16_t)0;
            }
        }
        return;
    }
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
    char* const g = reinterpret_cast<char*>(a.g);
    for (int p = tid * 8; p < a.Np; p += 2048) {  // Np is a multiple of 32
        uint32_t o[4], r[4];
        if (p + 8 <= N) {
            const u16x8_any v = *reinterpret_cast<const u16x8_any*>(dy + p);
            const f4_any8 s0 = *reinterpret_cast<const f4_any8*>(a.s + p), s1 = *reinterpret_cast<const f4_any8*>(a.s + p + 4);
#pragma unroll
            for (int e = 0; e < 4; e++)
                dx_pairs(h2f(v[2 * e]) * (e < 2 ? s0[2 * e] : s1[2 * e - 4]) * f,
                         h2f(v[2 * e + 1]) * (e < 2 ? s0[2 * e + 1] : s1[2 * e - 3]) * f, o[e], r[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int n = p + 2 * e;
                dx_pairs(n < N ? h2f(dy[n]) * a.s[n] * f : 0.0f, n + 1 < N ? h2f(dy[n + 1]) * a.s[n + 1] * f : 0.0f, o[e], r[e]);
            }
        }
        // (a panel's stages of 32 rows, two planes each)
        char* const at = g + m / kDxTokens * kDxTokens * 4 * a.Np + (int64_t)(p / kDxRows) * (2 * kDxPlane) + m % kDxTokens * 64 +
                         p % kDxRows * 2;
        *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(at + kDxPlane) = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// ------------------------------------------------------------------ weak sums --

constexpr int kWeakParts = 8;  // of a sum: a wave each in k_int8_weak_sums, two per wave in k_int8_dx

typedef float* WeakLds[kWeakParts];

// A part's 32 x 32 sums to LDS
__device__ __forceinline__ void weak_part(const WeakLds& red, const i8_f16v& acc, int part, int lane)
{
#pragma unroll
    for (int w = 0; w < kWeakParts; w++)
        if (w == part)
#pragma unroll
            for (int r = 0; r < 16; r++)
                red[w][r * 64 + lane] = acc[r];
}

// and the parts' in a fixed order, whoever made them; element r of lane l afterwards in
// red[0][r * 64 + l].
template <int W>
__device__ __forceinline__ void add_parts(const WeakLds& red)
{
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * 64; e += 64 * W) {
        float v = red[0][e];
#pragma unroll
        for (int w = 1; w < kWeakParts; w++)
            v += red[w][e];
        red[0][e] = v;
    }
    __syncthreads();
}

// dy w_weak: 32 tokens x 32 weak columns over a slice of the rows
template <int W>
__device__ __forceinline__ void weak_dx(const BwdArgs8& a, const WeakLds& red, int block, int cb)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int c0 = cb * 32, sl = block % a.slices, m0 = block / a.slices * 32;
    const int steps = a.Np >> 4, per = (steps + a.slices - 1) / a.slices;
    const int s0 = sl * per, s1 = min(steps, s0 + per);
    const uint16_t* dy = a.dy + (int64_t)min(m0 + l32, a.M - 1) * a.N;
    const uint16_t* w = a.wwt + (int64_t)(c0 + l32) * a.Np;
#pragma unroll 1
    for (int part = wave; part < kWeakParts; part += W) {
        i8_f16v acc;
#pragma unroll
        for (int r = 0; r < 16; r++)
            acc[r] = 0.0f;
        for (int st = s0 + part; st < s1; st += kWeakParts) {
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
        weak_part(red, acc, part, lane);
    }
    add_parts<W>(red);
    for (int e = threadIdx.x; e < 1024; e += 64 * W) {
        const int r = e >> 6, l = e & 63;
        const int m = m0 + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), c = c0 + (l & 31);
        if (m < a.M)
            a.part[((int64_t)sl * a.M + m) * a.kp + c] = red[0][e];
    }
}

// dy^T x_weak: 32 rows x 32 weak columns over all tokens
template <int W>
__device__ __forceinline__ void weak_dw(const BwdArgs8& a, const WeakLds& red, int block, int cb)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int i0 = block * 32, c0 = cb * 32;
    const uint16_t* dy = a.dy + min(i0 + l32, a.N - 1);
    const uint16_t* xw = a.xwt + (int64_t)(c0 + l32) * a.Mp;
#pragma unroll 1
    for (int part = wave; part < kWeakParts; part += W) {
        i8_f16v acc;
#pragma unroll
        for (int r = 0; r < 16; r++)
            acc[r] = 0.0f;
        for (int st = part; st < a.Mp >> 4; st += kWeakParts) {
            const int m = st * 16 + 8 * h;
            half8_t av;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const uint16_t v = dy[(int64_t)min(m + e, a.M - 1) * a.N];
                av[e] = __builtin_bit_cast(_Float16, m + e < a.M ? v : (uint16_t)0);
            }
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(av, *reinterpret_cast<const half8_t*>(xw + m), acc, 0, 0, 0);
        }
        weak_part(red, acc, part, lane);
    }
    add_parts<W>(red);
    for (int e = threadIdx.x; e < 1024; e += 64 * W) {
        const int r = e >> 6, l = e & 63;
        const int i = i0 + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), c = c0 + (l & 31);
        if (i < a.N && c < a.k)
            a.dw[(int64_t)i * a.k + c] = red[0][e];
    }
}

// Both sums over dy in one launch: the first `dws` blocks the weights', the others the tokens'.
// 2048 tokens, 11008 rows, 32 weak columns: 31 us for 45 MB of dy that both read, at 2.9 TB/s;
// the blocks take two rounds. (Four steps of loads in flight instead of one: no change.)
__global__ __launch_bounds__(64 * kWeakParts) void k_int8_weak_sums(const BwdArgs8 a, int dws)
{
    __shared__ float lds[kWeakParts][16 * 64];
    const WeakLds red = {lds[0], lds[1], lds[2], lds[3], lds[4], lds[5], lds[6], lds[7]};
    if ((int)blockIdx.x < dws)
        weak_dw<kWeakParts>(a, red, xcd_place((int)blockIdx.x, dws), (int)blockIdx.y);  // neighbours share lines of dy: 34 -> 31 us
    else
        weak_dx<kWeakParts>(a, red, (int)blockIdx.x - dws, (int)blockIdx.y);
}

// The weak columns among columns j0 .. j0 + cols - 1: places first .. last - 1 of idx. at: of
// up to 64 weak columns, one per lane (one load; a search has a latency per halving).
struct WeakRange {
    int first, last, at;
};
__device__ __forceinline__ WeakRange weak_range(const BwdArgs8& a, int j0, int cols)
{
    WeakRange r{0, 0, 0};
    const int end = min(j0 + cols, a.K);
    if (a.k <= 64) {
        const int lane = threadIdx.x & 63;
        r.at = lane < a.k ? a.idx[lane] : a.K;
        r.first = __builtin_popcountll(__builtin_amdgcn_ballot_w64(r.at < j0));
        r.last = __builtin_popcountll(__builtin_amdgcn_ballot_w64(r.at < end));
        return r;
    }
    auto below = [&](int j) {  // (they ascend)
        int c = 0;
        for (int hi = a.k; c < hi;) {
            const int mid = (c + hi) >> 1;
            if (__builtin_amdgcn_readfirstlane(a.idx[mid]) < j)
                c = mid + 1;
            else
                hi = mid;
        }
        return c;
    };
    r.first = below(j0);
    r.last = r.first;
    while (r.last < a.k && __builtin_amdgcn_readfirstlane(a.idx[r.last]) < end)
        r.last++;
    return r;
}

// dx's weak columns of a range, of tokens m0 .. m0 + n - 1, from the slices' sums, by one wave,
// which has written other values there: over those.
__device__ __forceinline__ void weak_put(const BwdArgs8& a, const WeakRange& r, int m0, int n)
{
    if (r.first == r.last)
        return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int c = r.first; c < r.last; c++) {
        const int j = __builtin_amdgcn_readfirstlane(a.k <= 64 ? __builtin_amdgcn_readlane(r.at, c) : a.idx[c]);
        for (int t = threadIdx.x & 63; t < n; t += 64) {
            float v = 0.0f;
            for (int sl = 0; sl < a.slices; sl++)
                v += a.part[((int64_t)sl * a.M + m0 + t) * a.kp + c];
            a.dx[(int64_t)(m0 + t) * a.K + j] = f2h(v);
        }
    }
}

// ------------------------------------------------------------- dense part of dx --

typedef int i32x2 __attribute__((ext_vector_type(2)));

// 128 tokens x 128 columns per block of 4 waves (64 x 64 each), two blocks per CU, which
// run at their own pace; the contraction runs over the layer's rows, 32 at a time, in a
// ring of four stages that is filled three ahead by direct-to-LDS loads: g (panels of 128
// tokens, 64 bytes of each together, high and low halves apart) as in the forward product,
// the codes as they lie. ds_read_tr turns 8 rows of the codes round on the way to the
// registers, where they become fp16: a byte pair is read as two fp16 subnormals, which one
// fused multiply-add makes code 2^-9, exactly. (Turning the codes round on the way into LDS
// instead needs registers and eight-way bank conflicts: 315 us for 2048 tokens, 11008 x
// 4096.) The columns are the matrix instruction's A, so that a lane ends with four
// consecutive columns of one token. Blocks past the `blocks` of the product (where k_int8_dx_sum
// adds the product's parts and puts the weak columns in) make the weak sums beside it. 2048
// tokens, 11008 x 4096: 336 us, 1.1 PFLOP/s of both halves' products, matrix cores busy 79 % (the
// library's fp16 product reaches 1.4 at 8192^3; the card's power holds the clock). Strips of 2, 4 or 8
// token panels per XCD, which share more of g: no change.
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_int8_dx(const BwdArgs8 a, int blocks, int dws)
{
    __shared__ __attribute__((aligned(1024))) char s0[kDxStage];
    __shared__ __attribute__((aligned(1024))) char s1[kDxStage];
    __shared__ __attribute__((aligned(1024))) char s2[kDxStage];
    __shared__ __attribute__((aligned(1024))) char s3[kDxStage];  // (four stages of two blocks are a CU's whole LDS)
    constexpr int FM = 2, FJ = 2;
    const int M = a.M, N = a.N, K = a.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wj = wave >> 1;
    const int l32 = lane & 31, h = lane >> 5;
    if ((int)blockIdx.x >= blocks) {
        auto half = [](char* p, int i) { return reinterpret_cast<float*>(p) + 1024 * i; };
        const WeakLds red = {half(s0, 0), half(s0, 1), half(s1, 0), half(s1, 1), half(s2, 0), half(s2, 1), half(s3, 0), half(s3, 1)};
        const int e = (int)blockIdx.x - blocks, cbs = (a.k + 31) >> 5, block = e / cbs;
        if (block < dws)
            weak_dw<4>(a, red, block, e % cbs);
        else
            weak_dx<4>(a, red, block - dws, e % cbs);
        return;
    }
    const int place = xcd_place((int)blockIdx.x, blocks), tiles = blocks / a.splits;
    const int tile = place % tiles, split = place / tiles;
    const int m0 = (tile % a.mblocks) * kDxTokens, j0 = (tile / a.mblocks) * kDxCols;
    const __amdgpu_buffer_rsrc_t gr = uniform_rsrc(a.g + (int64_t)2 * m0 * a.Np, (int64_t)4 * kDxTokens * a.Np);
    int gsrc[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const int u = (wave * 2 + t) * 64 + lane;
        gsrc[t] = stage_row(u) * 64 + stage_piece(u) * 16;
    }
    // codes: 128 bytes per row; the 16-byte piece p of row r in slot p ^ (r % 8)
    const int qrow = tid >> 3, qcol = ((tid & 7) ^ (qrow & 7)) * 16;
    const int qsrc = j0 + qcol < K ? qrow * K + qcol : kDeadLoad;
    const int all = a.Np / kDxRows;
    const int c0 = (int)((int64_t)all * split / a.splits), c1 = (int)((int64_t)all * (split + 1) / a.splits);
    auto dma = [&](int c, char* stage) {
        const int dead = c < c1 ? 0 : kDeadLoad;
        const int i0 = min(c, c1 - 1) * kDxRows;  // (Np is N rounded up: the last stage has a row)
        const __amdgpu_buffer_rsrc_t qr = uniform_rsrc(a.q + (int64_t)i0 * K + j0, (int64_t)min(kDxRows, N - i0) * K - j0);
#pragma unroll
        for (int t = 0; t < 4; t++)
            dma16_lds(gr, stage + (t >> 1) * kDxPlane + (wave * 2 + (t & 1)) * 1024,
                      gsrc[t & 1] + (t >> 1) * kDxPlane + (i0 * (4 * kDxTokens) | dead));
        dma16_lds(qr, stage + 2 * kDxPlane + wave * 1024, qsrc | dead);
    };
    i8_f16v acc[FM][FJ];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int f = 0; f < FJ; f++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[i][f][r] = 0.0f;
    // g: this lane's pieces h and 2 + h of its tokens. Codes: in a group of 16 lanes, lane i
    // names 8 bytes of row i / 2, columns 8 (i % 2), and gets column i of the 8 rows.
    const int p0 = wm * FM * 2048 + stage_at(l32, h), p1 = wm * FM * 2048 + stage_at(l32, 2 + h);
    int qa[2][FJ];
#pragma unroll
    for (int st = 0; st < 2; st++)
#pragma unroll
        for (int f = 0; f < FJ; f++) {
            const int r = 16 * st + 8 * h + ((lane & 15) >> 1), piece = (wj * FJ + f) * 2 + ((lane >> 4) & 1);
            qa[st][f] = 2 * kDxPlane + r * kDxCols + ((piece ^ (r & 7)) * 16) + (lane & 1) * 8;
        }
    // codes as read (two 16-row steps of a stage) and as fp16, g: the codes are read two
    // steps ahead of their products and widened one ahead, g is read one ahead
    i32x2 raw[2][FJ];
    half8_t cv[2][FJ], gv[2][2][FM];  // [step][high, low]
    auto read_codes = [&](const char* stage, int st) {
#pragma unroll
        for (int f = 0; f < FJ; f++)
            raw[st][f] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(stage + qa[st][f]));
    };
    auto read_g = [&](const char* stage, int st) {
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
            for (int i = 0; i < FM; i++)
                gv[st][e][i] = *reinterpret_cast<const half8_t*>(stage + e * kDxPlane + (st ? p1 : p0) + i * 2048);
    };
    const half2_t mul = {(_Float16)32768.0f, (_Float16)32768.0f}, add = {(_Float16)-0.25f, (_Float16)-0.25f};
    auto widen = [&](int st) {
#pragma unroll
        for (int f = 0; f < FJ; f++) {
            const uint32_t d[2] = {(uint32_t)raw[st][f].x ^ 0x80808080u, (uint32_t)raw[st][f].y ^ 0x80808080u};  // code + 128
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t two = __builtin_amdgcn_perm(0u, d[e >> 1], e & 1 ? 0x0c030c02u : 0x0c010c00u);
                w[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, two), mul, add));
            }
            cv[st][f] = __builtin_bit_cast(half8_t, make_uint4(w[0], w[1], w[2], w[3]));
        }
    };
    auto product = [&](int st) {
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int f = 0; f < FJ; f++)
                    acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(cv[st][f], gv[st][e][i], acc[i][f], 0, 0, 0);
        // the reads and the widening between the products
#pragma unroll
        for (int i = 0; i < 2 * FM * FJ; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        }
    };
    // products of the stage in cur, and the reads ahead from next
    auto stage = [&](const char* cur, const char* next) {
        read_codes(next, 0);
        read_g(cur, 1);
        widen(1);
        product(0);
        read_codes(next, 1);
        read_g(next, 0);
        widen(0);
        product(1);
    };
    // c in cur and c + 1 in next, whole; c + 3 goes where c - 1 was
    auto step = [&](int c, const char* cur, const char* next, char* fill) {
        stage_barrier<kDxLoads, 15>();
        dma(c + 3, fill);
        if (c < c1) {
            stage(cur, next);
            // its reads are done before this wave lets it be overwritten
#pragma unroll
            for (int i = 0; i < FM; i++)
                asm volatile("" ::"v"(gv[1][0][i]), "v"(gv[1][1][i]));
        }
    };
    dma(c0, s0);
    dma(c0 + 1, s1);
    dma(c0 + 2, s2);
    stage_barrier<0>();
    read_codes(s0, 0);
    read_codes(s0, 1);
    read_g(s0, 0);
    widen(0);
    for (int c = c0; c < c1; c += 4) {  // (a stage past c1 holds zeros)
        step(c, s0, s1, s3);
        step(c + 1, s1, s2, s0);
        step(c + 2, s2, s3, s1);
        step(c + 3, s3, s0, s2);
    }
#pragma unroll
    for (int f = 0; f < FJ; f++)
        asm volatile("" ::"v"(raw[0][f]), "v"(raw[1][f]));
    stage_barrier<0>();  // the loads past the end have written their zeros
    if (a.splits > 1) {
        i8_f4v* const sums = a.sums + ((int64_t)place * 4 + wave) * (FM * FJ * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int f = 0; f < FJ; f++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    sums[((i * FJ + f) * 4 + q) * 64] =
                        i8_f4v{acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3]};
        return;
    }
    const WeakRange range = weak_range(a, j0 + wj * 64, 64);
    // 32 tokens x 64 columns of the wave at a time: token t's piece p of 8 columns in slot
    // p ^ (t % 8) of its 128 bytes
    char* const mine = (wave < 2 ? s0 : s1) + (wave & 1) * 4096;
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const float sc = a.unscale[min(m0 + wm * 32 * FM + 32 * i + l32, M - 1)];
#pragma unroll
        for (int f = 0; f < FJ; f++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const i8_f16v& o = acc[i][f];
                *reinterpret_cast<uint2*>(mine + l32 * 128 + ((f * 4 + q) ^ (l32 & 7)) * 16 + h * 8) =
                    make_uint2(f2h(o[4 * q] * sc) | ((uint32_t)f2h(o[4 * q + 1] * sc) << 16),
                               f2h(o[4 * q + 2] * sc) | ((uint32_t)f2h(o[4 * q + 3] * sc) << 16));
            }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int t = e * 8 + (lane >> 3), p = lane & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(mine + t * 128 + (p ^ (t & 7)) * 16);
            const int m = m0 + wm * 32 * FM + 32 * i + t;
            if (m < M)
                store8(a.dx + (int64_t)m * K, j0 + wj * 64 + 8 * p, K, v);
        }
        asm volatile("" ::: "memory");
    }
    weak_put(a, range, m0 + wm * 64, min(64, M - (m0 + wm * 64)));
}

// The splits' sums of 32 tokens x 32 columns, a wave each
__global__ __launch_bounds__(64) void k_int8_dx_sum(const BwdArgs8 a, int tiles)
{
    const int lane = threadIdx.x, l32 = lane & 31, h = lane >> 5;
    const int piece = (int)blockIdx.x & 15, tile = (int)blockIdx.x >> 4;
    const int wave = piece >> 2, i = (piece >> 1) & 1, f = piece & 1;  // as in k_int8_dx
    const int m0 = (tile % a.mblocks) * kDxTokens + (wave & 1) * 64 + 32 * i;
    const int j0 = (tile / a.mblocks) * kDxCols + (wave >> 1) * 64 + 32 * f;
    if (m0 >= a.M || j0 >= a.K)
        return;
    const WeakRange range = weak_range(a, j0, 32);
    const i8_f4v* p = a.sums + ((int64_t)tile * 4 + wave) * (16 * 64) + (i * 2 + f) * (4 * 64) + lane;
    i8_f4v sum[4];
#pragma unroll
    for (int q = 0; q < 4; q++)
        sum[q] = p[q * 64];
    for (int s = 1; s < a.splits; s++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            sum[q] += p[(int64_t)s * tiles * 4 * (16 * 64) + q * 64];
    const int m = m0 + l32;
    if (m < a.M) {
        const float f = a.unscale[m];
#pragma unroll
        for (int q = 0; q < 4; q++)
            store4(a.dx + (int64_t)m * a.K, j0 + 8 * q + 4 * h, a.K, sum[q] * f);
    }
    weak_put(a, range, m0, min(32, a.M - m0));
}

// Blocks per tile: as many as leave one per CU (a CU takes two, but a part is 64 KB of sums
// written and read again, and the weak sums beside the product want CUs too), each with at least 8
// stages. The whole backward in us with 1 | 256 / tiles | 512 / tiles parts: one token of
// 4096 x 4096 (32 tiles) 56 | 26 | 32; 64 of 11008 x 4096 (32) 138 | 48 | 55; 150 of 3584 x 3584 (56) 55 | 32 |
// 34; 512 of 4096 x 4096 (128) 67 | 54 | 55; 1000 of 4096 x 1024 (64) 69 | 42 | 48; 400 of 11008 x 512 (16)
// 153 | 56 | 67, and 51 with half as many; 2000 of 2816 x 320 (48) 57 | 41 | 53, and 37 with two; 1000 of
// 28672 x 256 without weak columns (16) 321 | 82 | 89; 2048 of 768 x 768 (96) 33 | 33 | 37.
int dx_splits(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = (M + kDxTokens - 1) / kDxTokens * ((K + kDxCols - 1) / kDxCols);
    int64_t sp = 256 / tiles;
    const int64_t most = (N + kDxRows - 1) / kDxRows / 8;
    sp = sp < most ? sp : most;
    return (int)(sp < 1 ? 1 : sp);
}

constexpr int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace

Int8BwdPlan int8_bwd_plan(int64_t N, int64_t K, int32_t k, int64_t M)
{
    Int8BwdPlan p{};
    p.Np = up(N, kDxRows);
    p.Mp = up(M, 16);
    p.kp = up(k, 32);
    p.splits = dx_splits(M, N, K);
    p.tiles = up(M, kDxTokens) / kDxTokens * (up(K, kDxCols) / kDxCols);
    // slices of the weak columns' sums: enough blocks, at least 512 rows each. Whole backward with
    // 1 | these | twice as many, us: 64 tokens of 11008 x 4096 (21) 105 | 53 | 53; 77 of 2731 x 1056 (5)
    // 32 | 20 | 22; 1000 of 4096 x 1024 (8) 61 | 47 | 52
    const int64_t tiles = (M + 31) / 32 * (p.kp / 32 > 0 ? p.kp / 32 : 1);
    int64_t sl = (512 + tiles - 1) / tiles;
    sl = sl < p.Np / 512 ? sl : p.Np / 512;
    p.slices = sl < 1 ? 1 : sl;
    size_t off = (size_t)(4 * up(M, kDxTokens) * p.Np);  // whole panels
    auto take = [&](size_t& at, int64_t bytes) {
        at = off;
        off += (size_t)up(bytes, 256);
    };
    take(p.off_un, 4 * M);
    take(p.off_wwt, 2 * p.kp * p.Np);
    take(p.off_xwt, 2 * p.kp * p.Mp);
    take(p.off_part, 4 * p.slices * M * p.kp);
    take(p.off_sums, p.splits > 1 ? 4LL * p.splits * p.tiles * kDxTokens * kDxCols : 0);
    p.total = off;
    return p;
}

hipError_t launch_linear_int8_backward(const Int8Desc& d, const uint16_t* dy, int64_t M, uint16_t* dx, float* dw,
                                       void* ws, const Int8BwdPlan& p, hipStream_t s)
{
    char* const w = static_cast<char*>(ws);
    const BwdArgs8 a{d.q, d.s, d.idx, d.ww, d.x, dy, dx, d.k > 0 ? dw : nullptr, reinterpret_cast<uint16_t*>(w),
                     reinterpret_cast<float*>(w + p.off_un), reinterpret_cast<uint16_t*>(w + p.off_wwt),
                     reinterpret_cast<uint16_t*>(w + p.off_xwt), reinterpret_cast<float*>(w + p.off_part),
                     reinterpret_cast<i8_f4v*>(w + p.off_sums), (int32_t)M, (int32_t)d.N, (int32_t)d.K, d.k, (int32_t)p.Np,
                     (int32_t)p.Mp, (int32_t)p.kp, (int32_t)p.slices, (int32_t)(up(M, kDxTokens) / kDxTokens), p.splits};
    const int64_t turned = d.k > 0 ? ((dx ? p.kp * p.Np : 0) + (a.dw ? p.kp * p.Mp : 0) + 255) / 256 : 0;
    const int64_t tokens = dx ? M : 0;
    hipLaunchKernelGGL(k_int8_prepare, dim3((unsigned)(tokens + (turned < 1024 ? turned : 1024))), dim3(256), 0, s, a,
                       (int)tokens);
    const int64_t dws = a.dw ? (d.N + 31) / 32 : 0, dxs = dx && d.k > 0 ? (M + 31) / 32 * p.slices : 0;
    // the weak sums: beside the product where its parts are added in a launch of their own
    // (they go into dx there) and one grid holds both, else before it. Beside | before, us: 77 tokens of
    // 2731 x 1056 20 | 25; 64 of 11008 x 4096 48 | 53; 1000 of 4096 x 1024 42 | 47; 1000 of 28672 x 256 161 |
    // 174; 2048 of 11008 x 512 119 | 119. First in that grid instead of last: mostly within 5 %
    // either way, 36 % worse at worst (300 tokens of 11008 x 4096).
    const int64_t blocks = p.tiles * p.splits, sums = (dws + dxs) * (p.kp / 32);
    const bool beside = dx && p.splits > 1 && grid_fits(blocks + sums, 256);
    if (!beside && sums > 0)
        hipLaunchKernelGGL(k_int8_weak_sums, dim3((unsigned)(dws + dxs), (unsigned)(p.kp / 32)), dim3(64 * kWeakParts), 0, s, a,
                           (int)dws);
    if (dx) {
        hipLaunchKernelGGL(k_int8_dx, dim3((unsigned)(blocks + (beside ? sums : 0))), dim3(256), 0, s, a, (int)blocks, (int)dws);
        if (p.splits > 1)
            hipLaunchKernelGGL(k_int8_dx_sum, dim3((unsigned)(16 * p.tiles)), dim3(64), 0, s, a, (int)p.tiles);
    }
    return hipGetLastError();
}

}  // namespace owq
