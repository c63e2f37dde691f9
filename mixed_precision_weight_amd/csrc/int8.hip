// int8.hip -- the 8-bit form: pack and product (gfx950).
//
//   y[m][i] = s_m scale_i sum_j q_mj code_ij + sum_c x[m][idx_c] w_weak[i][c]
// with a token's dense columns quantised on the way in (s_m = t_m / 127, q_mj =
// rint(x_mj * (127 / t_m)), t_m the token's largest dense magnitude). The integer sums
// are exact; scales, weak columns and their sums are fp32, y is rounded to fp16 once.
#include "owq_int8.h"
#include "owq_pair_gemm.h"

namespace owq {

namespace {

// -------------------------------------------------------------------- pack --

// One block per row: the largest dense magnitude, then the codes and the weak weights.
// Compiled like the rest of the file with FMA contraction: code8 has no sum to contract.
__global__ __launch_bounds__(256) void k_pack_int8(const uint16_t* __restrict__ W, int K, const int32_t* __restrict__ idx,
                                                   int k, int8_t* __restrict__ codes, float* __restrict__ scales,
                                                   uint16_t* __restrict__ ww)
{
    __shared__ uint32_t mask[65536 / 32];
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint4* w = reinterpret_cast<const uint4*>(W + row * K);
    weak_mask<256>(mask, idx, k, K);
    const uint8_t* m8 = reinterpret_cast<const uint8_t*>(mask);
    uint32_t top = 0;
    for (int p = tid; p < K >> 3; p += 256)
        top = top8(w[p], m8[p], top);
    top = wave_max_u32(top);
    if ((tid & 63) == 0)
        red[tid >> 6] = top;
    __syncthreads();
    const RowScale rs = row_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (tid == 0)
        scales[row] = rs.scale;
    uint2* q = reinterpret_cast<uint2*>(codes + row * K);
    for (int p = tid; p < K >> 3; p += 256) {
        const uint4 v = w[p];
        uint2 c = make_uint2(code8x4(v.x, v.y, rs.factor), code8x4(v.z, v.w, rs.factor));
        const uint32_t b = m8[p];
        if (b) {
            uint32_t keep[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                keep[h] = 0;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    keep[h] |= (b >> (4 * h + e)) & 1u ? 0u : 0xffu << (8 * e);
            }
            c.x &= keep[0];
            c.y &= keep[1];
        }
        q[p] = c;
    }
    for (int c = tid; c < k; c += 256) {
        const int j = idx[c];
        ww[row * k + c] = j >= 0 && j < K ? W[row * K + j] : (uint16_t)0;
    }
}

// ---------------------------------------------------------------- the tokens --

struct QuantLayer {
    const uint16_t* x;
    const int32_t* idx;
    int8_t* x8;
    float* sx;
    uint16_t* xw;
    int32_t K, Kq, k, kp;
};
struct QuantBatch {
    QuantLayer L[kInt8MaxLayers];
};

// One block per token (and layer, blockIdx.y): its scale, its codes up to Kq columns
// (zeros past K) and its weak columns padded to kp with zeros. OPERAND: the codes in the
// order of the decode's B operand (64-column steps, lane 16 g + m holds the 16 columns
// g of token m); else row-major [M][Kq].
template <bool OPERAND>
__global__ __launch_bounds__(256) void k_int8_tokens(const QuantBatch b)
{
    __shared__ uint32_t mask[65536 / 32];
    __shared__ uint32_t red[4];
    const QuantLayer& L = b.L[blockIdx.y];
    const int tid = threadIdx.x;
    const int64_t m = blockIdx.x;
    const int K = L.K;
    const uint16_t* xr = L.x + m * K;
    const uint4* xp = reinterpret_cast<const uint4*>(xr);
    weak_mask<256>(mask, L.idx, L.k, K);
    const uint8_t* m8 = reinterpret_cast<const uint8_t*>(mask);
    uint32_t top = 0;
    for (int p = tid; p < K >> 3; p += 256)
        top = top8(xp[p], m8[p], top);
    top = wave_max_u32(top);
    if ((tid & 63) == 0)
        red[tid >> 6] = top;
    __syncthreads();
    const RowScale rs = row_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (tid == 0)
        L.sx[m] = rs.scale;
    for (int p = tid; p < L.Kq >> 4; p += 256) {  // 16 columns, K is a multiple of 32
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        if (p < K >> 4) {
            const uint4 v = xp[2 * p], w = xp[2 * p + 1];
            c = make_uint4(code8x4(v.x, v.y, rs.factor), code8x4(v.z, v.w, rs.factor), code8x4(w.x, w.y, rs.factor),
                           code8x4(w.z, w.w, rs.factor));
        }
        const int64_t at = OPERAND ? (int64_t)(p >> 2) * 1024 + (p & 3) * 256 + m * 16 : m * L.Kq + (int64_t)p * 16;
        *reinterpret_cast<uint4*>(L.x8 + at) = c;
    }
    for (int c = tid; c < L.kp; c += 256) {
        const int j = c < L.k ? L.idx[c] : -1;
        L.xw[m * L.kp + c] = j >= 0 && j < K ? xr[j] : (uint16_t)0;
    }
}

// ---------------------------------------------- up to four tokens: one launch --

struct DecLayer {
    const int8_t* q;
    const float* s;
    const int32_t* idx;
    const uint16_t* ww;
    const uint16_t* x;
    uint16_t* y;
    int32_t N, K, k, block0;
};
struct DecBatch {
    DecLayer L[kInt8MaxLayers];
    int32_t count;
};

constexpr int kDecRows = 4;       // rows per wave
constexpr int kDecChunk = 4096;   // columns staged at a time
constexpr int kDecTiles = kDecChunk / 1024;

// A block of 4 waves computes 4 kDecRows rows; it quantises the tokens for itself (they
// come from the caches), which saves the launch that would do it once.
template <int M>
__global__ __launch_bounds__(256) void k_int8_gemv(const DecBatch b)
{
    constexpr int R = kDecRows;
    __shared__ uint32_t mask[65536 / 32];
    __shared__ uint4 x8[M][kDecChunk / 16];
    __shared__ uint32_t red[M][4];
    int li = 0;
    for (int l = 1; l < b.count; l++)
        if ((int)blockIdx.x >= b.L[l].block0)
            li = l;
    const DecLayer& L = b.L[li];
    const int N = L.N, K = L.K, k = L.k;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int brow = ((int)blockIdx.x - L.block0) * 4 * R;
    const int nb = min(N - brow, 4 * R);
    const __amdgpu_buffer_rsrc_t qr = bytes_rsrc(L.q + (int64_t)brow * K, (int64_t)nb * K);
    int qoff[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        qoff[r] = min(wave * R + r, nb - 1) * K + lane * 16;
    auto load = [&](int c0, uint4 (&v)[R][kDecTiles]) {
#pragma unroll
        for (int t = 0; t < kDecTiles; t++) {
            const int dead = c0 + t * 1024 + lane * 16 < K ? 0 : 0x40000000;
#pragma unroll
            for (int r = 0; r < R; r++)
                v[r][t] = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(qr, qoff[r] + c0 + t * 1024 + dead, 0, 2));
        }
    };
    uint4 cv[R][kDecTiles];
    load(0, cv);
    weak_mask<256>(mask, L.idx, k, K);
    const uint8_t* m8 = reinterpret_cast<const uint8_t*>(mask);
    RowScale rs[M];
    {
        uint32_t top[M];
#pragma unroll
        for (int m = 0; m < M; m++) {
            top[m] = 0;
            const uint4* xp = reinterpret_cast<const uint4*>(L.x + (int64_t)m * K);
            for (int p = tid; p < K >> 3; p += 256)
                top[m] = top8(xp[p], m8[p], top[m]);
            top[m] = wave_max_u32(top[m]);
            if (lane == 0)
                red[m][wave] = top[m];
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; m++)
            rs[m] = row_scale(max(max(red[m][0], red[m][1]), max(red[m][2], red[m][3])));
    }
    int acc[R][M];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int m = 0; m < M; m++)
            acc[r][m] = 0;
    for (int c0 = 0; c0 < K; c0 += kDecChunk) {
        if (c0 > 0) {
            __syncthreads();
            load(c0, cv);
        }
#pragma unroll
        for (int m = 0; m < M; m++) {
            const uint4* xp = reinterpret_cast<const uint4*>(L.x + (int64_t)m * K + c0);
            const int p = tid;  // kDecChunk / 16 == 256 pieces of 16 columns
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            if (c0 + p * 16 < K) {
                const uint4 v = xp[2 * p], w = xp[2 * p + 1];
                c = make_uint4(code8x4(v.x, v.y, rs[m].factor), code8x4(v.z, v.w, rs[m].factor),
                               code8x4(w.x, w.y, rs[m].factor), code8x4(w.z, w.w, rs[m].factor));
            }
            x8[m][p] = c;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kDecTiles; t++)
#pragma unroll
            for (int m = 0; m < M; m++) {
                const uint4 xv = x8[m][t * 64 + lane];
#pragma unroll
                for (int r = 0; r < R; r++) {
                    acc[r][m] = __builtin_amdgcn_sdot4((int)cv[r][t].x, (int)xv.x, acc[r][m], false);
                    acc[r][m] = __builtin_amdgcn_sdot4((int)cv[r][t].y, (int)xv.y, acc[r][m], false);
                    acc[r][m] = __builtin_amdgcn_sdot4((int)cv[r][t].z, (int)xv.z, acc[r][m], false);
                    acc[r][m] = __builtin_amdgcn_sdot4((int)cv[r][t].w, (int)xv.w, acc[r][m], false);
                }
            }
    }
    float part[R][M];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float sw = L.s[brow + min(wave * R + r, nb - 1)];
#pragma unroll
        for (int m = 0; m < M; m++)
            part[r][m] = (float)acc[r][m] * (rs[m].scale * sw);  // a lane's sum is below 2^24: exact
    }
    for (int c = lane; c < k; c += 64) {
        int j = L.idx[c];
        j = j >= 0 && j < K ? j : 0;
        float xw[M];
#pragma unroll
        for (int m = 0; m < M; m++)
            xw[m] = h2f(L.x[(int64_t)m * K + j]);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float w = h2f(L.ww[(int64_t)(brow + min(wave * R + r, nb - 1)) * k + c]);
#pragma unroll
            for (int m = 0; m < M; m++)
                part[r][m] = __builtin_fmaf(xw[m], w, part[r][m]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int m = 0; m < M; m++) {
            const float v = wave_sum_dpp(part[r][m]);
            if (lane == 0 && wave * R + r < nb)
                L.y[(int64_t)m * N + brow + wave * R + r] = f2h(v);
        }
}

// ------------------------------------------------ up to 16 tokens: one B tile --

struct MfvLayer {
    const int8_t* q;
    const float* s;
    const uint16_t* ww;
    uint16_t* y;
    const int8_t* x8;
    const float* sx;
    const uint16_t* xw;
    int32_t N, K, k, kp, block0;
};
struct MfvBatch {
    MfvLayer L[kInt8MaxLayers];
    int32_t count, M;
};

constexpr int kMfvWaves = 4;  // waves that split K
constexpr int kMfvStep = 8;   // 64-column steps whose loads are in flight together

// A block computes 16 rows for all tokens: v_mfma_i32_16x16x64_i8 with the codes as A
// (lane l: row l % 16, 16 columns 16 (l / 16) of a 64-column step) and the tokens as B.
__global__ __launch_bounds__(64 * kMfvWaves) void k_int8_mfv(const MfvBatch b)
{
    __shared__ i32x4 part[kMfvWaves - 1][64];
    int li = 0;
    for (int l = 1; l < b.count; l++)
        if ((int)blockIdx.x >= b.L[l].block0)
            li = l;
    const MfvLayer& L = b.L[li];
    const int N = L.N, K = L.K;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = ((int)blockIdx.x - L.block0) * 16;
    const int nb = min(N - row0, 16);
    const int r16 = lane & 15, g = lane >> 4;
    const __amdgpu_buffer_rsrc_t qr = bytes_rsrc(L.q + (int64_t)row0 * K, (int64_t)nb * K);
    const int steps = (K + 63) >> 6;
    const int per = (steps + kMfvWaves - 1) / kMfvWaves;
    const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
    const int qoff = min(r16, nb - 1) * K + g * 16;
    const uint4* xb = reinterpret_cast<const uint4*>(L.x8) + lane;
    i32x4 acc = {0, 0, 0, 0};
    for (int st = s0; st < s1; st += kMfvStep) {
        uint4 cv[kMfvStep], xv[kMfvStep];
#pragma unroll
        for (int u = 0; u < kMfvStep; u++) {
            const int dead = st + u < s1 ? 0 : 0x40000000;
            cv[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(qr, qoff + (st + u) * 64 + dead, 0, 2));
        }
#pragma unroll
        for (int u = 0; u < kMfvStep; u++)
            xv[u] = xb[min(st + u, s1 - 1) * 64];
#pragma unroll
        for (int u = 0; u < kMfvStep; u++)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, cv[u]),
                                                        __builtin_bit_cast(i32x4, xv[u]), acc, 0, 0, 0);
    }
    if (wave > 0)
        part[wave - 1][lane] = acc;
    __syncthreads();
    if (wave > 0)
        return;
#pragma unroll
    for (int w = 0; w < kMfvWaves - 1; w++)
        acc += part[w][lane];
    // lane l: token l % 16, rows 4 (l / 16) + r
    const int m = min(r16, b.M - 1);
    const float sm = L.sx[m];
    i8_f4v out;
#pragma unroll
    for (int r = 0; r < 4; r++)
        out[r] = (float)acc[r] * (sm * L.s[row0 + min(4 * g + r, nb - 1)]);
    const PairLayer P{nullptr, nullptr, nullptr, nullptr, L.ww, L.k};
    for (int c = 0; c < L.kp; c += 32) {
        const half8_t wv = pair_weak(P, row0 + min(r16, nb - 1), c + 8 * g);
        const half8_t xv = *reinterpret_cast<const half8_t*>(L.xw + (int64_t)m * L.kp + c + 8 * g);
        out = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, xv, out, 0, 0, 0);
    }
    if (r16 < b.M)
#pragma unroll
        for (int r = 0; r < 4; r++)
            if (4 * g + r < nb)
                L.y[(int64_t)r16 * N + row0 + 4 * g + r] = f2h(out[r]);
}

// ----------------------------------------------------- more tokens: tiled GEMM --

struct GemmArgs8 {
    const int8_t* q;
    const float* s;
    const uint16_t* ww;
    uint16_t* y;
    const int8_t* x8;
    const float* sx;
    const uint16_t* xw;
    int32_t M, N, K, Kq, k, kp;
    int32_t mblocks;
};

template <int FM, int FN, int WM, int WN>
struct Tile8 {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    static constexpr int DA = BM * 128 / 16 / NT, DB = BN * 128 / 16 / NT;  // 16-byte units per thread and stage
    static_assert(DA * NT * 16 == BM * 128 && DB * NT * 16 == BN * 128, "a stage must split evenly over the threads");
};

// BM tokens x BN rows per block, both operands through LDS in stages of 128 columns
// (direct-to-LDS loads, the piece c of row r in slot c ^ (r & 7) of the row's 128 bytes,
// so that the operand reads of a wave spread over the banks), two stages.
template <int FM, int FN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void k_int8_gemm(const GemmArgs8 a)
{
    using T = Tile8<FM, FN, WM, WN>;
    constexpr int BM = T::BM, BN = T::BN;
    __shared__ __attribute__((aligned(1024))) char s0[(BM + BN) * 128];
    __shared__ __attribute__((aligned(1024))) char s1[(BM + BN) * 128];
    const int M = a.M, N = a.N, K = a.K, Kq = a.Kq;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int l32 = lane & 31, h = lane >> 5;
    const int m0 = ((int)blockIdx.x % a.mblocks) * BM, n0 = ((int)blockIdx.x / a.mblocks) * BN;
    const int mv = min(BM, M - m0), nv = min(BN, N - n0);
    const __amdgpu_buffer_rsrc_t xr = bytes_rsrc(a.x8 + (int64_t)m0 * Kq, (int64_t)mv * Kq);
    const __amdgpu_buffer_rsrc_t qr = bytes_rsrc(a.q + (int64_t)n0 * K, (int64_t)nv * K);
    int xsrc[T::DA], qsrc[T::DB];
#pragma unroll
    for (int t = 0; t < T::DA; t++) {
        const int u = (wave * T::DA + t) * 64 + lane, row = u >> 3;
        xsrc[t] = min(row, mv - 1) * Kq + ((u & 7) ^ (row & 7)) * 16;
    }
#pragma unroll
    for (int t = 0; t < T::DB; t++) {
        const int u = (wave * T::DB + t) * 64 + lane, row = u >> 3;
        qsrc[t] = min(row, nv - 1) * K + ((u & 7) ^ (row & 7)) * 16;
    }
    // (pieces past K of the last stage hold the next row's codes, or zeros past the
    // last row: the tokens' codes there are zeros)
    auto dma = [&](int c, char* stage) {
#pragma unroll
        for (int t = 0; t < T::DA; t++)
            dma16_lds(xr, stage + (wave * T::DA + t) * 1024, xsrc[t] + c * 128);
#pragma unroll
        for (int t = 0; t < T::DB; t++)
            dma16_lds(qr, stage + BM * 128 + (wave * T::DB + t) * 1024, qsrc[t] + c * 128);
    };
    i32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[i][f][r] = 0;
    const int arow = (wm * 32 * FM + l32) * 128, brow = (BM + wn * 32 * FN + l32) * 128;
    const int chunks = Kq >> 7;
    auto step = [&](int c, const char* cur, char* nxt) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (c + 1 < chunks)
            dma(c + 1, nxt);
        if (c < chunks) {
#pragma unroll
            for (int st = 0; st < 4; st++) {
                const int slot = ((st * 2 + h) ^ (l32 & 7)) * 16;
                i32x4 av[FM], bv[FN];
#pragma unroll
                for (int i = 0; i < FM; i++)
                    av[i] = *reinterpret_cast<const i32x4*>(cur + arow + i * 4096 + slot);
#pragma unroll
                for (int f = 0; f < FN; f++)
                    bv[f] = *reinterpret_cast<const i32x4*>(cur + brow + f * 4096 + slot);
#pragma unroll
                for (int i = 0; i < FM; i++)
#pragma unroll
                    for (int f = 0; f < FN; f++)
                        acc[i][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[i], bv[f], acc[i][f], 0, 0, 0);
            }
        }
    };
    dma(0, s0);
    for (int c = 0; c < chunks; c += 2) {
        step(c, s0, s1);
        step(c + 1, s1, s0);
    }
    // D element r of lane l: token 8 (r / 4) + 4 h + r % 4, row l % 32
    const PairLayer P{nullptr, nullptr, nullptr, nullptr, a.ww, a.k};
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int mb = wm * 32 * FM + 32 * i;
        float sm[16];
#pragma unroll
        for (int r = 0; r < 16; r++)
            sm[r] = a.sx[m0 + min(mb + 8 * (r >> 2) + 4 * h + (r & 3), mv - 1)];
#pragma unroll
        for (int f = 0; f < FN; f++) {
            const int nr = min(wn * 32 * FN + 32 * f + l32, nv - 1);
            const float sn = a.s[n0 + nr];
            i8_f16v out;
#pragma unroll
            for (int r = 0; r < 16; r++)
                out[r] = (float)acc[i][f][r] * (sm[r] * sn);
            for (int c = 0; c < a.kp; c += 16) {
                const half8_t xv = *reinterpret_cast<const half8_t*>(a.xw + (int64_t)(m0 + min(mb + l32, mv - 1)) * a.kp + c + 8 * h);
                out = __builtin_amdgcn_mfma_f32_32x32x16_f16(xv, pair_weak(P, n0 + nr, c + 8 * h), out, 0, 0, 0);
            }
            const int n = n0 + wn * 32 * FN + 32 * f + l32;
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int m = m0 + mb + 8 * (r >> 2) + 4 * h + (r & 3);
                if (m < M && n < N)
                    a.y[(int64_t)m * N + n] = f2h(out[r]);
            }
        }
    }
}

template <int FM, int FN, int WM, int WN>
bool tile8_fits(int64_t M, int64_t N)
{
    using T = Tile8<FM, FN, WM, WN>;
    return grid_fits((M + T::BM - 1) / T::BM * ((N + T::BN - 1) / T::BN), T::NT);
}

template <int FM, int FN, int WM, int WN>
hipError_t launch_tile8(GemmArgs8 a, hipStream_t s)
{
    using T = Tile8<FM, FN, WM, WN>;
    a.mblocks = (a.M + T::BM - 1) / T::BM;
    const int64_t blocks = (int64_t)a.mblocks * ((a.N + T::BN - 1) / T::BN);
    hipLaunchKernelGGL((k_int8_gemm<FM, FN, WM, WN>), dim3((unsigned)blocks), dim3(T::NT), 0, s, a);
    return hipGetLastError();
}

constexpr int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace

Int8Plan int8_plan(int64_t N, int64_t K, int32_t k, int64_t M)
{
    (void)N;
    Int8Plan p{};
    if (M <= kInt8GemvMaxM)
        return p;
    p.Kq = up(K, 128);
    p.kp = (int32_t)up(k, 32);
    p.off_sx = (size_t)(p.Kq * (M <= kInt8DecodeMaxM ? 16 : M));
    p.off_xw = p.off_sx + (size_t)up(M * 4, 256);
    p.total = p.off_xw + (size_t)up(M * p.kp * 2, 256);
    return p;
}

bool int8_grid_fits(int64_t M, int64_t N)
{
    if (M <= kInt8GemvMaxM)
        return grid_fits((N + 4 * kDecRows - 1) / (4 * kDecRows), 256);
    if (M <= kInt8DecodeMaxM)
        return grid_fits((N + 15) / 16, 64 * kMfvWaves);
    return grid_fits(M, 256) && (M > 128 ? tile8_fits<4, 2, 2, 4>(M, N) : tile8_fits<1, 1, 1, 4>(M, N));
}

hipError_t launch_pack_int8(const uint16_t* W, int64_t N, int64_t K, const int32_t* idx, int32_t k, int8_t* codes,
                            float* scales, uint16_t* ww, hipStream_t s)
{
    hipLaunchKernelGGL(k_pack_int8, dim3((unsigned)N), dim3(256), 0, s, W, (int)K, idx, k, codes, scales, ww);
    return hipGetLastError();
}

hipError_t launch_linear_int8(const Int8Desc* d, int count, int64_t M, void* const* ws, hipStream_t s)
{
    if (M <= kInt8GemvMaxM) {
        DecBatch b{};
        b.count = count;
        int64_t blocks = 0;
        for (int l = 0; l < count; l++) {
            b.L[l] = DecLayer{d[l].q, d[l].s, d[l].idx, d[l].ww, d[l].x, d[l].y, (int32_t)d[l].N, (int32_t)d[l].K, d[l].k,
                              (int32_t)blocks};
            blocks += (d[l].N + 4 * kDecRows - 1) / (4 * kDecRows);
        }
        if (!grid_fits(blocks, 256))
            return hipErrorInvalidConfiguration;
        const dim3 grid((unsigned)blocks), block(256);
        if (M == 1)
            hipLaunchKernelGGL(k_int8_gemv<1>, grid, block, 0, s, b);
        else if (M == 2)
            hipLaunchKernelGGL(k_int8_gemv<2>, grid, block, 0, s, b);
        else if (M == 3)
            hipLaunchKernelGGL(k_int8_gemv<3>, grid, block, 0, s, b);
        else
            hipLaunchKernelGGL(k_int8_gemv<4>, grid, block, 0, s, b);
        return hipGetLastError();
    }
    QuantBatch qb{};
    Int8Plan p[kInt8MaxLayers];
    int64_t mfv_blocks = 0;
    for (int l = 0; l < count; l++) {
        p[l] = int8_plan(d[l].N, d[l].K, d[l].k, M);
        char* const w = static_cast<char*>(ws[l]);
        qb.L[l] = QuantLayer{d[l].x, d[l].idx, reinterpret_cast<int8_t*>(w), reinterpret_cast<float*>(w + p[l].off_sx),
                             reinterpret_cast<uint16_t*>(w + p[l].off_xw), (int32_t)d[l].K, (int32_t)p[l].Kq, d[l].k, p[l].kp};
        mfv_blocks += (d[l].N + 15) / 16;
    }
    const dim3 tokens((unsigned)M, (unsigned)count);
    if (M <= kInt8DecodeMaxM) {
        if (!grid_fits(mfv_blocks, 64 * kMfvWaves))
            return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(k_int8_tokens<true>, tokens, dim3(256), 0, s, qb);
        MfvBatch b{};
        b.count = count;
        b.M = (int32_t)M;
        int64_t blocks = 0;
        for (int l = 0; l < count; l++) {
            const QuantLayer& q = qb.L[l];
            b.L[l] = MfvLayer{d[l].q, d[l].s, d[l].ww, d[l].y, q.x8, q.sx, q.xw, (int32_t)d[l].N, (int32_t)d[l].K, d[l].k,
                              q.kp, (int32_t)blocks};
            blocks += (d[l].N + 15) / 16;
        }
        hipLaunchKernelGGL(k_int8_mfv, dim3((unsigned)blocks), dim3(64 * kMfvWaves), 0, s, b);
        return hipGetLastError();
    }
    if (count != 1 || !int8_grid_fits(M, d[0].N))  // before the first launch
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(k_int8_tokens<false>, tokens, dim3(256), 0, s, qb);
    const QuantLayer& q = qb.L[0];
    const GemmArgs8 a{d[0].q, d[0].s, d[0].ww, d[0].y, q.x8, q.sx, q.xw, (int32_t)M, (int32_t)d[0].N, (int32_t)d[0].K,
                      q.Kq, q.k, q.kp, 1};
    if (M > 128)
        return launch_tile8<4, 2, 2, 4>(a, s);  // 256 tokens x 256 rows
    return launch_tile8<1, 1, 1, 4>(a, s);      // 32 tokens x 128 rows
}

}  // namespace owq
