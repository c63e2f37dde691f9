// int8.hip -- the integer form: pack and product (gfx950).
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

// One block per row: the largest dense magnitude, then the codes and the weak weights, the row
// read again from L2. 11008 x 4096: 37 us, 135 MB at 3.6 TB/s (a copy's 5.15 would take 26); what is
// missing is the chain mask, row, largest magnitude, row in each block, of which the mask's 32 KB
// of LDS leaves four to a CU. It runs once per layer.
template <bool WIDE>
__global__ __launch_bounds__(256) void k_pack_int8(const uint16_t* __restrict__ W, int K, const int32_t* __restrict__ idx,
                                                   int k, int8_t* __restrict__ codes, float* __restrict__ scales,
                                                   uint16_t* __restrict__ ww)
{
    __shared__ DenseMask<WIDE> mask;
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint4* w = reinterpret_cast<const uint4*>(W + row * K);
    mask.template fill<256>(idx, k, K);
    uint32_t top = 0;
    for (int p = tid; p < K >> 3; p += 256)
        top = mask.top(w[p], p, top);
    top = wave_max_u32(mask.both(top));
    if ((tid & 63) == 0)
        red[tid >> 6] = top;
    __syncthreads();
    const RowScale rs = row_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (tid == 0)
        scales[row] = rs.scale;
    uint2* q = reinterpret_cast<uint2*>(codes + row * K);
    for (int p = tid; p < K >> 3; p += 256) {
        const uint4 v = w[p];
        uint32_t c[2] = {code8x4(v.x, v.y, rs.factor), code8x4(v.z, v.w, rs.factor)};
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (mask.weak(8 * p + e))
                c[e >> 2] &= ~(0xffu << (8 * (e & 3)));
        q[p] = make_uint2(c[0], c[1]);
    }
    for (int c = tid; c < k; c += 256) {
        const int j = idx[c];
        ww[row * k + c] = j >= 0 && j < K ? W[row * K + j] : (uint16_t)0;
    }
}

// The tiled product's sizes
constexpr int kGemmCols = 64;     // columns per stage
constexpr int kGemmTokens = 256;  // tokens per tile, and per panel of their codes
constexpr int kWeakPanel = 128;   // rows per panel of the weak weights: a small tile's
constexpr int kSumVectors = 256 * 128 / 4;  // four sums each: of a small tile

// ---------------------------------------------------------------- the tokens --

struct QuantLayer {
    const uint16_t* x;
    const int32_t* idx;
    const uint16_t* ww;
    int8_t* x8;
    float* sx;
    uint16_t* xw;
    uint16_t* wwp;
    int32_t N, K, Kq, k, kp;
};
struct QuantBatch {
    QuantLayer L[kInt8MaxLayers];
};

// The tokens of the streaming product: one block per token and layer (blockIdx.y), its
// scale, its codes up to Kq columns (zeros past K) and its weak columns padded to kp with
// zeros. The codes go in the order of that product's B operand (16 tokens together,
// 64-column steps, lane 16 g + m holds the 16 columns g of token m). P: 16-column pieces a
// thread holds (the rest of a longer row is read twice): one up to 4096 columns, else three. One | three,
// us, tokens not in the caches: 16 tokens, 4096 x 11008, 21.3 | 20.7, 1024 x 12288 16.7 | 16.3; from
// them, 1024 x 4096, 9.1 | 9.3. A launch and a chain of three latencies (weak
// columns, token, largest magnitude): 3.6 us for 16 tokens of 4096.
template <bool WIDE, int P>
__global__ __launch_bounds__(256) void k_int8_tokens(const QuantBatch b)
{
    __shared__ DenseMask<WIDE> mask;
    __shared__ uint32_t red[4];
    const QuantLayer& L = b.L[blockIdx.y];
    const int tid = threadIdx.x;
    const int K = L.K, kp = L.kp;
    const int64_t m = blockIdx.x;
    const uint16_t* xr = L.x + m * K;
    const uint4* xp = reinterpret_cast<const uint4*>(xr);
    const int pieces = K >> 4;
    uint4 v[P][2];
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = tid + 256 * i;
        if (p < pieces) {
            v[i][0] = xp[2 * p];
            v[i][1] = xp[2 * p + 1];
        }
    }
    mask.template fill<256>(L.idx, L.k, K);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = tid + 256 * i;
        if (p < pieces) {
            top = mask.top(v[i][0], 2 * p, mask.top(v[i][1], 2 * p + 1, top));
        }
    }
    for (int p = tid + 256 * P; p < pieces; p += 256)
        top = mask.top(xp[2 * p], 2 * p, mask.top(xp[2 * p + 1], 2 * p + 1, top));
    top = wave_max_u32(mask.both(top));
    if ((tid & 63) == 0)
        red[tid >> 6] = top;
    __syncthreads();
    const RowScale rs = row_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (tid == 0)
        L.sx[m] = rs.scale;
    int8_t* x8 = L.x8 + (m >> 4) * 16 * L.Kq + (m & 15) * 16;
    auto put = [&](int p, uint4 c) { *reinterpret_cast<uint4*>(x8 + (int64_t)(p >> 2) * 1024 + (p & 3) * 256) = c; };
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = tid + 256 * i;
        if (p < pieces)
            put(p, code8x16(v[i][0], v[i][1], rs.factor));
    }
    for (int p = tid + 256 * P; p < pieces; p += 256)
        put(p, code8x16(xp[2 * p], xp[2 * p + 1], rs.factor));
    for (int p = pieces + tid; p < L.Kq >> 4; p += 256)
        put(p, make_uint4(0u, 0u, 0u, 0u));
    for (int c = tid; c < kp; c += 256) {
        const int j = c < L.k ? L.idx[c] : -1;
        L.xw[m * kp + c] = j >= 0 && j < K ? xr[j] : (uint16_t)0;
    }
}

// The tokens of the tiled product: a wave per token, which holds P pieces of 16 columns per
// lane (the rest of a longer row is read twice): 4 up to 4096 columns, else 11. 4 | 11 | 16 pieces, us:
// 2048 tokens of 4096 columns 9.6 | 10.6 | - (this kernel); 300 tokens, 4096 x 11008, 49.0 | 47.7 | 48.2, 2048
// tokens 108 | 106 | 107, 300 of 4096 x 16384 60.7 | 60.0 | 58.9 (the whole product, tokens not in the
// caches). So only the mask of the weak columns is shared (one barrier). Codes and weak
// columns go in panels, and the blocks past the tokens lay the layer's weak weights out
// alike. 2048 tokens of 4096: 25 MB at 2.6 TB/s, each wave one chain of latencies; 300 tokens of
// 11008: 9.3 us.
template <bool WIDE, int P>
__global__ __launch_bounds__(256) void k_int8_token_panels(const QuantLayer L, int M)
{
    __shared__ DenseMask<WIDE> mask;
    const int tid = threadIdx.x, lane = tid & 63;
    const int K = L.K, kp = L.kp;
    const int rows = (M + 3) >> 2;  // blocks of tokens
    if ((int)blockIdx.x >= rows) {
        const PairLayer pl{nullptr, nullptr, nullptr, nullptr, L.ww, L.k};
        for (int64_t u = (int64_t)((int)blockIdx.x - rows) * 256 + tid; u < (int64_t)L.N * (kp >> 3);
             u += (int64_t)((int)gridDim.x - rows) * 256) {
            const int64_t row = u / (kp >> 3);
            const int p = (int)(u - row * (kp >> 3));
            *reinterpret_cast<half8_t*>(reinterpret_cast<char*>(L.wwp) + panel_at(row, kWeakPanel, 2 * kp, p)) =
                pair_weak(pl, row, 8 * p);
        }
        return;
    }
    const int64_t m = min((int)blockIdx.x * 4 + (tid >> 6), M - 1);  // (the last block's spare waves repeat the last token)
    const uint16_t* xr = L.x + m * K;
    const uint4* xp = reinterpret_cast<const uint4*>(xr);
    const int pieces = K >> 4;
    uint4 v[P][2];
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = lane + 64 * i;
        if (p < pieces) {
            v[i][0] = xp[2 * p];
            v[i][1] = xp[2 * p + 1];
        }
    }
    mask.template fill<256>(L.idx, L.k, K);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = lane + 64 * i;
        if (p < pieces) {
            top = mask.top(v[i][0], 2 * p, mask.top(v[i][1], 2 * p + 1, top));
        }
    }
    for (int p = lane + 64 * P; p < pieces; p += 64)
        top = mask.top(xp[2 * p], 2 * p, mask.top(xp[2 * p + 1], 2 * p + 1, top));
    const RowScale rs = row_scale(wave_max_u32(mask.both(top)));
    if (lane == 0)
        L.sx[m] = rs.scale;
    auto put = [&](int p, uint4 c) { *reinterpret_cast<uint4*>(L.x8 + panel_at(m, kGemmTokens, L.Kq, p)) = c; };
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int p = lane + 64 * i;
        if (p < pieces)
            put(p, code8x16(v[i][0], v[i][1], rs.factor));
    }
    for (int p = lane + 64 * P; p < pieces; p += 64)
        put(p, code8x16(xp[2 * p], xp[2 * p + 1], rs.factor));
    for (int p = pieces + lane; p < L.Kq >> 4; p += 64)
        put(p, make_uint4(0u, 0u, 0u, 0u));
    for (int c = lane; c < kp; c += 64) {
        const int j = c < L.k ? L.idx[c] : -1;
        *reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(L.xw) + panel_at(m, kGemmTokens, 2 * kp, c >> 3) + (c & 7) * 2) =
            j >= 0 && j < K ? xr[j] : (uint16_t)0;
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
// come from the caches), which saves the launch that would do it once: 4.1 against 7.6 us for
// one token of 768 x 768 in the two launches of the next form. That work grows with the
// tokens, so the form ends at four: 4096 x 4096, four tokens 10.0 us, five in two launches
// 9.7; 768 x 768: 7.4 and 7.6. Bound by the codes' stream: the seven linears of a 7B layer,
// one token, 203 MB in 42 .. 45 us (4.5 .. 4.8 TB/s; a copy reaches 5.15).
template <int M, bool WIDE>
__global__ __launch_bounds__(256) void k_int8_gemv(const DecBatch b)
{
    constexpr int R = kDecRows;
    __shared__ DenseMask<WIDE> mask;
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
    mask.template fill<256>(L.idx, k, K);
    RowScale rs[M];
    {
        uint32_t top[M];
#pragma unroll
        for (int m = 0; m < M; m++) {
            top[m] = 0;
            const uint4* xp = reinterpret_cast<const uint4*>(L.x + (int64_t)m * K);
            for (int p = tid; p < K >> 3; p += 256)
                top[m] = mask.top(xp[p], p, top[m]);
            top[m] = wave_max_u32(mask.both(top[m]));
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
                c = code8x16(v, w, rs[m].factor);
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
    // the codes' sums over the wave in integers, so that they are exact, the weak columns' in fp32
    float part[R][M], y[R][M];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float sw = L.s[brow + min(wave * R + r, nb - 1)];
#pragma unroll
        for (int m = 0; m < M; m++) {
            y[r][m] = (float)wave_sum_dpp(acc[r][m]) * (rs[m].scale * sw);
            part[r][m] = 0.0f;
        }
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
            const float v = k > 0 ? y[r][m] + wave_sum_dpp(part[r][m]) : y[r][m];
            if (lane == 0 && wave * R + r < nb)
                L.y[(int64_t)m * N + brow + wave * R + r] = f2h(v);
        }
}

// ------------------------------ few tokens: codes straight into the operands --

struct MfvLayer {
    const int8_t* q;
    const float* s;
    const uint16_t* ww;
    uint16_t* y;
    const int8_t* x8;
    const float* sx;
    const uint16_t* xw;
    int32_t N, K, Kq, k, kp, block0;
};
struct MfvBatch {
    MfvLayer L[kInt8MaxLayers];
    int32_t count, M;
};

constexpr int kMfvWaves = 4;  // waves that split K

// A block computes 16 RT rows for 16 MT tokens: v_mfma_i32_16x16x64_i8 with the codes as A
// (lane l: row l % 16, 16 columns 16 (l / 16) of a 64-column step) and the tokens as B,
// which k_int8_tokens has laid out in that order. Both come straight from memory into the
// operands, U steps ahead of their products. The waves' sums meet in LDS. Bound by the
// codes' stream: 16 tokens, 11008 x 4096, 45 MB in 12 us (3.8 TB/s).
template <int RT, int MT, int U>
__global__ __launch_bounds__(64 * kMfvWaves) void k_int8_mfv(const MfvBatch b)
{
    constexpr int W = kMfvWaves;
    __shared__ i32x4 part[W][RT * MT][64];
    int li = 0;
    for (int l = 1; l < b.count; l++)
        if ((int)blockIdx.x >= b.L[l].block0)
            li = l;
    const MfvLayer& L = b.L[li];
    const int N = L.N, K = L.K;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = ((int)blockIdx.x - L.block0) * 16 * RT, m0 = (int)blockIdx.y * 16 * MT;
    const int nb = min(N - row0, 16 * RT);
    const int r16 = lane & 15, g = lane >> 4;
    const __amdgpu_buffer_rsrc_t qr = bytes_rsrc(L.q + (int64_t)row0 * K, (int64_t)nb * K);
    // (the range holds the tiles that have tokens, others read zeros)
    const __amdgpu_buffer_rsrc_t xr = bytes_rsrc(L.x8, (int64_t)((b.M + 15) & ~15) * L.Kq);
    const int steps = (K + 63) >> 6;
    const int per = (steps + W - 1) / W;
    const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
    int qoff[RT];
#pragma unroll
    for (int r = 0; r < RT; r++)
        qoff[r] = min(16 * r + r16, nb - 1) * K + g * 16;
    struct Set {
        i32x4 c[U][RT], x[U][MT];
    };
    // steps past the wave's last are read out of range: zeros
    auto load = [&](int st, Set& v) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int dead = st + u < s1 ? 0 : kDeadLoad;
#pragma unroll
            for (int r = 0; r < RT; r++)
                v.c[u][r] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(qr, qoff[r] + (st + u) * 64 + dead, 0, 0));
#pragma unroll
            for (int m = 0; m < MT; m++)
                v.x[u][m] = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, (m0 + m * 16) * L.Kq + lane * 16 + (st + u) * 1024 + dead, 0, 0));
        }
    };
    i32x4 acc[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int m = 0; m < MT; m++)
            acc[r][m] = i32x4{0, 0, 0, 0};
    auto mul = [&](const Set& v) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[r][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v.c[u][r], v.x[u][m], acc[r][m], 0, 0, 0);
    };
    Set a, c;
    load(s0, a);
    for (int st = s0; st < s1; st += 2 * U) {
        load(st + U, c);
        mul(a);
        load(st + 2 * U, a);
        mul(c);
    }
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int m = 0; m < MT; m++)
            part[wave][r * MT + m][lane] = acc[r][m];
    __syncthreads();
    const PairLayer P{nullptr, nullptr, nullptr, nullptr, L.ww, L.k};
    for (int t = wave; t < RT * MT; t += W) {
        const int rb = 16 * (t / MT), m = m0 + 16 * (t % MT) + r16;
        if (rb >= nb)
            continue;
        i32x4 sum = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < W; w++)
            sum += part[w][t][lane];
        // lane l: token l % 16, rows 4 (l / 16) + r
        const int mc = min(m, b.M - 1);
        const float sm = L.sx[mc];
        i8_f4v out;
#pragma unroll
        for (int r = 0; r < 4; r++)
            out[r] = (float)sum[r] * (sm * L.s[row0 + min(rb + 4 * g + r, nb - 1)]);
        for (int e = 0; e < L.kp; e += 32) {
            const half8_t wv = pair_weak(P, row0 + min(rb + r16, nb - 1), e + 8 * g);
            const half8_t xv = *reinterpret_cast<const half8_t*>(L.xw + (int64_t)mc * L.kp + e + 8 * g);
            out = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, xv, out, 0, 0, 0);
        }
        if (m < b.M)
            store4(L.y + (int64_t)m * N, row0 + rb + 4 * g, N, out);
    }
}

// ----------------------------------------------------- more tokens: tiled GEMM --

struct GemmArgs8 {
    const int8_t* q;
    const float* s;
    uint16_t* y;
    const int8_t* x8;     // panels
    const float* sx;
    const uint16_t* xw;   // panels, [M][kp]
    const uint16_t* wwp;  // panels, [N][kp]
    int32_t M, N, K, Kq, kp;
    int32_t mblocks;
    int32_t whole;   // 256 x 256 tiles that stay whole
    int32_t splits;  // runs of stages that the blocks of one 256 x 128 tile take
    i32x4* sums;     // their sums, where splits > 1: [split][tile][wave][registers / 4][lane]
};


template <int FM, int FN, int WM, int WN>
struct Tile8 {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    static constexpr int STAGE = (BM + BN) * kGemmCols;
    static constexpr int DA = BM * 4 / NT, DB = BN * 4 / NT;  // 16-byte units per thread and stage
    static_assert(DA * NT == BM * 4 && DB * NT == BN * 4, "a stage must split evenly over the threads");
};

// BM tokens x BN rows per tile, both operands through LDS by direct-to-LDS loads in a ring
// of four stages of 64 columns, up to three stages ahead; operands are read from LDS one
// 32-column step ahead of their products, also across the stages: at a barrier the stage
// after the current one has landed too. The weak columns follow as stages of 32 fp16
// columns in the same ring, for which the sums have become fp32 and scaled. The rows are
// the matrix instruction's A, so that a lane ends with four consecutive outputs of one
// token; they leave through LDS in whole lines. PART: only the integer sums of stages
// c0 .. c1 - 1, to `sums`.
template <int FM, int FN, int WM, int WN, bool PART = false>
__device__ __forceinline__ void gemm_tile(const GemmArgs8& a, char* s0, char* s1, char* s2, char* s3, float* sm, float* sn,
                                          int m0, int n0, int c0, int c1, i32x4* sums = nullptr)
{
    using T = Tile8<FM, FN, WM, WN>;
    constexpr int BM = T::BM, BN = T::BN, DPW = T::DA + T::DB;
    const int M = a.M, N = a.N, K = a.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int l32 = lane & 31, h = lane >> 5;
    // this lane's pieces h and 2 + h of its rows
    const int p0 = stage_at(l32, h), p1 = stage_at(l32, 2 + h);
    const int abase = wm * FM * 2048, bbase = (BM + wn * 32 * FN) * kGemmCols;
    const int mv = min(BM, M - m0), nv = min(BN, N - n0);
    __amdgpu_buffer_rsrc_t xr = uniform_rsrc(a.x8 + (int64_t)m0 * a.Kq, (int64_t)BM * a.Kq);
    __amdgpu_buffer_rsrc_t qr = uniform_rsrc(a.q + (int64_t)n0 * K, (int64_t)nv * K);
    int xsrc[T::DA], qsrc[T::DB];
#pragma unroll
    for (int t = 0; t < T::DA; t++) {
        const int u = (wave * T::DA + t) * 64 + lane;
        xsrc[t] = stage_row(u) * kGemmCols + stage_piece(u) * 16;
    }
#pragma unroll
    for (int t = 0; t < T::DB; t++) {
        const int u = (wave * T::DB + t) * 64 + lane;
        qsrc[t] = min(stage_row(u), nv - 1) * K + stage_piece(u) * 16;
    }
    // (pieces past K of the last stage hold the next row's codes, or zeros past the
    // last row: the tokens' codes there are zeros)
    int end = c1, row_step = kGemmCols;
    auto dma = [&](int c, char* stage) {
        const int ox = c < end ? c * (BM * kGemmCols) : kDeadLoad, oq = c < end ? c * row_step : kDeadLoad;
#pragma unroll
        for (int t = 0; t < T::DA; t++)
            dma16_lds(xr, stage + (wave * T::DA + t) * 1024, xsrc[t] + ox);
#pragma unroll
        for (int t = 0; t < T::DB; t++)
            dma16_lds(qr, stage + BM * kGemmCols + (wave * T::DB + t) * 1024, qsrc[t] + oq);
    };
    i32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[i][f][r] = 0;
    i32x4 av[2][FM], bv[2][FN];
    auto read = [&](const char* stage, int set, int p) {
#pragma unroll
        for (int f = 0; f < FN; f++)
            bv[set][f] = *reinterpret_cast<const i32x4*>(stage + bbase + f * 2048 + p);
#pragma unroll
        for (int i = 0; i < FM; i++)
            av[set][i] = *reinterpret_cast<const i32x4*>(stage + abase + i * 2048 + p);
    };
    auto mul = [&](int set) {
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int f = 0; f < FN; f++)
                acc[i][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bv[set][f], av[set][i], acc[i][f], 0, 0, 0);
        // the other set's reads between these products
        constexpr int per = FM * FN / (FM + FN);
#pragma unroll
        for (int i = 0; i < FM + FN; i++) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, per, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, FM * FN - (FM + FN) * per, 0);
    };
    auto arrived = [&](int set) {  // the reads of a set are done
#pragma unroll
        for (int i = 0; i < FM; i++)
            asm volatile("" ::"v"(av[set][i]));
#pragma unroll
        for (int f = 0; f < FN; f++)
            asm volatile("" ::"v"(bv[set][f]));
    };
    // stage c is in cur and stage c + 1 in next, whole; stage c + 3 goes where c - 1 was
    auto step = [&](int c, const char* cur, const char* next, char* fill) {
        stage_barrier<DPW, 15>();
        dma(c + 3, fill);
        if (c < c1) {
            read(cur, 1, p1);
            mul(0);
            read(next, 0, p0);
            mul(1);
            arrived(1);  // before this wave lets cur be overwritten
        }
    };
    __syncthreads();  // the stages are free
    dma(c0, s0);
    dma(c0 + 1, s1);
    dma(c0 + 2, s2);
    for (int e = tid; e < BM + BN; e += T::NT) {
        if (e < BM)
            sm[e] = a.sx[m0 + min(e, mv - 1)];
        else
            sn[e - BM] = a.s[n0 + min(e - BM, nv - 1)];
    }
    stage_barrier<0>();
    read(s0, 0, p0);
    for (int c = c0; c < c1; c += 4) {
        step(c, s0, s1, s3);
        step(c + 1, s1, s2, s0);
        step(c + 2, s2, s3, s1);
        step(c + 3, s3, s0, s2);
    }
    arrived(0);
    stage_barrier<0>();  // the loads past the end have written their zeros
    if (PART) {
        sums += (int64_t)wave * (FM * FN * 4) * 64 + lane;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int f = 0; f < FN; f++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    sums[((i * FN + f) * 4 + q) * 64] =
                        i32x4{acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3]};
        return;
    }
    // the weak columns' first stages
    const int ws = a.kp >> 5;
    xr = uniform_rsrc(a.xw + (int64_t)m0 * a.kp, (int64_t)2 * BM * a.kp);
    // (panels of pn rows: this tile's are one or two, the second may lie past N)
    qr = uniform_rsrc(a.wwp + (int64_t)n0 * a.kp, (int64_t)2 * ((nv + kWeakPanel - 1) / kWeakPanel * kWeakPanel) * a.kp);
#pragma unroll
    for (int t = 0; t < T::DB; t++) {
        const int u = (wave * T::DB + t) * 64 + lane;
        const int row = stage_row(u), in = row & (kWeakPanel - 1);
        qsrc[t] = (row - in) * 2 * a.kp + in * kGemmCols + stage_piece(u) * 16;
    }
    end = ws;
    row_step = kWeakPanel * kGemmCols;
    if (ws > 0) {
        dma(0, s0);
        dma(1, s1);
    }
    // element r of a lane: row 8 (r / 4) + 4 h + r % 4, token l % 32
    i8_f16v out[FM][FN];
#pragma unroll
    for (int f = 0; f < FN; f++) {
        i8_f4v sr[4];
#pragma unroll
        for (int q = 0; q < 4; q++)
            sr[q] = *reinterpret_cast<const i8_f4v*>(&sn[wn * 32 * FN + 32 * f + 8 * q + 4 * h]);
#pragma unroll
        for (int i = 0; i < FM; i++) {
            const float sx = sm[wm * 32 * FM + 32 * i + l32];
#pragma unroll
            for (int r = 0; r < 16; r++)
                out[i][f][r] = (float)acc[i][f][r] * (sx * sr[r >> 2][r & 3]);
        }
    }
    for (int c = 0; c < ws; c++) {
        stage_barrier<0>();
        const char* const cur = c & 1 ? s1 : s0;
#pragma unroll
        for (int st = 0; st < 2; st++) {
            read(cur, st, st ? p1 : p0);
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int f = 0; f < FN; f++)
                    out[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, bv[st][f]),
                                                                       __builtin_bit_cast(half8_t, av[st][i]), out[i][f], 0,
                                                                       0, 0);
        }
        if (c + 2 < ws) {
            stage_barrier<0>();
            dma(c + 2, c & 1 ? s1 : s0);
        }
    }
    // 32 tokens x 32 FN rows of the wave at a time: token t's piece of 8 rows p in slot
    // p ^ (t % 8) of its 64 FN bytes
    static_assert(WM * WN / 2 * 32 * FN * 64 <= T::STAGE, "the waves' outputs pass through two stages");
    char* const mine = (wave < (WM * WN + 1) / 2 ? s2 : s3) + wave % ((WM * WN + 1) / 2) * (32 * FN * 64);
    constexpr int PIECES = 4 * FN;
#pragma unroll
    for (int i = 0; i < FM; i++) {
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const i8_f16v& o = out[i][f];
                *reinterpret_cast<uint2*>(mine + l32 * (64 * FN) + ((f * 4 + q) ^ (l32 & (PIECES - 1) & 7)) * 16 + h * 8) =
                    make_uint2(f2h(o[4 * q]) | ((uint32_t)f2h(o[4 * q + 1]) << 16),
                               f2h(o[4 * q + 2]) | ((uint32_t)f2h(o[4 * q + 3]) << 16));
            }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int e = 0; e < 32 * PIECES / 64; e++) {
            const int t = (e * 64 + lane) / PIECES, p = lane % PIECES;
            const uint4 v = *reinterpret_cast<const uint4*>(mine + t * (64 * FN) + (p ^ (t & (PIECES - 1) & 7)) * 16);
            const int m = m0 + wm * 32 * FM + 32 * i + t, n = n0 + wn * 32 * FN + 8 * p;
            if (m < M)
                store8(a.y + (int64_t)m * N, n, N, v);
        }
        asm volatile("" ::: "memory");
    }
}

// Tiles of 256 tokens x 256 rows, one per block, as many as fill whole rounds of the GPU;
// the rest as tiles of 256 x 128, two in place of one (blocks start in this order, so the
// small ones fill the last round). Where even the small ones leave CUs idle, `splits`
// blocks share each, and k_int8_gemm_sum adds their sums up.
// 2048 tokens, 11008 x 4096: 90 us, 2.05 POPS (the library's integer product of that shape,
// without scales and weak columns, 101; 2.14 POPS at 8192^3). The matrix cores are busy 66 %
// of the cycles at 1.7 GHz: products alone run at 2.2 GHz, loads, LDS and products together
// at what the card's power allows. 300 tokens, 4096 x 11008: 28 us and 8 for the sums; its
// 512 rows of tiles are 59 % full.
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_int8_gemm(const GemmArgs8 a)
{
    using T = Tile8<4, 2, 2, 4>;
    __shared__ __attribute__((aligned(1024))) char s0[T::STAGE];
    __shared__ __attribute__((aligned(1024))) char s1[T::STAGE];
    __shared__ __attribute__((aligned(1024))) char s2[T::STAGE];
    __shared__ __attribute__((aligned(1024))) char s3[T::STAGE];
    __shared__ float sm[T::BM], sn[T::BN];
    const int chunks = a.Kq / kGemmCols;
    if ((int)blockIdx.x < a.whole) {
        const int tile = xcd_place((int)blockIdx.x, a.whole);
        gemm_tile<4, 2, 2, 4>(a, s0, s1, s2, s3, sm, sn, (tile % a.mblocks) * T::BM, (tile / a.mblocks) * T::BN, 0, chunks);
        return;
    }
    const int part = xcd_place((int)blockIdx.x - a.whole, (int)gridDim.x - a.whole);
    if (a.splits == 1) {
        // parts 2 t and 2 t + 1: the halves of tile whole + t
        const int tile = a.whole + (part >> 1), n0 = (tile / a.mblocks) * T::BN + (part & 1) * (T::BN / 2);
        if (n0 < a.N)
            gemm_tile<2, 2, 4, 2>(a, s0, s1, s2, s3, sm, sn, (tile % a.mblocks) * T::BM, n0, 0, chunks);
        return;
    }
    const int tiles = ((int)gridDim.x - a.whole) / a.splits, tile = part % tiles, split = part / tiles;
    gemm_tile<2, 2, 4, 2, true>(a, s0, s1, s2, s3, sm, sn, (tile % a.mblocks) * T::BM, (tile / a.mblocks) * (T::BN / 2),
                                (int)((int64_t)chunks * split / a.splits), (int)((int64_t)chunks * (split + 1) / a.splits),
                                a.sums + (int64_t)part * kSumVectors);
}

// The splits' sums of one 32 x 32 piece, a wave each: scaled, the weak columns, stored.
__global__ __launch_bounds__(64) void k_int8_gemm_sum(const GemmArgs8 a, int tiles)
{
    const int lane = threadIdx.x, l32 = lane & 31, h = lane >> 5;
    const int piece = (int)blockIdx.x & 31, tile = (int)blockIdx.x >> 5;
    const int wave = piece >> 2, i = (piece >> 1) & 1, f = piece & 1;  // as in gemm_tile<2, 2, 4, 2>
    const int mb = (tile % a.mblocks) * 256 + (wave % 4) * 64 + 32 * i, nb = (tile / a.mblocks) * 128 + (wave / 4) * 64 + 32 * f;
    if (mb >= a.M || nb >= a.N)
        return;
    const i32x4* p = a.sums + (int64_t)tile * kSumVectors + (wave * 16 + (i * 2 + f) * 4) * 64 + lane;
    i32x4 sum[4];
#pragma unroll
    for (int q = 0; q < 4; q++)
        sum[q] = p[q * 64];
    for (int s = 1; s < a.splits; s++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            sum[q] += p[(int64_t)s * tiles * kSumVectors + q * 64];
    const int m = min(mb + l32, a.M - 1);
    const float sx = a.sx[m];
    i8_f16v out;
#pragma unroll
    for (int r = 0; r < 16; r++)
        out[r] = (float)sum[r >> 2][r & 3] * (sx * a.s[min(nb + 8 * (r >> 2) + 4 * h + (r & 3), a.N - 1)]);
    const char* xw = reinterpret_cast<const char*>(a.xw);
    const char* wwp = reinterpret_cast<const char*>(a.wwp);
    const int n = min(nb + l32, a.N - 1);
    for (int c = 0; c < a.kp >> 3; c += 2)
        out = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const half8_t*>(wwp + panel_at(n, kWeakPanel, 2 * a.kp, c + h)),
                                                     *reinterpret_cast<const half8_t*>(xw + panel_at(m, 256, 2 * a.kp, c + h)), out,
                                                     0, 0, 0);
    if (mb + l32 < a.M)
#pragma unroll
        for (int q = 0; q < 4; q++)
            store4(a.y + (int64_t)m * a.N, nb + 8 * q + 4 * h, a.N, i8_f4v{out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]});
}

constexpr int kCus = 256;

// How the tiles of a product are dealt out: whole 256 x 256 tiles, small ones (256 x 128),
// blocks per small one
struct GemmGrid {
    int64_t whole, small;
    int32_t splits;
    int64_t blocks() const { return whole + small * splits; }
};

GemmGrid gemm_grid(int64_t M, int64_t N, int64_t chunks)
{
    const int64_t mb = (M + kGemmTokens - 1) / kGemmTokens, large = mb * ((N + 255) / 256), small = mb * ((N + 127) / 128);
    if (2 * small <= kCus) {
        // fewer small tiles than half the CUs; a block keeps at least 8 stages
        int64_t sp = kCus / small;
        sp = sp < chunks / 8 ? sp : chunks / 8;
        if (sp > 1)
            return GemmGrid{0, small, (int32_t)sp};
    }
    const int64_t rest = large % kCus, whole = 2 * rest <= kCus ? large - rest : large;
    return GemmGrid{whole, 2 * (large - whole), 1};
}

constexpr int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Rows per block of the streaming product
int mfv_rows(int64_t M) { return M <= 32 ? 16 : 32; }

// Whether the codes stream past LDS. Above 64 tokens every further 64 read them again (from
// L2 and the memory's cache), but in one launch after the tokens', where the tiles split K
// and add the parts in a third: so where they would split, and the blocks together read at most 3
// 2^20 columns. Streamed against tiled, us: 768 x 768, 128 tokens 9.1 | 11.9, 1024: 12.6 | 12.7;
// 2731 x 1056, 128: 9.7 | 15.7, 1024: 25.1 | 28.5; 4096 x 4096, 128: 14.3 | 24.7, 256: 21.0 | 26.9,
// 384 (at the limit): 28.2 | 28.1, 512: 34.8 | 29.9; 4096 x 11008, 128: 27.6 | 36.5, 192: 44.0 |
// 37.0; without a split, 28672 x 1024, 128: 23.0 | 17.5.
bool streams(int64_t M, int64_t N, int64_t K)
{
    if (M <= 64)
        return true;
    const int64_t tiles = (M + kGemmTokens - 1) / kGemmTokens * ((N + 127) / 128);
    return M <= kInt8StreamMaxM && 2 * tiles <= kCus && (N + 31) / 32 * ((M + 63) / 64) * K <= 3 << 20;
}

}  // namespace

Int8Plan int8_plan(int64_t N, int64_t K, int32_t k, int64_t M)
{
    Int8Plan p{};
    if (M <= kInt8GemvMaxM)
        return p;
    p.Kq = up(K, kGemmCols);
    p.kp = (int32_t)up(k, 32);
    if (streams(M, N, K)) {
        p.off_sx = (size_t)(p.Kq * up(M, 16));
        p.off_xw = p.off_sx + (size_t)up(M * 4, 256);
        p.total = p.off_xw + (size_t)up(M * p.kp * 2, 256);
        return p;
    }
    const GemmGrid g = gemm_grid(M, N, p.Kq / kGemmCols);
    const int64_t Mp = up(M, kGemmTokens), Np = up(N, kWeakPanel);  // whole panels
    p.off_sx = (size_t)(p.Kq * Mp);
    p.off_xw = p.off_sx + (size_t)up(M * 4, 256);
    p.off_wwp = p.off_xw + (size_t)up(Mp * p.kp * 2, 256);
    p.off_sums = p.off_wwp + (size_t)up(Np * p.kp * 2, 256);
    p.total = p.off_sums + (g.splits > 1 ? (size_t)(g.splits * g.small) * kSumVectors * 16 : 0);
    return p;
}

bool int8_grid_fits(int64_t M, int64_t N, int64_t K)
{
    if (M <= kInt8GemvMaxM)
        return grid_fits((N + 4 * kDecRows - 1) / (4 * kDecRows), 256);
    if (streams(M, N, K))
        return grid_fits((N + mfv_rows(M) - 1) / mfv_rows(M), 64 * kMfvWaves);
    return grid_fits(M, 256) && grid_fits(gemm_grid(M, N, 1024).blocks(), 512);
}

hipError_t launch_pack_int8(const uint16_t* W, int64_t N, int64_t K, const int32_t* idx, int32_t k, int8_t* codes,
                            float* scales, uint16_t* ww, hipStream_t s)
{
    if (K <= kWideMask)
        hipLaunchKernelGGL(k_pack_int8<true>, dim3((unsigned)N), dim3(256), 0, s, W, (int)K, idx, k, codes, scales, ww);
    else
        hipLaunchKernelGGL(k_pack_int8<false>, dim3((unsigned)N), dim3(256), 0, s, W, (int)K, idx, k, codes, scales, ww);
    return hipGetLastError();
}

hipError_t launch_linear_int8(const Int8Desc* d, int count, int64_t M, void* const* ws, hipStream_t s)
{
    int64_t longest = 0;
    for (int l = 0; l < count; l++)
        longest = longest < d[l].K ? d[l].K : longest;
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
        auto launch = [&](auto wide) {
            constexpr bool WIDE = decltype(wide)::value;
            if (M == 1)
                hipLaunchKernelGGL((k_int8_gemv<1, WIDE>), grid, block, 0, s, b);
            else if (M == 2)
                hipLaunchKernelGGL((k_int8_gemv<2, WIDE>), grid, block, 0, s, b);
            else if (M == 3)
                hipLaunchKernelGGL((k_int8_gemv<3, WIDE>), grid, block, 0, s, b);
            else
                hipLaunchKernelGGL((k_int8_gemv<4, WIDE>), grid, block, 0, s, b);
        };
        if (longest <= kWideMask)
            launch(std::true_type{});
        else
            launch(std::false_type{});
        return hipGetLastError();
    }
    QuantBatch qb{};
    Int8Plan p[kInt8MaxLayers];
    for (int l = 0; l < count; l++) {
        p[l] = int8_plan(d[l].N, d[l].K, d[l].k, M);
        char* const w = static_cast<char*>(ws[l]);
        qb.L[l] = QuantLayer{d[l].x, d[l].idx, d[l].ww, reinterpret_cast<int8_t*>(w),
                             reinterpret_cast<float*>(w + p[l].off_sx), reinterpret_cast<uint16_t*>(w + p[l].off_xw), nullptr,
                             (int32_t)d[l].N, (int32_t)d[l].K, (int32_t)p[l].Kq, d[l].k, p[l].kp};
    }
    if (streams(M, d[0].N, d[0].K)) {
        MfvBatch b{};
        b.count = count;
        b.M = (int32_t)M;
        int64_t blocks = 0;
        const int rows = mfv_rows(M);
        for (int l = 0; l < count; l++) {
            const QuantLayer& q = qb.L[l];
            b.L[l] = MfvLayer{d[l].q, d[l].s, d[l].ww, d[l].y, q.x8, q.sx, q.xw, (int32_t)d[l].N, (int32_t)d[l].K, q.Kq, d[l].k,
                              q.kp, (int32_t)blocks};
            blocks += (d[l].N + rows - 1) / rows;
        }
        if (!grid_fits(blocks, 64 * kMfvWaves))
            return hipErrorInvalidConfiguration;
        const dim3 tokens((unsigned)M, (unsigned)count);
        if (longest <= 4096)
            hipLaunchKernelGGL((k_int8_tokens<true, 1>), tokens, dim3(256), 0, s, qb);
        else if (longest <= kWideMask)
            hipLaunchKernelGGL((k_int8_tokens<true, 3>), tokens, dim3(256), 0, s, qb);
        else
            hipLaunchKernelGGL((k_int8_tokens<false, 3>), tokens, dim3(256), 0, s, qb);
        const dim3 grid((unsigned)blocks, M <= 64 ? 1u : (unsigned)((M + 63) / 64)), block(64 * kMfvWaves);
        if (M <= 16)
            hipLaunchKernelGGL((k_int8_mfv<1, 1, 8>), grid, block, 0, s, b);
        else if (M <= 32)
            hipLaunchKernelGGL((k_int8_mfv<1, 2, 8>), grid, block, 0, s, b);
        else
            hipLaunchKernelGGL((k_int8_mfv<2, 4, 2>), grid, block, 0, s, b);
        return hipGetLastError();
    }
    if (count != 1 || !int8_grid_fits(M, d[0].N, d[0].K))  // before the first launch
        return hipErrorInvalidConfiguration;
    char* const w = static_cast<char*>(ws[0]);
    QuantLayer& q = qb.L[0];
    q.wwp = reinterpret_cast<uint16_t*>(w + p[0].off_wwp);
    const int64_t units = (d[0].N * (q.kp / 8) + 255) / 256;
    const dim3 panels((unsigned)((M + 3) / 4 + (units < 512 ? units : 512)));
    if (longest <= 4096)
        hipLaunchKernelGGL((k_int8_token_panels<true, 4>), panels, dim3(256), 0, s, q, (int)M);
    else if (longest <= kWideMask)
        hipLaunchKernelGGL((k_int8_token_panels<true, 11>), panels, dim3(256), 0, s, q, (int)M);
    else
        hipLaunchKernelGGL((k_int8_token_panels<false, 11>), panels, dim3(256), 0, s, q, (int)M);
    const GemmGrid g = gemm_grid(M, d[0].N, q.Kq / kGemmCols);
    const GemmArgs8 a{d[0].q, d[0].s, d[0].y, q.x8, q.sx, q.xw, q.wwp, (int32_t)M, (int32_t)d[0].N, (int32_t)d[0].K, q.Kq, q.kp,
                      (int32_t)((M + kGemmTokens - 1) / kGemmTokens), (int32_t)g.whole, g.splits,
                      reinterpret_cast<i32x4*>(w + p[0].off_sums)};
    hipLaunchKernelGGL(k_int8_gemm, dim3((unsigned)g.blocks()), dim3(512), 0, s, a);
    if (g.splits > 1)
        hipLaunchKernelGGL(k_int8_gemm_sum, dim3((unsigned)(32 * g.small)), dim3(64), 0, s, a, (int)g.small);
    return hipGetLastError();
}

}  // namespace owq
