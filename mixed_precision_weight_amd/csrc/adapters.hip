// adapters.hip -- the shrink half of low-rank adapters (gfx950):
//   t[m][c] = sum_j x[m][j] A_r[c][j],   r = which[m]
// for tokens of many requests at once, each with its own adapter or none. The
// expand half runs in the epilogue of the shared projection (owq_adapters.h: up to
// 16 tokens in the linear's decode kernels, above in k_adapter_gemm), so the whole
// operator is two launches.
//
// Work: A_r is rank x K fp16 (128 KB at rank 16, K = 4096), read once per tile of
// 16 tokens that uses it; the products are negligible. A block takes a tile of 16
// tokens, 16 ranks and every S-th of the distinct adapters among the tile's
// tokens; its 16 waves split K, so that even one token of one request has all
// loads of a row in flight at once, and add their sums in wave order in LDS
// (results do not depend on timing). v_mfma_f32_16x16x32_f16: A operand x (token
// l % 16, columns 8 (l / 16) .. + 7 of each 32), B operand the adapter's row
// l % 16, both read from memory in 16-byte pieces without staging: every byte is
// used by one lane once. Exact fp16 products, fp32 sums.
//
// Both halves run once per distinct adapter of a tile of tokens, so above 16 tokens
// the tiles are taken from an order in which the tokens of one adapter stand
// together (runs of 1024 tokens ordered each by itself, group_tokens; every block
// computes its run's order, the first of each tile stores it for the second half):
// 2000 tokens of 20 requests in turn, 4096 -> 4096, rank 64: 645 -> 153 us, 1000 of
// 3 (11008 -> 4096) 199 -> 155; where requests follow one another it costs 2 - 3 us.
//
// Measured: one token of rank 16, K = 4096, 7 us (which, then x and A: two memory
// latencies, the launch); 16 tokens of 15 requests 8 - 9; 1000 tokens of three requests
// one after the other, rank 64, K = 11008, 25: the 16 x 16 tile reads x once per 16
// ranks and A once per 16 tokens, 142 MB through the L2s, and each XCD fetches the
// adapters of its tiles, 50 MB for 26 MB of x and A. The products above 16 tokens: see
// owq_pair_gemm.h; 1000 tokens of 11008 -> 4096 in 111 us (810 TFLOP/s: 256 blocks,
// one wave per SIMD).
#include <algorithm>

#include "owq_adapters.h"
#include "owq_pair_gemm.h"

namespace owq {

namespace {

constexpr int kShrinkWaves = 16;
constexpr int kShrinkFlight = 8;  // 32-column steps whose loads are in flight together
constexpr int kBuckets = 256;     // that tokens are grouped by: the adapter's index modulo this

struct GroupScratch {
    int count[kShrinkWaves][kBuckets];  // tokens of a bucket in earlier waves
    int first[kBuckets];                // position of its first token
    int part[4];
    int token[16], id[16];              // the block's tile
};

// The tokens base .. base + kPairRun - 1, one per thread, in the order of their
// buckets, each bucket's in their own order; tokens without an adapter share the
// last one. Fills g.token and g.id (-1: no adapter) with the 16 tokens from position
// p0, those that exist.
__device__ __forceinline__ void group_tokens(GroupScratch& g, const int32_t* which, int M, int count, int base, int p0)
{
    static_assert(kPairRun == 64 * kShrinkWaves, "one token of a run per thread");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool on = tid < M - base;
    const int w = on ? which[base + tid] : -1;
    const int id = w < count ? w : -1;
    const int key = id >= 0 ? id & (kBuckets - 1) : kBuckets - 1;
#pragma unroll
    for (int i = 0; i < kShrinkWaves * kBuckets; i += kPairRun)
        (&g.count[0][0])[i + tid] = 0;
    uint64_t same = __ballot(on);  // this wave's tokens of the same bucket
#pragma unroll
    for (int b = 1; b < kBuckets; b *= 2) {
        const uint64_t set = __ballot((key & b) != 0);
        same &= (key & b) ? set : ~set;
    }
    const int before = (int)__popcll(same & ((1ull << lane) - 1));
    __syncthreads();
    if (on && before == 0)
        g.count[wave][key] = (int)__popcll(same);
    __syncthreads();
    int sum = 0, upto = 0;
    if (tid < kBuckets) {
#pragma unroll
        for (int w = 0; w < kShrinkWaves; w++) {
            const int c = g.count[w][tid];
            g.count[w][tid] = sum;
            sum += c;
        }
        upto = sum;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const int v = __shfl_up(upto, o, 64);
            upto += lane >= o ? v : 0;
        }
        if (lane == 63)
            g.part[wave] = upto;
    }
    __syncthreads();
    if (tid < kBuckets) {
        for (int w = 0; w < wave; w++)
            upto += g.part[w];
        g.first[tid] = upto - sum;
    }
    __syncthreads();
    const int at = g.first[key] + g.count[wave][key] + before - (p0 - base);
    if (on && at >= 0 && at < 16)
        g.token[at] = base + tid, g.id[at] = id;
    __syncthreads();
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t shrink_rsrc(const uint16_t* p, int64_t elems)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), (short)0, (int)(elems * 2), 0x00020000);
}

// Units (a tile's slot) are counted by this many tiles: whole rounds of the XCDs
__host__ __device__ constexpr int shrink_round(int tiles)
{
    return tiles < 8 ? tiles : (tiles + 7) / 8 * 8;
}

__global__ __launch_bounds__(64 * kShrinkWaves) void k_adapter_shrink(const uint16_t* __restrict__ x,
                                                                      const uint16_t* __restrict__ A,
                                                                      const int32_t* __restrict__ which,
                                                                      float* __restrict__ t, int32_t* __restrict__ order,
                                                                      int M, int K, int count, int rank, int rpad, int slots)
{
    __shared__ float4 red[kShrinkWaves][64];
    __shared__ GroupScratch group;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, qd = lane >> 4;
    // Blocks go to the 8 XCDs in turn: the rank tiles of a token tile run on one XCD,
    // so its x comes into one L2 once (47 -> 25 us at 1000 tokens, rank 64, K = 11008).
    // Token tiles go round the XCDs (with runs of tiles on one, 27 us became 46). The
    // slots of a tile stay on its XCD, too (33 us where they did not), but for few
    // tiles, whose adapters would all come through one XCD (8 tokens of 8 requests,
    // rank 100, K = 4096: 16.8 us on one, 9.5 on all)
    const int xcd = (int)blockIdx.x & 7, i = (int)blockIdx.x >> 3;
    const int rt = (rank + 15) >> 4, tiles = (M + 15) >> 4;
    const int unit = xcd + 8 * (i / rt), r0 = (i % rt) * 16;
    const int round = shrink_round(tiles);
    const int tile = unit % round, slot = unit / round;
    if (tile >= tiles || slot >= slots)
        return;
    // this lane's token, at position p of the order
    const int p = tile * 16 + l16;
    const int base = M > kMfvMaxM ? tile * 16 / kPairRun * kPairRun : 0;
    int m = min(p, M - 1), id;
    if (M > kMfvMaxM) {  // uniform
        group_tokens(group, which, M, count, base, tile * 16);
        const int at = m - tile * 16;  // (m < M: that position is filled)
        m = group.token[at], id = group.id[at];
        if (r0 == 0 && slot == 0 && threadIdx.x < 16 && p < M)
            order[p] = m;
    } else {
        id = which[m];
    }
    if (p >= M || id < 0 || id >= count)
        id = -1;
    const __amdgpu_buffer_rsrc_t xr = shrink_rsrc(x + (int64_t)base * K, (int64_t)min(M - base, kPairRun) * K);
    const int xo = (m - base) * K * 2 + 16 * qd;
    const int ao = min(r0 + l16, rank - 1) * K * 2 + 16 * qd;
    const int steps = K >> 5;
    const int per = (steps + kShrinkWaves - 1) / kShrinkWaves;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const bool live = r0 + l16 < rank;

    uint64_t left = __ballot(id >= 0) & 0xffffu;
    for (int d = 0; left != 0; d++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == a);
        if (d % slots != slot)
            continue;
        const __amdgpu_buffer_rsrc_t ar = shrink_rsrc(A + (int64_t)a * rank * K, (int64_t)rank * K);
        float4_t acc[2] = {float4_t{0.0f, 0.0f, 0.0f, 0.0f}, float4_t{0.0f, 0.0f, 0.0f, 0.0f}};
        // steps past the wave's end, and the tokens of other adapters, are read out of
        // range: zeros, nothing fetched (16 tokens of 15 requests: 11 -> 8.5 us)
        const int other = id == a ? 0 : kPairDead;
        half8_t xv[kShrinkFlight], av[kShrinkFlight];
        auto load = [&](int s, int u) {
            const int past = s + u < s1 ? 0 : kPairDead, o = past ? 0 : (s + u) * 64;
            xv[u] = __builtin_bit_cast(half8_t,
                                       __builtin_amdgcn_raw_buffer_load_b128(xr, pair_offset(xo, o, past, other), 0, 0));
            av[u] = __builtin_bit_cast(half8_t, __builtin_amdgcn_raw_buffer_load_b128(ar, pair_offset(ao, o, past, 0), 0, 0));
        };
        auto product = [&](int u) {
            acc[u & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[u], av[u], acc[u & 1], 0, 0, 0);
        };
#pragma unroll
        for (int u = 0; u < kShrinkFlight; u++)
            load(s0, u);
        int s = s0;
        for (; s + kShrinkFlight < s1; s += kShrinkFlight) {
#pragma unroll
            for (int u = 0; u < kShrinkFlight; u++) {
                product(u);
                load(s + kShrinkFlight, u);
            }
        }
#pragma unroll
        for (int u = 0; u < kShrinkFlight; u++)
            product(u);
        const float4_t sum = acc[0] + acc[1];
        __syncthreads();  // the previous adapter's sums are no longer read
        red[wave][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (wave == 0) {
            float4 v = red[0][lane];
#pragma unroll
            for (int w = 1; w < kShrinkWaves; w++) {
                const float4 q = red[w][lane];
                v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
            }
            // D element r of lane l: token 4 (l / 16) + r, rank l % 16
            const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int tok = 4 * qd + r;
                if (__shfl(id, tok, 64) == a) {
                    float* tr = t + ((int64_t)tile * 16 + tok) * rpad + r0 + l16;
                    tr[0] = live ? o[r] : 0.0f;
                    if (r0 + 16 >= rank && r0 + 16 < rpad)
                        tr[16] = 0.0f;
                }
            }
        }
    }
}

// The adapters of 32 tokens (tk: this lane's) for 32 rows of each of the two row
// sets (n: this lane's): z[l][r] += their sum for D element r. CS 16-rank steps at a
// time: this lane's token's values are split into their operands once, and the
// weights of both row sets and all steps are loaded together, one adapter ahead of
// the products where the registers allow (AHEAD).
template <int CS, bool AHEAD, int PIECE, int NL>
__device__ __forceinline__ void adapter_block(const AdapterArgs& ad, const AdapterToken& tk, int N, const int (&n)[NL],
                                              f32x16 (&z)[NL])
{
    const int h = (threadIdx.x & 63) >> 5;
    const uint64_t all = __ballot(tk.id >= 0) & 0xffffffffu;
    if (all == 0)
        return;
    for (int c0 = 8 * h; c0 < ad.rpad; c0 += 16 * CS) {
        half8_t th[CS], tl[CS];
#pragma unroll
        for (int c = 0; c < CS; c++)
            adapter_operand(tk, c0 + 16 * c < ad.rpad ? tk.id : -2, min(c0 + 16 * c, ad.rpad - 8), th[c], tl[c]);
        struct Weights {
            half8_t w[NL][CS];
        };
        auto load = [&](int id, Weights& w) {
#pragma unroll
            for (int l = 0; l < NL; l++)
#pragma unroll
                for (int c = 0; c < CS; c++)
                    w.w[l][c] = adapter_weights<PIECE>(ad, id, N, n[l], c0 + 16 * c);
        };
        auto products = [&](int id, const Weights& w) {
            // (by the tokens' adapters, not their factors: 0 times a NaN is NaN)
            const int mine = (int)((uint32_t)__ballot(tk.id == id) >> (4 * h));
#pragma unroll
            for (int l = 0; l < NL; l++) {
                f32x16 s;
#pragma unroll
                for (int r = 0; r < 16; r++)
                    s[r] = 0.0f;
#pragma unroll
                for (int c = 0; c < CS; c++) {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(th[c], w.w[l][c], s, 0, 0, 0);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(tl[c], w.w[l][c], s, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const float fr = __shfl(tk.f, 8 * (r >> 2) + 4 * h + (r & 3), 64);
                    const int on = __builtin_amdgcn_sbfe(mine, 8 * (r >> 2) + (r & 3), 1);  // 0 or all bits
                    z[l][r] += __builtin_bit_cast(float, __builtin_bit_cast(int, fr * s[r]) & on);
                }
            }
        };
        uint64_t left = all;
        auto next_id = [&]() {  // wave-uniform: the next distinct adapter, -1 after the last
            if (left == 0)
                return -1;
            const int id = __builtin_amdgcn_readlane(tk.id, __builtin_ctzll(left));
            left &= ~__ballot(tk.id == id);
            return id;
        };
        int id = next_id();
        if constexpr (AHEAD) {
            Weights wa, wb;
            load(id, wa);
            while (id >= 0) {
                const int nid = next_id();
                load(max(nid, 0), wb);
                products(id, wa);
                id = nid;
                if (id < 0)
                    break;
                const int mid = next_id();
                load(max(mid, 0), wa);
                products(id, wb);
                id = mid;
            }
        } else {
            while (id >= 0) {
                Weights w;
                load(id, w);
                products(id, w);
                id = next_id();
            }
        }
    }
}

struct AdapterGemmArgs {
    PairLayer L;
    const uint16_t* x;
    uint16_t* y;
    int32_t M, N, K, mblocks;
};

// More than 16 tokens: the pair product (owq_pair_gemm.h) over two runs of rows of
// the layer, the adapters added block by block before the one rounding (only one
// block's sums are carried through their loop, so no register is spilled).
template <int FM, int WN, int S>
__global__ __launch_bounds__(64 * WN * S) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_adapter_gemm(
    const AdapterGemmArgs a, const AdapterArgs ad)
{
    using T = PairTile<FM, WN, S>;
    const int M = a.M, N = a.N;
    const int m0 = ((int)blockIdx.x % a.mblocks) * T::BM;
    const int n0 = ((int)blockIdx.x / a.mblocks) * 2 * T::BN;
    const int rows[2] = {n0, n0 + T::BN};
    f32x16 acc[2][FM];
    if (!pair_gemm<FM, WN, S, true>(&a.L, a.x, ad.order, M, N, a.K, m0, rows, acc))
        return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wn = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) % WN;
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int mt = m0 + 32 * i + l32, mc = min(mt, M - 1);
        const int tok = ad.order[mc];
        const AdapterToken tk = adapter_token<2, 32>(ad, tok, mc, mt < M, h);
        const int dst = mt < M ? tok : -1;
        // both row sets together where the registers allow
        constexpr int NL = FM == 4 ? 1 : 2;
#pragma unroll
        for (int l0 = 0; l0 < 2; l0 += NL) {
            int nc[NL];
            f32x16 z[NL];
#pragma unroll
            for (int l = 0; l < NL; l++) {
                nc[l] = min(rows[l0 + l] + wn * 32 + l32, N - 1);
#pragma unroll
                for (int r = 0; r < 16; r++)
                    z[l][r] = 0.0f;
            }
            if ((ad.rank & 7) == 0)  // uniform
                adapter_block<FM == 4 ? 1 : FM == 2 ? 4 : 2, FM == 1, 8, NL>(ad, tk, N, nc, z);
            else if ((ad.rank & 3) == 0)
                adapter_block<1, false, 4, NL>(ad, tk, N, nc, z);
            else
                adapter_block<1, false, 1, NL>(ad, tk, N, nc, z);
#pragma unroll
            for (int l = 0; l < NL; l++) {
                const int n = rows[l0 + l] + wn * 32 + l32;
                uint16_t* y = a.y + n;
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int t = __shfl(dst, 8 * (r >> 2) + 4 * h + (r & 3), 64);
                    if (t >= 0 && n < N)
                        y[(int64_t)t * N] = f2h(acc[l0 + l][i][r] + z[l][r]);
                }
            }
        }
    }
}

}  // namespace

size_t adapter_workspace_bytes(int rank, int64_t M)
{
    return (size_t)M * (adapter_rpad(rank) * sizeof(float) + sizeof(int32_t));
}

namespace {

// blocks per tile that share its distinct adapters: the 16 of a decode step's tile
// side by side; grouped tiles hold one mostly, and the few that hold two would run
// on alone after the others (1000 tokens, rank 64: 43 us with one slot, 27 with two)
int64_t shrink_slots(int rank, int64_t M)
{
    const int64_t slots = 512 / ((M + 15) / 16 * ((rank + 15) / 16));
    return std::min(M, std::clamp<int64_t>(slots, 2, 16));
}

int64_t shrink_blocks(int rank, int64_t M)
{
    const int tiles = (int)((M + 15) / 16);
    return (shrink_round(tiles) * shrink_slots(rank, M) + 7) / 8 * 8 * ((rank + 15) / 16);
}

// f(tile as integral constants, blocks) for launch_adapter_gemm's choice of tile
template <typename F>
hipError_t adapter_gemm_tile(int64_t M, int64_t N, F f)
{
    return pair_tile(M, (N + 1) / 2, [&](auto fm, auto wn, auto sk) {
        using T = PairTile<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>;
        const int64_t nb = (M + T::BM - 1) / T::BM * ((N + 2 * T::BN - 1) / (2 * T::BN));
        return grid_fits(nb, T::NT) ? f(fm, wn, sk, nb) : hipErrorInvalidConfiguration;
    });
}

}  // namespace

bool adapter_shrink_grid_fits(int rank, int64_t M) { return grid_fits(shrink_blocks(rank, M), 64 * kShrinkWaves); }

bool adapter_gemm_grid_fits(int64_t M, int64_t N)
{
    return adapter_gemm_tile(M, N, [](auto, auto, auto, int64_t) { return hipSuccess; }) == hipSuccess;
}

hipError_t launch_adapter_shrink(const AdapterDesc& a, const uint16_t* x, int64_t M, int64_t K, hipStream_t s)
{
    if (!adapter_shrink_grid_fits(a.rank, M))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(k_adapter_shrink, dim3((unsigned)shrink_blocks(a.rank, M)), dim3(64 * kShrinkWaves), 0, s, x, a.A,
                       a.which, a.t, a.order, (int)M, (int)K, a.count, a.rank, adapter_rpad(a.rank),
                       (int)shrink_slots(a.rank, M));
    return hipGetLastError();
}

hipError_t launch_adapter_gemm(const LinearDesc& d, const AdapterDesc& ad, int64_t M, hipStream_t s)
{
    AdapterGemmArgs a{pair_layer(d), d.x, d.y, (int32_t)M, (int32_t)d.N, (int32_t)d.K, 1};
    return adapter_gemm_tile(M, d.N, [&](auto fm, auto wn, auto sk, int64_t nb) {
        using T = PairTile<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>;
        a.mblocks = (int32_t)((M + T::BM - 1) / T::BM);
        hipLaunchKernelGGL((k_adapter_gemm<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>),
                           dim3((unsigned)nb), dim3(T::NT), 0, s, a, adapter_args(ad));
        return hipGetLastError();
    });
}

}  // namespace owq
