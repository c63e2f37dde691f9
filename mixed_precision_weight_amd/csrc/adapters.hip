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
#include "owq_adapters.h"
#include "owq_pair_gemm.h"

namespace owq {

namespace {

constexpr int kShrinkWaves = 16;
constexpr int kShrinkFlight = 8;  // 32-column steps whose loads are in flight together

__global__ __launch_bounds__(64 * kShrinkWaves) void k_adapter_shrink(const uint16_t* __restrict__ x,
                                                                      const uint16_t* __restrict__ A,
                                                                      const int32_t* __restrict__ which,
                                                                      float* __restrict__ t, int M, int K, int count,
                                                                      int rank, int rpad)
{
    __shared__ float4 red[kShrinkWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, qd = lane >> 4;
    // The rank tiles of a token tile run on one XCD (blocks go to the 8 XCDs in
    // turn), so its x comes into one L2 once: 47 -> 25 us at 1000 tokens, rank 64,
    // K = 11008
    const int xcd = (int)blockIdx.x & 7, slot = (int)blockIdx.x >> 3;
    const int rt = rpad >> 4;
    const int tile = xcd + 8 * (slot / rt), r0 = (slot % rt) * 16;
    if (tile * 16 >= M)
        return;
    const int64_t m = (int64_t)tile * 16 + l16;
    const int64_t mc = m < M ? m : M - 1;
    int id = which[mc];
    if (m >= M || id < 0 || id >= count)
        id = -1;
    const uint16_t* xr = x + mc * K + 8 * qd;
    const int steps = K >> 5;
    const int per = (steps + kShrinkWaves - 1) / kShrinkWaves;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const bool live = r0 + l16 < rank;

    uint64_t left = __ballot(id >= 0) & 0xffffu;
    for (int d = 0; left != 0; d++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == a);
        if (d % (int)gridDim.y != (int)blockIdx.y)
            continue;
        const uint16_t* ar = A + ((int64_t)a * rank + min(r0 + l16, rank - 1)) * K + 8 * qd;
        float4_t acc[2] = {float4_t{0.0f, 0.0f, 0.0f, 0.0f}, float4_t{0.0f, 0.0f, 0.0f, 0.0f}};
        // (a tile of padding ranks only stores its zeros)
        for (int s = r0 < rank ? s0 : s1; s < s1; s += kShrinkFlight) {
            half8_t xv[kShrinkFlight], av[kShrinkFlight];
#pragma unroll
            for (int u = 0; u < kShrinkFlight; u++) {
                const int64_t o = (int64_t)min(s + u, s1 - 1) * 32;
                xv[u] = *reinterpret_cast<const half8_t*>(xr + o);
                av[u] = *reinterpret_cast<const half8_t*>(ar + o);
            }
#pragma unroll
            for (int u = 0; u < kShrinkFlight; u++)
                if (s + u < s1)  // wave-uniform
                    acc[u & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[u], av[u], acc[u & 1], 0, 0, 0);
        }
        const float4_t sum = acc[0] + acc[1];
        __syncthreads();  // the previous adapter's sums are no longer read
        red[wave][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (wave == 0) {
            float4 v = red[0][lane];
#pragma unroll
            for (int w = 1; w < kShrinkWaves; w++) {
                const float4 p = red[w][lane];
                v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
            }
            // D element r of lane l: token 4 (l / 16) + r, rank l % 16
            const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int tok = 4 * qd + r;
                if (__shfl(id, tok, 64) == a)
                    t[((int64_t)tile * 16 + tok) * rpad + r0 + l16] = live ? o[r] : 0.0f;
            }
        }
    }
}

// The adapters of 32 tokens (tk: this lane's) for 32 rows of each of the two row
// sets (n: this lane's): z[l][r] += their sum for D element r. CS 16-rank steps at a
// time: this lane's token's values are split into their operands once, and the
// weights of both row sets and all steps are loaded together, one adapter ahead of
// the products where the registers allow (AHEAD).
template <int CS, bool AHEAD, bool WIDE, int NL>
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
                    w.w[l][c] = adapter_weights<WIDE>(ad, id, N, n[l], c0 + 16 * c);
        };
        auto products = [&](int id, const Weights& w) {
            const float f = tk.id == id ? tk.f : 0.0f;
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
                    const float fr = __shfl(f, 8 * (r >> 2) + 4 * h + (r & 3), 64);
                    z[l][r] += fr != 0.0f ? fr * s[r] : 0.0f;
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
    if (!pair_gemm<FM, WN, S, true>(&a.L, a.x, M, N, a.K, m0, rows, acc))
        return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wn = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) % WN;
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int mt = m0 + 32 * i + l32;
        const AdapterToken tk = adapter_token<2, 32>(ad, min(mt, M - 1), mt < M, h);
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
                adapter_block<FM == 4 ? 1 : 4, FM == 1, true, NL>(ad, tk, N, nc, z);
            else
                adapter_block<1, false, false, NL>(ad, tk, N, nc, z);
#pragma unroll
            for (int l = 0; l < NL; l++) {
                const int n = rows[l0 + l] + wn * 32 + l32;
                uint16_t* y = a.y + (int64_t)(m0 + 32 * i + 4 * h) * N + n;
                int left = n < N ? M - (m0 + 32 * i + 4 * h) : 0;
                // opaque: shared between the row sets, the 16 comparisons below would
                // be kept in scalar registers and spill
                asm volatile("" : "+v"(left));
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int t = 8 * (r >> 2) + (r & 3);
                    if (t < left)
                        y[(int64_t)t * N] = f2h(acc[l0 + l][i][r] + z[l][r]);
                }
            }
        }
    }
}

}  // namespace

size_t adapter_workspace_bytes(int rank, int64_t M)
{
    return (size_t)M * adapter_rpad(rank) * sizeof(float);
}

hipError_t launch_adapter_shrink(const AdapterDesc& a, const uint16_t* x, int64_t M, int64_t K, hipStream_t s)
{
    const int rpad = adapter_rpad(a.rank);
    const int64_t tiles = (M + 15) / 16;
    const int rt = rpad / 16;
    // blocks per tile that share its distinct adapters: all 16 of a decode step's
    // tile side by side; with many tiles each walks its own (prompts: one or two)
    int64_t slots = 512 / (tiles * rt);
    slots = slots < 1 ? 1 : (slots > 16 ? 16 : slots);
    if (slots > M)
        slots = M;
    const int64_t nb = (tiles + 7) / 8 * 8 * rt;
    if (nb > INT32_MAX)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_adapter_shrink, dim3((unsigned)nb, (unsigned)slots), dim3(64 * kShrinkWaves), 0, s, x, a.A, a.which, a.t, (int)M, (int)K, a.count, a.rank, rpad);
    return hipGetLastError();
}

hipError_t launch_adapter_gemm(const LinearDesc& d, const AdapterDesc& ad, int64_t M, hipStream_t s)
{
    AdapterGemmArgs a{pair_layer(d), d.x, d.y, (int32_t)M, (int32_t)d.N, (int32_t)d.K, 1};
    return pair_tile(M, (d.N + 1) / 2, [&](auto fm, auto wn, auto sk) {
        using T = PairTile<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>;
        a.mblocks = (int32_t)((M + T::BM - 1) / T::BM);
        const int64_t nb = (int64_t)a.mblocks * ((d.N + 2 * T::BN - 1) / (2 * T::BN));
        if (nb > INT32_MAX)
            return hipErrorInvalidValue;
        hipLaunchKernelGGL((k_adapter_gemm<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>),
                           dim3((unsigned)nb), dim3(T::NT), 0, s, a, adapter_args(ad));
        return hipGetLastError();
    });
}

}  // namespace owq
