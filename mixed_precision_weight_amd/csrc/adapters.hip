// adapters.hip -- the shrink half of low-rank adapters (gfx950):
//   t[m][c] = sum_j x[m][j] A_r[c][j],   r = which[m]
// for tokens of many requests at once, each with its own adapter or none. The
// expand half runs in the epilogue of the shared projection (owq_adapters.h), so
// the whole operator is two launches.
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
    const int r0 = (int)blockIdx.y * 16;
    const int64_t m = (int64_t)blockIdx.x * 16 + l16;
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
        if (d % (int)gridDim.z != (int)blockIdx.z)
            continue;
        const uint16_t* ar = A + ((int64_t)a * rank + min(r0 + l16, rank - 1)) * K + 8 * qd;
        float4_t acc[2] = {float4_t{0.0f, 0.0f, 0.0f, 0.0f}, float4_t{0.0f, 0.0f, 0.0f, 0.0f}};
        for (int s = s0; s < s1; s += kShrinkFlight) {
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
                    t[((int64_t)blockIdx.x * 16 + tok) * rpad + r0 + l16] = live ? o[r] : 0.0f;
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
    hipLaunchKernelGGL(k_adapter_shrink, dim3((unsigned)tiles, (unsigned)rt, (unsigned)slots),
                       dim3(64 * kShrinkWaves), 0, s, x, a.A, a.which, a.t, (int)M, (int)K, a.count, a.rank, rpad);
    return hipGetLastError();
}

}  // namespace owq
