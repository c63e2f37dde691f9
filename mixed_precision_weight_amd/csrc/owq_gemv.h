// owq_gemv.h -- what the vector-ALU decode kernels share (gfx950): the layout of
// the staged x and the reduction that ends their rows.
#pragma once

#include "owq_device.h"

namespace owq {
namespace {

constexpr int kChunkTiles = 2;  // 64-group tiles per K chunk (4096 columns)
constexpr int kNonTemporal = 2;  // buffer-load cache-policy bits: nt

// Staged x layout (uint4 units): [m][tile u][quad qd][lane l] for group g = 64 u + l,
// so a lane's four quads of a tile are at immediate offsets and the lanes of a
// wave read consecutive 16-byte words. The quads are 68 slots apart: the
// staging writes, which take consecutive 16-byte pieces of x (group g / 4, quad
// g % 4 per lane), then spread over all 64 banks.
constexpr int kQuadStride = 68;
__device__ __forceinline__ int xs_slot(int m, int T, int g, int qd)
{
    return (m * T + (g >> 6)) * (4 * kQuadStride) + qd * kQuadStride + (g & 63);
}

__device__ __forceinline__ float f_of(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t u_of(float v) { return __builtin_bit_cast(uint32_t, v); }

// Sum over the 64 lanes of 4 per-lane values at once: a v_permlane32_swap and a
// v_permlane16_swap step each add two values while halving their lane span, then
// a DPP reduction inside 16-lane rows. On return a[0] holds, in lanes
// 16 q .. 16 q + 15, the total of input reduced_index(q).
__device__ __forceinline__ void reduce4(float (&a)[4])
{
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {  // lanes 0-31 keep input i, lanes 32-63 input i + 2
        auto t = __builtin_amdgcn_permlane32_swap(u_of(a[i]), u_of(a[i + 2]), false, false);
        b[i] = f_of(t[0]) + f_of(t[1]);
    }
    auto t = __builtin_amdgcn_permlane16_swap(u_of(b[0]), u_of(b[1]), false, false);
    float v = f_of(t[0]) + f_of(t[1]);
    v += dpp_f<0xb1>(v);   // quad_perm [1,0,3,2]
    v += dpp_f<0x4e>(v);   // quad_perm [2,3,0,1]
    v += dpp_f<0x124>(v);  // row_ror:4
    v += dpp_f<0x128>(v);  // row_ror:8
    a[0] = v;
}
// quarter q of the lanes holds input (q & 1) + 2 (q >> 1)
__device__ __forceinline__ int reduced_index(int q) { return (q & 1) + ((q >> 1) << 1); }

}  // namespace
}  // namespace owq
