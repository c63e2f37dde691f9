// owq_int8.h -- what the kernels of the integer form share (gfx950).
//
// The integer form: codes int8 [N][K], rint(w * (127 / t)) with t the row's largest
// |w| over its dense columns, 0 at the weak columns; scale t / 127 per row; the weak
// columns in fp16. A token is treated alike: its dense columns become int8 with the
// token's own scale, its weak columns stay fp16. The products of codes are exact in
// int32 (K 127^2 < 2^31 up to K = 65536).
#pragma once

#include "owq_device.h"
#include "owq_launch.h"
#include "owq_stage.h"

namespace owq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float i8_f16v __attribute__((ext_vector_type(16)));
typedef float i8_f4v __attribute__((ext_vector_type(4)));

// Scale and factor of a row whose largest dense magnitude has these bits: t / 127 and
// 127 / t, each one IEEE division; a row of zeros has both 0. An infinity or a NaN gives
// a scale that makes every output of the row NaN or infinite (its codes are 0).
struct RowScale {
    float scale, factor;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top)
{
    const float t = h2f((uint16_t)top);
    return RowScale{t / 127.0f, top == 0 ? 0.0f : (top >= 0x7c00u ? 0.0f : 127.0f / t)};
}

// The codes of four values (two pairs): each fp32 product v factor rounded half to even.
// Adding 1.5 2^23 rounds to integers and leaves the code in the low byte, for the fitted
// columns, where |v factor| <= 127 (1 + 2^-23). Weak columns' values may lie outside and
// give any byte: it is multiplied by 0.
__device__ __forceinline__ uint32_t code8x4(uint32_t a, uint32_t b, float factor)
{
    constexpr float kRound = 12582912.0f;
    const half2_t va = __builtin_bit_cast(half2_t, a), vb = __builtin_bit_cast(half2_t, b);
    // (a fused multiply-add with zero is the product rounded once, and takes fp16 operands)
    const uint32_t c0 = __builtin_bit_cast(uint32_t, __builtin_fmaf((float)va.x, factor, 0.0f) + kRound);
    const uint32_t c1 = __builtin_bit_cast(uint32_t, __builtin_fmaf((float)va.y, factor, 0.0f) + kRound);
    const uint32_t c2 = __builtin_bit_cast(uint32_t, __builtin_fmaf((float)vb.x, factor, 0.0f) + kRound);
    const uint32_t c3 = __builtin_bit_cast(uint32_t, __builtin_fmaf((float)vb.y, factor, 0.0f) + kRound);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(c3, c2, 0x0c0c0400u), __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u),
                                 0x05040100u);
}

__device__ __forceinline__ uint4 code8x16(uint4 a, uint4 b, float f)
{
    return make_uint4(code8x4(a.x, a.y, f), code8x4(a.z, a.w, f), code8x4(b.x, b.y, f), code8x4(b.z, b.w, f));
}

// The dense columns' mask in LDS, for the largest magnitude of a row: a 16-bit word per
// column (0x7fff, or 0 for a weak one: two instructions per pair of values) up to
// kWideMask columns, a bit per column (set: weak) above.
constexpr int kWideMask = 16384;
template <bool WIDE>
struct DenseMask {
    uint32_t w[WIDE ? kWideMask / 2 : 65536 / 32];

    // All threads of the block call it.
    template <int NT>
    __device__ __forceinline__ void fill(const int32_t* idx, int k, int K)
    {
        for (int i = threadIdx.x; i < (WIDE ? K >> 3 : K >> 7); i += NT)
            reinterpret_cast<uint4*>(w)[i] = WIDE ? make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu)
                                                  : make_uint4(0u, 0u, 0u, 0u);
        if (!WIDE && (int)threadIdx.x < ((K >> 5) & 3))
            w[((K >> 7) << 2) + threadIdx.x] = 0;
        __syncthreads();
        for (int c = threadIdx.x; c < k; c += NT) {
            const int j = idx[c];
            if (j >= 0 && j < K) {
                if (WIDE)
                    reinterpret_cast<uint16_t*>(w)[j] = 0;
                else
                    atomicOr(&w[j >> 5], 1u << (j & 31));
            }
        }
        __syncthreads();
    }

    // The largest of top and |v| over the dense ones of the 8 columns 8 p ..., as bits of
    // the magnitudes (which order like them, a NaN above infinity), two 16-bit maxima
    __device__ __forceinline__ uint32_t top(uint4 v, int p, uint32_t t) const
    {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
        uint32_t m[4];
        if (WIDE) {
            const uint4 q = reinterpret_cast<const uint4*>(w)[p];
            m[0] = q.x, m[1] = q.y, m[2] = q.z, m[3] = q.w;
        } else {
            const uint32_t b = reinterpret_cast<const uint8_t*>(w)[p];
#pragma unroll
            for (int e = 0; e < 4; e++)
                m[e] = ((b >> (2 * e)) & 1u ? 0u : 0x7fffu) | ((b >> (2 * e + 1)) & 1u ? 0u : 0x7fff0000u);
        }
        u16x2 r = __builtin_bit_cast(u16x2, t);
#pragma unroll
        for (int e = 0; e < 4; e++)
            r = __builtin_elementwise_max(r, __builtin_bit_cast(u16x2, d[e] & m[e]));
        return __builtin_bit_cast(uint32_t, r);
    }
    static __device__ __forceinline__ uint32_t both(uint32_t t) { return max(t & 0xffffu, t >> 16); }

    __device__ __forceinline__ bool weak(int j) const
    {
        return WIDE ? reinterpret_cast<const uint16_t*>(w)[j] == 0 : (w[j >> 5] >> (j & 31)) & 1u;
    }
};

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// Eight consecutive values of a row of n fp16 from column c on (those that lie in the row)
__device__ __forceinline__ void store8(uint16_t* row, int c, int n, uint4 v)
{
    typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));  // rows begin anywhere
    if (c + 8 <= n) {
        *reinterpret_cast<u4_any*>(row + c) = u4_any{v.x, v.y, v.z, v.w};
        return;
    }
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (c + e < n)
            row[c + e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
}

// Four of them, from a lane's sums
__device__ __forceinline__ void store4(uint16_t* row, int c, int n, i8_f4v v)
{
    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
    const uint32_t lo = f2h(v[0]) | ((uint32_t)f2h(v[1]) << 16), hi = f2h(v[2]) | ((uint32_t)f2h(v[3]) << 16);
    if (c + 4 <= n) {
        *reinterpret_cast<u2_any*>(row + c) = u2_any{lo, hi};
        return;
    }
    const uint32_t d[2] = {lo, hi};
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (c + e < n)
            row[c + e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
}

// Byte of the 16-byte piece p of a row in the panel layout: panels of `rows` rows, 64
// bytes of each row together (a stage of the tiled product; rows K bytes apart would
// keep the loads to 64-byte pieces all over the matrix).
__device__ __forceinline__ int64_t panel_at(int64_t row, int rows, int64_t row_bytes, int p)
{
    const int64_t panel = row / rows;
    return panel * rows * row_bytes + ((int64_t)(p >> 2) * rows + (row - panel * rows)) * 64 + (p & 3) * 16;
}

}  // namespace
}  // namespace owq
