// owq_int8.h -- what the kernels of the 8-bit form share (gfx950).
//
// The 8-bit form: codes int8 [N][K], rint(w * (127 / t)) with t the row's largest
// |w| over its dense columns, 0 at the weak columns; scale t / 127 per row; the weak
// columns in fp16. A token is treated alike: its dense columns become int8 with the
// token's own scale, its weak columns stay fp16. The products of codes are exact in
// int32 (K 127^2 < 2^31 up to K = 65536).
#pragma once

#include "owq_device.h"
#include "owq_launch.h"

namespace owq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float i8_f16v __attribute__((ext_vector_type(16)));
typedef float i8_f4v __attribute__((ext_vector_type(4)));

// |v| of both halves as integers: they order like the values, and a NaN lies above
// infinity, so the largest of a row that holds one is a NaN
__device__ __forceinline__ uint32_t abs_bits_max(uint32_t pair, uint32_t top)
{
    const uint32_t lo = pair & 0x7fffu, hi = (pair >> 16) & 0x7fffu;
    return max(top, max(lo, hi));
}

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

// The code of one value: the fp32 product rounded half to even. Values outside the
// fitted columns may exceed the range (their codes are multiplied by 0): they are
// held to it, and a NaN becomes some code.
__device__ __forceinline__ int code8(float v, float factor)
{
    return (int)__builtin_amdgcn_fmed3f(rintf(v * factor), -127.0f, 127.0f);
}

__device__ __forceinline__ uint32_t code8x4(uint32_t a, uint32_t b, float f)
{
    const int c0 = code8(h2f((uint16_t)(a & 0xffffu)), f), c1 = code8(h2f((uint16_t)(a >> 16)), f);
    const int c2 = code8(h2f((uint16_t)(b & 0xffffu)), f), c3 = code8(h2f((uint16_t)(b >> 16)), f);
    return (uint32_t)(c0 & 0xff) | ((uint32_t)(c1 & 0xff) << 8) | ((uint32_t)(c2 & 0xff) << 16) | ((uint32_t)c3 << 24);
}

// Bits of the weak columns, K / 32 words in LDS. All threads of the block call it.
template <int NT>
__device__ __forceinline__ void weak_mask(uint32_t* mask, const int32_t* idx, int k, int K)
{
    for (int i = threadIdx.x; i < K >> 5; i += NT)
        mask[i] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < k; c += NT) {
        const int j = idx[c];
        if (j >= 0 && j < K)
            atomicOr(&mask[j >> 5], 1u << (j & 31));
    }
    __syncthreads();
}

// Largest |v| bits of 8 values whose weak columns have their bit set in w
__device__ __forceinline__ uint32_t top8(uint4 v, uint32_t w, uint32_t top)
{
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t lo = (w >> (2 * e)) & 1u ? 0u : d[e] & 0x7fffu;
        const uint32_t hi = (w >> (2 * e + 1)) & 1u ? 0u : (d[e] >> 16) & 0x7fffu;
        top = max(top, max(lo, hi));
    }
    return top;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

__device__ __forceinline__ void dma16_lds(__amdgpu_buffer_rsrc_t r, char* lds, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t bytes_rsrc(const void* p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0,
                                             (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00020000);
}

}  // namespace
}  // namespace owq
