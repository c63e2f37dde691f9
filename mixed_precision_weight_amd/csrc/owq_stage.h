// owq_stage.h -- stages of LDS that direct-to-LDS loads fill ahead of a tiled product (gfx950).
#pragma once

#include "owq_device.h"

namespace owq {
namespace {

// A block's place among `blocks`: consecutive places share an XCD (blocks go to the eight
// XCDs in turn), so that neighbouring tiles meet in one L2.
__device__ __forceinline__ int xcd_place(int block, int blocks)
{
    const int per = blocks >> 3, even = per << 3;
    return block < even ? (block & 7) * per + (block >> 3) : block;
}

__device__ __forceinline__ void dma16_lds(__amdgpu_buffer_rsrc_t r, char* lds, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

// At most VM of the wave's loads are still in flight (and LGKM of its LDS accesses, 15: any),
// then the block's barrier. The builtin wait is one the compiler counts: it adds no wait of its
// own for the loads of other stages before a stage is read (an asm statement's wait does
// not spare that one).
template <int VM, int LGKM = 0>
__device__ __forceinline__ void stage_barrier()
{
    static_assert(VM < 64 && LGKM < 16, "fields of the instruction");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | 0x70 | (LGKM << 8) | ((VM >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Stages of 64 bytes per row, four 16-byte pieces: piece p of row r lies in line r / 2
// (128 bytes), slot (4 (r % 2) + p) ^ ((r / 4) % 4), so that 16 consecutive rows' pieces p
// fall on all 64 banks. Byte of a piece; row and piece of the 16-byte unit u of a stage.
__device__ __forceinline__ int stage_at(int r, int p)
{
    return (r >> 1) * 128 + ((((r & 1) << 2) | p) ^ ((r >> 2) & 3)) * 16;
}
__device__ __forceinline__ int stage_row(int u) { return (u >> 3) * 2 + ((((u & 7) ^ ((u >> 4) & 3))) >> 2); }
__device__ __forceinline__ int stage_piece(int u) { return ((u & 7) ^ ((u >> 4) & 3)) & 3; }

constexpr int kDeadLoad = 0x40000000;  // added to an offset: out of the buffer's range, zeros, nothing fetched

__device__ __forceinline__ __amdgpu_buffer_rsrc_t bytes_rsrc(const void* p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0,
                                             (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00020000);
}

// The same where the compiler cannot see that every lane has the same pointer (the
// descriptor of a load must be scalar, or the load becomes a loop over the lanes)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* p, int64_t bytes)
{
    const uint64_t u = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    const int n = __builtin_amdgcn_readfirstlane((int)(bytes < 0x7fffffff ? bytes : 0x7fffffff));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uintptr_t)(((uint64_t)hi << 32) | lo)), (short)0, n,
                                             0x00020000);
}

}  // namespace
}  // namespace owq
