// owq_adapters.h -- the expand half of low-rank adapters inside the linear
// kernels' epilogues (gfx950):
//   y[m][i] += alpha_r sum_c B_r[i][c] t[m][c],   r = which[m], t[m] = A_r x[m]
// t is fp32 [M][rpad] (adapters.hip writes it, rpad = rank rounded up to 32, the
// padding zero); a token whose which[m] lies outside [0, count) has no adapter,
// and its row of t is not defined. Above 16 tokens the products take the tokens
// grouped by adapter: position p of that order is token order[p], and row p of t
// is that token's.
//
// On the matrix cores the tokens of a tile may belong to different adapters: the
// tile runs once per distinct adapter among them, into accumulators of its own,
// and each token takes the result of its own adapter only (a select, so a value
// that is not finite in one adapter cannot reach another request's row). t goes
// in as the sum of two fp16 values after scaling the token's row by a power of
// two (largest |t| in [2^14, 2^15)): 22 bits of the row's largest value, against
// which the fp32 sums and the fp16 output are the coarser roundings.
#pragma once

#include "owq_device.h"
#include "owq_launch.h"

namespace owq {
namespace {

struct AdapterArgs {
    const uint16_t* B;    // [count][N][rank]
    const float* alpha;   // [count]
    const int32_t* which; // [M]
    const float* t;       // [M][rpad]
    const int32_t* order; // [M], above 16 tokens
    int32_t count, rank, rpad;
};

inline AdapterArgs adapter_args(const AdapterDesc& a)
{
    return AdapterArgs{a.B, a.alpha, a.which, a.t, a.order, a.count, a.rank, adapter_rpad(a.rank)};
}

// A lane's view of one token's adapter: its index (-1: none), the exponent that
// t is scaled by and the factor that undoes it with alpha in it (0 without one).
struct AdapterToken {
    const float* t;
    int id, e;
    float f;
};

// The token m of this lane (live: it exists), row p of t; PARTS lanes share a token, at lane
// distances D, 2 D, ..., and lane part p reads values 8 p .. 8 p + 7 of every
// 8 PARTS of the row.
template <int PARTS, int D>
__device__ __forceinline__ AdapterToken adapter_token(const AdapterArgs& ad, int64_t m, int64_t p, bool live, int part)
{
    AdapterToken k;
    k.t = ad.t + p * ad.rpad;
    const int id = ad.which[m];
    k.id = live && id >= 0 && id < ad.count ? id : -1;
    float mx = 0.0f;
    if (k.id >= 0)
        for (int c = 8 * part; c < ad.rpad; c += 8 * PARTS)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(k.t + c + e);
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
            }
#pragma unroll
    for (int o = D; o < D * PARTS; o *= 2)
        mx = fmaxf(mx, __shfl_xor(mx, o, 64));
    // |t| < 2^49 for finite inputs, so no exponent here leaves fp32's range
    k.e = mx > 0.0f && mx < 0x1p100f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
    k.f = k.id >= 0 ? __builtin_amdgcn_ldexpf(ad.alpha[k.id], -k.e) : 0.0f;
    return k;
}

// This lane's MFMA A operand: values c .. c + 7 of its token's row as hi + lo
// (zero for a token of another adapter).
__device__ __forceinline__ void adapter_operand(const AdapterToken& k, int id, int c, half8_t& hi, half8_t& lo)
{
    const float4 a = *reinterpret_cast<const float4*>(k.t + c), b = *reinterpret_cast<const float4*>(k.t + c + 4);
    const bool on = k.id == id && id >= 0;  // (the row of a token without one is workspace: readable, not used)
    float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = on ? v[e] : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float s = __builtin_amdgcn_ldexpf(v[e], k.e);
        hi[e] = (_Float16)s;
        lo[e] = (_Float16)(s - (float)hi[e]);
    }
}

// Values c .. c + 7 of row B_id[i], zeros past the rank. PIECE: values per load, 8 or
// 4 where the rank is a multiple (pieces are then whole and aligned), else 1: single
// values cost the vector memory path as many cycles as whole pieces (8 tokens of 8
// requests, 4096 -> 4096 at rank 100: 38 us by ones, 24 by fours).
template <int PIECE>
__device__ __forceinline__ half8_t adapter_weights(const AdapterArgs& ad, int id, int64_t N, int64_t i, int c)
{
    // loads clamped to the row, values past it selected away: no branch per lane
    const uint16_t* row = ad.B + ((int64_t)id * N + i) * ad.rank;
    if constexpr (PIECE == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + min(c, ad.rank - 8));
        const bool on = c < ad.rank;
        return __builtin_bit_cast(half8_t, make_uint4(on ? v.x : 0u, on ? v.y : 0u, on ? v.z : 0u, on ? v.w : 0u));
    }
    if constexpr (PIECE == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + min(c, ad.rank - 4));
        const uint2 w = *reinterpret_cast<const uint2*>(row + min(c + 4, ad.rank - 4));
        const bool on = c < ad.rank, on4 = c + 4 < ad.rank;
        return __builtin_bit_cast(half8_t, make_uint4(on ? v.x : 0u, on ? v.y : 0u, on4 ? w.x : 0u, on4 ? w.y : 0u));
    }
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = row[min(c + e, ad.rank - 1)];
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = c + e < ad.rank ? v[e] : 0u;
    return __builtin_bit_cast(half8_t, make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                                                  v[6] | (v[7] << 16)));
}

}  // namespace
}  // namespace owq
