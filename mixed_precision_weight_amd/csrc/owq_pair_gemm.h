// owq_pair_gemm.h -- matrix-core product of a tile of tokens with two sets of
// packed rows (gfx950), shared by the gated block (rows of gate and of up) and the
// linear with low-rank adapters (two runs of rows of one layer):
//   acc[l][i] = x[m0 ..] W_l^T for 32 FM tokens and 32 rows per wave of set l = 0, 1
//
// A wave holds all the block's tokens and 32 rows of each set, so every code group
// is decoded once per block, straight into the B operand of v_mfma_f32_32x32x16_f16
// (lane l: row l % 32, group 2 chunk + l / 32; the 32 exact q - z of a group feed
// four steps). x goes by direct-to-LDS loads three chunks of 64 columns deep, codes
// two chunks ahead in registers, one barrier per chunk. S groups of WN waves split
// K (stages of their own, all in step) and add up in LDS at the end: where tokens
// and rows give few waves, and where K is long, the chain of chunks is what counts.
#pragma once

#include <type_traits>

#include "owq_decode.h"
#include "owq_device.h"
#include "owq_launch.h"

namespace owq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float pair_f4 __attribute__((ext_vector_type(4)));

struct PairLayer {
    const uint32_t* q;
    const uint16_t* s;
    const uint8_t* z;
    const int32_t* idx;
    const uint16_t* ww;
    int32_t k;
};

inline PairLayer pair_layer(const LinearDesc& d)
{
    // with no weak columns, the weak arrays point at valid memory (never used)
    return PairLayer{d.q, d.s, d.z, d.k > 0 ? d.idx : reinterpret_cast<const int32_t*>(d.x), d.k > 0 ? d.ww : d.s, d.k};
}

__device__ __forceinline__ half8_t pair_h8(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(half8_t, make_uint4(a, b, c, d));
}

__device__ __forceinline__ void pair_dma(__amdgpu_buffer_rsrc_t r, char* lds, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

template <int FM, int WN, int S>
struct PairTile {
    static constexpr int NT = 64 * WN * S;
    static constexpr int BM = 32 * FM;
    static constexpr int BN = 32 * WN;  // rows of each set
    static constexpr int STAGE = BM * 128;
    static constexpr int DPW = STAGE / 16 / (64 * WN);
    // What a K group's waves hold at the end (not ONE): OWN 32-token blocks from block
    // kg OWN on where the groups share them, else, of four groups, tokens 8 kg ..
    // 8 kg + 7 of the one block in registers 0 .. 3
    static constexpr int SHARE = S > 1 && FM % S == 0 ? S : 1;
    static constexpr int OWN = FM / SHARE;
    static_assert(STAGE % (16 * 64 * WN) == 0, "a stage must split evenly over a group's threads");
    static_assert(S == 1 || (SHARE * WN * 4096 <= S * STAGE && (S - 1) * WN * 4096 <= S * STAGE), "the blocks handed over fit a stage set");
};

// w_weak[row][c .. c + 7] as an operand, zeros past the weak columns (c: a multiple of
// 8). The piece is loaded whole, clamped to the row, and moved down where it reaches
// past the end: no branch per lane, at whose end the loads would be waited for. (Value
// by value 1000 tokens, 2 x 86 columns took 4 us more.)
__device__ __forceinline__ half8_t pair_weak(const PairLayer& P, int64_t row, int c)
{
    typedef uint16_t u16x8 __attribute__((ext_vector_type(8), aligned(2)));  // any address
    const uint16_t* w = P.ww + row * P.k;
    if (P.k >= 8) {  // uniform
        uint4 u = __builtin_bit_cast(uint4, *reinterpret_cast<const u16x8*>(w + min(c, P.k - 8)));
        if ((P.k & 7) != 0) {  // uniform
            const uint32_t past = (uint32_t)max(c - (P.k - 8), 0), bits = 16 * (past & 1);
            u = make_uint4(__builtin_amdgcn_alignbit(u.y, u.x, bits), __builtin_amdgcn_alignbit(u.z, u.y, bits),
                           __builtin_amdgcn_alignbit(u.w, u.z, bits), u.w >> bits);
            if (past & 2)
                u = make_uint4(u.y, u.z, u.w, 0u);
            if (past & 4)
                u = make_uint4(u.z, u.w, 0u, 0u);
        }
        return __builtin_bit_cast(half8_t, c < P.k ? u : make_uint4(0u, 0u, 0u, 0u));
    }
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const uint32_t one = w[min(e, P.k - 1)];
        u[e] = c == 0 && e < P.k ? one : 0u;
    }
    return pair_h8(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
}

// Byte offset of a load that is put out of the buffer's range (zeros, nothing fetched)
// by any of its marks, each 0 or kPairDead: together they are one bit, so the sum stays
// an int for offsets below 2^30.
constexpr int kPairDead = 0x40000000;
__host__ __device__ constexpr int pair_offset(int start, int step, int dead, int dead2)
{
    return start + step + (dead | dead2);
}

// Tokens whose order is given are permuted within runs of this many, so that a run's
// rows of x stay within 32-bit offsets.
constexpr int kPairRun = 1024;
// (the last token of a run of the longest rows, the last piece, both marks; a constant
// expression does not overflow)
static_assert(pair_offset((kPairRun - 1) * 65536 * 2 + 112, 1023 * 128, kPairDead, kPairDead) > 0, "offsets are int");

// The sums of one wave of the block (its rows: row set l starts at n0[l], which may
// lie past N; tokens from m0; ONE: both sets are rows of the one layer L[0], and
// row m of the product is token order[m]). At the end the K groups hold shares (see
// PairTile), or with ONE group 0 holds all: returns false for the others' waves, which
// are done.
template <int FM, int WN, int S, bool ONE>
__device__ __forceinline__ bool pair_gemm(const PairLayer* L, const uint16_t* x, const int32_t* order, int M, int N, int K,
                                          int m0, const int (&n0)[2], f32x16 (&acc)[2][FM])
{
    using T = PairTile<FM, WN, S>;
    constexpr int BM = T::BM, BN = T::BN, STAGE = T::STAGE, DPW = T::DPW;
    __shared__ __attribute__((aligned(1024))) char xs0[S][STAGE];
    __shared__ __attribute__((aligned(1024))) char xs1[S][STAGE];
    __shared__ __attribute__((aligned(1024))) char xs2[S][STAGE];

    const int G = K >> 5;
    const int nchunks = (G + 1) >> 1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wid % WN, kg = wid / WN;  // row wave in the block, K group
    const int per = (nchunks + S - 1) / S;
    const int c0 = kg * per, c1 = min(nchunks, c0 + per);  // this group's chunks (none: it only keeps the barriers)
    const int l32 = lane & 31, h = lane >> 5;
    const int mv = min(BM, M - m0);

    static_assert(kPairRun % BM == 0, "a tile lies in one run");
    const int base = ONE ? m0 / kPairRun * kPairRun : m0;
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(x) + (int64_t)base * K, (short)0, (ONE ? min(kPairRun, M - base) : mv) * K * 2, 0x00020000);
    // row of x, relative to the base, of the tile's token t (past M: the last one)
    auto token = [&](int t) {
        if constexpr (ONE)
            return order[m0 + min(t, mv - 1)] - base;
        else
            return min(t, mv - 1);
    };
    // row sets: first row and rows (a set past N reads the last row; never stored)
    int nb[2], nv[2];
    __amdgpu_buffer_rsrc_t qr[2];
#pragma unroll
    for (int l = 0; l < 2; l++) {
        nb[l] = min(n0[l], N - 1);
        nv[l] = min(BN, N - nb[l]);
        qr[l] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(L[ONE ? 0 : l].q) + (int64_t)nb[l] * G * 3, (short)0,
                                                  nv[l] * G * 12, 0x00020000);
    }

    // DMA unit u: token u / 8, slot u % 8 holds piece slot ^ (token & 7); with an
    // odd group count the last chunk's second group is read out of range (zeros),
    // as are the chunks past the group's end
    const int last = nchunks - 1;
    const bool odd_tail = (G & 1) != 0;
    int xsrc[DPW], xdead[DPW];
#pragma unroll
    for (int t = 0; t < DPW; t++) {
        const int u = (wn * DPW + t) * 64 + lane;
        const int row = u >> 3, piece = (u & 7) ^ (row & 7);
        xsrc[t] = token(row) * K * 2 + piece * 16;
        xdead[t] = (odd_tail && piece >= 4) ? kPairDead : 0;
    }
    auto dma = [&](int c, char* stage) {
        const int cc = min(c, last);
        const int dead = c >= c1 ? kPairDead : 0;
#pragma unroll
        for (int t = 0; t < DPW; t++)
            pair_dma(xr, stage + (wn * DPW + t) * 1024, pair_offset(xsrc[t], cc * 128, cc == last ? xdead[t] : 0, dead));
    };

    // weak columns go in turns of 64; the lane's columns of this group's first turn are
    // loaded ahead, and so are the row steps where the registers allow. BOTH: the two
    // layers' turns run side by side
    constexpr bool BOTH = FM < 4 && !ONE;
    auto weak_column = [&](const PairLayer& P, int it) {
        const int j = P.idx[min(it * 64 + lane, P.k - 1)];
        return j >= 0 && j < K ? j : 0;
    };
    int jfirst[2];
#pragma unroll
    for (int l = 0; l < (BOTH ? 2 : 1); l++)
        jfirst[l] = FM < 4 && kg * 64 < L[l].k ? weak_column(L[l], kg) : 0;

    // this lane's row of each set, relative to the set's first
    int row[2];
    ZeroSub zs[2];
#pragma unroll
    for (int l = 0; l < 2; l++) {
        row[l] = min(wn * 32 + l32, nv[l] - 1);
        zs[l] = make_zero_sub((uint32_t)L[ONE ? 0 : l].z[nb[l] + row[l]]);
    }
    float sc[2];
    auto load_scales = [&]() {
#pragma unroll
        for (int l = 0; l < 2; l++)
            sc[l] = h2f(L[ONE ? 0 : l].s[nb[l] + row[l]]);
    };
    if constexpr (FM < 4)
        load_scales();
    typedef u32x3 QRegs[2];
    auto load_q = [&](int c, QRegs& cw) {
        const int g = min(2 * min(c, last) + h, G - 1);
        const int dead = c >= c1 ? kPairDead : 0;
#pragma unroll
        for (int l = 0; l < 2; l++)
            cw[l] = __builtin_amdgcn_raw_buffer_load_b96(qr[l], (row[l] * G + g) * 12 + dead, 0, 0);
    };

    const Magic mg = make_magic();
#pragma unroll
    for (int l = 0; l < 2; l++)
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[l][i][r] = 0.0f;

    const int arow = l32 * 128;
    int aoff[4];
#pragma unroll
    for (int st = 0; st < 4; st++)
        aoff[st] = ((h * 4 + st) ^ (l32 & 7)) * 16;
    auto step = [&](int c, const char* cur, char* nxt2, const QRegs& qc, QRegs& q2) {
        // x of chunk c has arrived once at most the codes of c and x and codes of
        // c + 1 remain; after the barrier every wave's has, and every wave is done
        // with the stage chunk c + 2 goes to
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(4 + DPW) : "memory");
        dma(c + 2, nxt2);
        load_q(c + 2, q2);
        if (c < c1) {  // wave-uniform
            half8_t av[4][FM];
#pragma unroll
            for (int st = 0; st < 4; st++)
#pragma unroll
                for (int i = 0; i < FM; i++)
                    av[st][i] =
                        __builtin_bit_cast(half8_t, *reinterpret_cast<const uint4*>(cur + arow + i * 32 * 128 + aoff[st]));
#pragma unroll
            for (int l = 0; l < 2; l++) {
                uint32_t p[16];
                decode_group(qc[l].x, qc[l].y, qc[l].z, mg, zs[l], p);
#pragma unroll
                for (int st = 0; st < 4; st++) {
                    const half8_t bv = pair_h8(p[4 * st], p[4 * st + 1], p[4 * st + 2], p[4 * st + 3]);
#pragma unroll
                    for (int i = 0; i < FM; i++)
                        acc[l][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[st][i], bv, acc[l][i], 0, 0, 0);
                }
            }
        }
    };

    QRegs qa, qb, qc3;
    dma(c0, xs0[kg]);
    load_q(c0, qa);
    asm volatile("" ::: "memory");
    dma(c0 + 1, xs1[kg]);
    load_q(c0 + 1, qb);
    asm volatile("" ::: "memory");
    for (int c = c0; c < c0 + per; c += 3) {  // the same trip count in every group
        step(c, xs0[kg], xs2[kg], qa, qc3);
        step(c + 1, xs1[kg], xs0[kg], qb, qa);
        step(c + 2, xs2[kg], xs1[kg], qc3, qb);
    }
    // no load may write LDS after this point (reused below, and the block may end)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // row steps (of every K group's sums), then the weak columns, 64 at a time: x at
    // their indices is gathered once per block into a stage, laid out as a chunk of x
    // (a gather reads a cache line per value, and the row waves need the same ones),
    // and meets w_weak as four 16-deep steps. The K groups take the 64s in turn. The
    // loads of a turn are issued before any of them is waited for (2731 x 1056 at 77
    // tokens 12.8 -> 10.8 us, 11008 x 4096 at 64 32.3 -> 29.1 against loads as they are
    // needed, one layer after the other).
    if constexpr (FM == 4)
        load_scales();
#pragma unroll
    for (int l = 0; l < 2; l++)
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[l][i][r] *= sc[l];
    constexpr int TW = BM / WN, TB = FM == 4 || ONE ? 8 : TW;  // tokens of a wave; of a batch of loads
    int tokens = 0;                                     // lane t: the row of x of this wave's token t
    if (lane < TW)
        tokens = token(wn + WN * lane);
    auto gather = [&](int j, int t0, uint32_t (&v)[TB]) {
#pragma unroll
        for (int t = 0; t < TB; t++)
            v[t] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                xr, 2 * j, 2 * K * __builtin_amdgcn_readlane(tokens, t0 + t), 0);
    };
    auto store = [&](char* stage, bool on, int t0, const uint32_t (&v)[TB]) {
#pragma unroll
        for (int t = 0; t < TB; t++) {
            const int tok = wn + WN * (t0 + t);
            *reinterpret_cast<uint16_t*>(stage + tok * 128 + (((lane >> 3) ^ (tok & 7)) << 4) + 2 * (lane & 7)) =
                (uint16_t)(on ? v[t] : 0u);
        }
    };
    auto weights = [&](const PairLayer& P, int set, int c, half8_t (&w)[4]) {
#pragma unroll
        for (int st = 0; st < 4; st++)
            w[st] = pair_weak(P, nb[set] + row[set], c + 32 * h + 8 * st);
    };
    auto product = [&](f32x16 (&sum)[FM], const char* stage, int st, const half8_t& w) {
#pragma unroll
        for (int i = 0; i < FM; i++)
            sum[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(half8_t, *reinterpret_cast<const uint4*>(stage + arow + i * 32 * 128 + aoff[st])), w,
                sum[i], 0, 0, 0);
    };
    if constexpr (BOTH) {
        char* const stage[2] = {xs0[kg], xs1[kg]};
        const int passes = (max(L[0].k, L[1].k) + 63) >> 6;
        for (int p0 = 0; p0 < passes; p0 += S) {  // the same trip count in every group
            const int it = p0 + kg;
            half8_t w[2][4];
            uint32_t v[2][TB];
#pragma unroll
            for (int l = 0; l < 2; l++)
                if (it * 64 < L[l].k) {  // wave-uniform
                    weights(L[l], l, it * 64, w[l]);
                    gather(p0 == 0 ? jfirst[l] : weak_column(L[l], it), 0, v[l]);
                }
            __syncthreads();  // the stages are no longer read
#pragma unroll
            for (int l = 0; l < 2; l++)
                if (it * 64 < L[l].k)
                    store(stage[l], it * 64 + lane < L[l].k, 0, v[l]);
            __syncthreads();
#pragma unroll
            for (int l = 0; l < 2; l++)
                if (it * 64 < L[l].k)
#pragma unroll
                    for (int st = 0; st < 4; st++)
                        product(acc[l], stage[l], st, w[l][st]);
        }
    } else {
        char* const stage = xs0[kg];
#pragma unroll
        for (int l = 0; l < (ONE ? 1 : 2); l++) {
            const PairLayer& P = L[l];
            for (int p0 = 0; p0 * 64 < P.k; p0 += S) {
                const int it = p0 + kg;
                const bool mine = it * 64 < P.k;  // wave-uniform
                const int j = FM < 4 && p0 == 0 ? jfirst[0] : (mine ? weak_column(P, it) : 0);
                constexpr bool EARLY = FM < 4;  // (128 tokens fill the registers: 344 us at 2048, else 340)
                constexpr int SETS = ONE ? 2 : 1;
                half8_t w[SETS][4];
                uint32_t v[TB];
                if (mine) {
                    if constexpr (EARLY)
#pragma unroll
                        for (int q = 0; q < SETS; q++)
                            weights(P, l + q, it * 64, w[q]);
                    gather(j, 0, v);
                }
                __syncthreads();  // the stage is no longer read
                if (mine) {
                    const bool on = it * 64 + lane < P.k;
                    store(stage, on, 0, v);
#pragma unroll 1
                    for (int t0 = TB; t0 < TW; t0 += TB) {
                        gather(j, t0, v);
                        store(stage, on, t0, v);
                    }
                }
                __syncthreads();
                if (mine)
#pragma unroll
                    for (int st = 0; st < 4; st++) {
                        if constexpr (!EARLY) {
                            asm volatile("" ::: "memory");  // one step's weights at a time
#pragma unroll
                            for (int q = 0; q < SETS; q++)
                                w[q][st] = pair_weak(P, nb[l + q] + row[l + q], it * 64 + 32 * h + 8 * st);
                        }
#pragma unroll
                        for (int q = 0; q < SETS; q++)
                            product(acc[l + q], stage, st, w[q][st]);
                    }
            }
        }
    }

    // The K groups add up, in group order. Each takes its share of the accumulator
    // blocks, or of four groups a quarter of the one block, so that all waves are busy
    // after this too (gated 2731 x 1056, 77 tokens, gelu 15.1 -> 12.3 us against group 0
    // alone); with ONE group 0 takes all (the adapters need whole blocks, and the
    // registers are full).
    pair_f4* const red = reinterpret_cast<pair_f4*>(&xs0[0][0]);
    auto put = [&](int slot, const f32x16& v) {  // a wave's block
#pragma unroll
        for (int q = 0; q < 4; q++)
            red[(slot * 4 + q) * 64 + lane] = pair_f4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    };
    auto get = [&](int slot) {
        f32x16 v;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const pair_f4 p = red[(slot * 4 + q) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[4 * q + e] = p[e];
        }
        return v;
    };
    if constexpr (T::SHARE > 1 && !ONE) {
        static_assert(S == 2, "each group hands the other its half");
#pragma unroll
        for (int l = 0; l < 2; l++)
#pragma unroll
            for (int i = 0; i < T::OWN; i++) {
                __syncthreads();
                put(wid, kg == 0 ? acc[l][T::OWN + i] : acc[l][i]);
                __syncthreads();
                acc[l][i] = get(kg == 0 ? wid + WN : wid - WN) + (kg == 0 ? acc[l][i] : acc[l][T::OWN + i]);
            }
    } else if constexpr (S > 1 && !ONE) {
        static_assert(FM == 1 && WN == 1 && S == 4, "a quarter of one block per group");
        pair_f4* const to[2] = {red, reinterpret_cast<pair_f4*>(&xs1[0][0])};
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 2; l++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                to[l][(kg * 4 + q) * 64 + lane] =
                    pair_f4{acc[l][0][4 * q], acc[l][0][4 * q + 1], acc[l][0][4 * q + 2], acc[l][0][4 * q + 3]};
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 2; l++) {
            pair_f4 sum = to[l][kg * 64 + lane];
#pragma unroll
            for (int g2 = 1; g2 < S; g2++)
                sum += to[l][(g2 * 4 + kg) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[l][0][e] = sum[e];
        }
    } else if constexpr (S > 1) {
#pragma unroll
        for (int l = 0; l < 2; l++)
#pragma unroll
            for (int i = 0; i < FM; i++) {
                __syncthreads();
                if (kg > 0)
                    put((kg - 1) * WN + wn, acc[l][i]);
                __syncthreads();
                if (kg == 0)
#pragma unroll
                    for (int g2 = 1; g2 < S; g2++)
                        acc[l][i] += get((g2 - 1) * WN + wn);
            }
        if (kg > 0)
            return false;
    }

    return true;
}

// The tile for M tokens and `rows` rows of each set: f(FM, WN, S) as integral
// constants. Measured for the gated block, us, N x K of each layer, as FM WN S: time
//   11008 x 4096  M = 32  114: 24, 222: 27, 241: 37     64  222: 29, 241: 38, 114: 40
//                    128  241: 42, 222: 44, 442: 60     256  442: 64, 441: 67, 241: 68, 222: 71
//                   2048  441: 336, 241: 388, 442: 399, 222: 449
//   4096 x 11008     64  114: 35, 222: 52, 241: 83     256  222: 65, 241: 87, 114: 109
//                    512  241: 101, 222: 114, 442: 130 640  442: 134, 441: 148, 222: 157, 241: 173
//                   1024  441: 165, 442: 166, 241: 191
//   28672 x 8192     64  241: 90, 222: 93, 442: 122     128  442: 133, 441: 135, 241: 144
//   2731 x 1056     256  222: 14, 241: 16, 114: 21     512  241: 18, 222: 21, 441: 26
// So: 64 x 128 while it gives 170 to 256 blocks, one for most CUs. Past that the CUs
// would hold two of them, and 128 x 128 takes over: K split in two up to 256 blocks, so
// that each SIMD still has two waves, whole above. For fewer blocks 64 x 64 with K
// split in two where that gives 128, else 32 x 32 with K split in four. (Tiles of 128 x
// 64, 64 x 32 and 32 x 32 with K whole or in two were never the fastest by more than
// 3 %; 64 x 128 with K split in two came to between - 7 and + 5 %.)
template <typename F>
hipError_t pair_tile(int64_t M, int64_t rows, F f)
{
    auto blocks = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((rows + bn - 1) / bn); };
    using std::integral_constant;
    if (M > 64 && blocks(128, 128) > 256)
        return f(integral_constant<int, 4>{}, integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (M > 64 && blocks(64, 128) > 256)
        return f(integral_constant<int, 4>{}, integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (blocks(64, 128) >= 170)
        return f(integral_constant<int, 2>{}, integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (M > 32 && blocks(64, 64) >= 128)
        return f(integral_constant<int, 2>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 1>{}, integral_constant<int, 1>{}, integral_constant<int, 4>{});
}

}  // namespace
}  // namespace owq
