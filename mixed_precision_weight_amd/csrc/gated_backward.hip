// gated_backward.hip -- backward of the gated feed-forward block (gfx950).
//
// For h = act(g) u, g = x Wg^T, u = x Wu^T, upstream dh and the kept fp32 g, u:
//   da = dh u act'(g),  db = dh act(g)                       fp32, never stored
//   dx[m][j]    = sum_i da[m][i] Wg[i][j] + db[m][i] Wu[i][j]        fp16
//   dw_g[i][c]  = sum_m da[m][i] x[m][idx_g[c]],  dw_u likewise      fp32
// with W the dequantised dense matrix (0 at the weak columns) plus the weak
// columns, the only trained part.
//
// dx is one product over the 2 N rows of both layers, on the fp16 matrix cores:
// W = s (q - z) splits into the exact small integers q - z (fp16, decoded from the
// codes) and A = 2^e_m s_i da[m][i], rounded to fp16 with a power of two per token
// that puts the token's largest |s da|, |s db| into [2^14, 2^15): 11 bits of every
// term that matters, whatever the gradient's scale, and no overflow. (The rounding
// is the one a caller who stored da as fp16 would make, without its range, and as
// large as the one of dx itself: 2.1e-4 of dx in the root mean square each, 2.9e-4
// together. With A in two fp16 values, 22 bits, the whole backward took 850 us in
// place of 500 at M = 2048, 2 x 11008 x 4096, 62 in place of 48 at M = 1.) The
// weak columns' part, da w_weak, is a product over the rows in fp32, and so is dw,
// over the tokens (v_mfma_f32_32x32x2_f32): their results are not limited by fp16.
//
// Launches:
//  1 k_gated_tok   per 32 tokens and a slab of rows: da, db; each token's largest
//                  |s da|, |s db|; the weak columns' part of dx per slab
//  2 k_gated_sums  the slabs added up: the token's power of two, its weak part
//  3 k_gated_rows  per 64 rows and a slab of tokens: da, db again (two elementwise
//                  passes read less than storing da, db in fp32 would move); dw;
//                  A written in the product's operand order, fp16
//  4 k_gated_dx    the product; splits the rows where tokens and columns alone
//                  do not fill the GPU
//  5 k_gated_fin   adds the splits' and the token slabs' partial sums, in order
// Every sum's order is fixed, so results are deterministic.
//
// Measured, M = 2048, two layers of 11008 x 4096, 32 weak columns each, us:
//  1   76  225 MB read, 2.9 TB/s; the vector memory path is 61 % busy (a token's row
//          per lane), the fp32 matrix instructions and the activations fill the rest
//  2    5
//  3   72  225 MB read, 90 written: 4.3 TB/s
//  4  316  369 GFLOP: 1.17 PFLOP/s; matrix cores and the decode that feeds them (over
//          390 in the first dozen launches after an idle time, at a lower clock: the
//          steps named below were timed so)
//  5   22  67 MB of partial sums read, 17 written: 3.8 TB/s
// Launches 1 and 3 run once per 32 weak columns, the reads and activations again for
// each: 63 columns 148 and 117, 86 columns 228 and 153, 130 columns 358 and 224.
// At M = 77, 2731 x 1056 each launch takes 4 - 13 us: their latencies (launch 2 with
// one thread per sum over all slabs took 6.4, now 3.9).
#include "owq_act.h"
#include "owq_decode.h"
#include "owq_device.h"
#include "owq_launch.h"

namespace owq {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct BwdLayer {
    const uint32_t* q;
    const uint16_t* s;
    const uint8_t* z;
    const int32_t* idx;
    const uint16_t* ww;
    float* dw;    // [N][k], NULL: not wanted
    float* PD;    // token slabs' partials [tslabs][N][k] (tslabs > 1)
    int32_t* map; // [K]: the weak column's position, -1 for a dense column
    int32_t k;
};

struct GatedBwdArgs {
    BwdLayer L[2];
    const uint16_t* x;
    const float* g;
    const float* u;
    const uint16_t* dh;
    uint16_t* dx;     // NULL: not wanted
    int32_t* texp;    // [M]: A is scaled by 2^texp
    float* slabmax;   // [M][slabs]
    float* PW;        // [slabs][M][kt], kt = k gate + k up
    float* PWs;       // [M][kt]
    uint16_t* XW;     // [M][kt]: x at the weak columns of gate, then of up
    uint16_t* A;      // operand order, see a_offset
    float* P;         // [split][M][K] (split > 1)
    int32_t M, N, K, Np;
    int32_t slabs, slab_rows;      // launch 1
    int32_t tslabs, slab_tokens;   // launch 3
    int32_t split, split_steps;    // launch 4
    int32_t work_blocks, map_blocks, mtiles;
};

// A is stored as launch 4 reads it: per 32 tokens and 16 rows (of the 2 Np) the 64
// lanes' operands of v_mfma_f32_32x32x16_f16, 16 bytes each: lane 32 h + t holds
// rows 8 h .. 8 h + 7 of token t. Element of (token, row):
__device__ __forceinline__ int64_t a_offset(int Np, int64_t token, int row)
{
    return ((token >> 5) * (Np >> 3) + (row >> 4)) * 512 + (((row >> 3) & 1) * 32 + (token & 31)) * 8 + (row & 7);
}

__device__ __forceinline__ f32x16 zero16()
{
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; r++)
        z[r] = 0.0f;
    return z;
}

// The elementwise passes load through buffer resources, whose range check returns
// zero past the end: no load sits under a branch (at whose end it would be waited
// for), and rows past N or tokens past M need no clamping, only the masks below.
// (p and bytes are wave-uniform; readfirstlane keeps them in scalar registers also
// where the compiler computed them on the vector ALUs)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uintptr_t)(((uint64_t)hi << 32) | lo)), (short)0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

__device__ __forceinline__ f32x4 buf_f4(__amdgpu_buffer_rsrc_t r, int off)
{
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

__device__ __forceinline__ uint32_t buf_u16(__amdgpu_buffer_rsrc_t r, int off)
{
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}

// ------------------------------------------------------------------- launch 1
// A wave: 32 tokens (lane l: token l % 32) x one slab of rows, 16 rows per step
// (lane half h: rows 8 h .. 8 h + 7, consecutive in memory). The matrix cores'
// k index is the row: step element e pairs da of row 8 h + e with w_weak of that
// row and column l % 32. The next step's loads are issued before this one's
// arithmetic. EVEN: rows of dh start at 4-byte addresses (N even), and so do the
// scales: 8 values are one load (the vector memory path's cycles count: 61 % busy at
// M = 2048 with the scales one by one, 80 us; now 77).
struct TokRows {
    f32x4 g[2], u[2];
    uint32_t d[8];             // EVEN: d[0..3], two values each
    uint32_t w[2][8];          // w_weak
};

template <int ACT, bool EVEN>
__device__ __forceinline__ void tok_slab(const GatedBwdArgs& a, int tile, int slab, int wt)
{
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int m = tile * 32 + l32;
    const bool live = m < a.M;
    const int N = a.N;
    const int r0 = slab * a.slab_rows, r1 = min(N, r0 + a.slab_rows);
    const int c = wt * 32 + l32;  // weak column
    const bool on[2] = {wt * 32 < a.L[0].k, wt * 32 < a.L[1].k};  // uniform
    const int64_t o0 = (int64_t)tile * 32 * N, n0 = (int64_t)min(32, a.M - tile * 32) * N;
    const __amdgpu_buffer_rsrc_t gr = rsrc(a.g + o0, n0 * 4), ur = rsrc(a.u + o0, n0 * 4), dr = rsrc(a.dh + o0, n0 * 2);
    const int lo = l32 * N + 8 * h;
    int woff[2];
#pragma unroll
    for (int l = 0; l < 2; l++)
        woff[l] = 2 * (8 * h * a.L[l].k + min(c, max(a.L[l].k - 1, 0)));
    auto load = [&](int r, TokRows& t) {  // r uniform
        const int o = lo + r;
#pragma unroll
        for (int v = 0; v < 2; v++) {
            t.g[v] = buf_f4(gr, 4 * o + 16 * v);
            t.u[v] = buf_f4(ur, 4 * o + 16 * v);
        }
        if constexpr (EVEN) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b128(dr, 2 * o, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; e++)
                t.d[e] = v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                t.d[e] = buf_u16(dr, 2 * (o + e));
        }
        const int left = max(min(N - r, 16), 0);  // rows of the step
#pragma unroll
        for (int l = 0; l < 2; l++) {
            // an empty resource (zeros) for a layer without this tile of weak columns
            const BwdLayer& L = a.L[l];
            const __amdgpu_buffer_rsrc_t wr =
                rsrc(L.ww + (int64_t)min(r, N) * L.k, on[l] ? (int64_t)left * L.k * 2 : 0);
#pragma unroll
            for (int e = 0; e < 8; e++)
                t.w[l][e] = buf_u16(wr, woff[l] + 2 * e * L.k);
        }
    };
    f32x16 acc[2] = {zero16(), zero16()};
    float mx = 0.0f;
    // one step on `cur`; `nxt` is loaded for the one after. The rows' steps s_i are
    // loaded ahead of that, so waiting for them waits for none of it.
    auto work = [&](int r, const TokRows& cur, TokRows& nxt) {
        uint32_t sv[2][8];  // EVEN: [0 .. 3], two values each
#pragma unroll
        for (int l = 0; l < 2; l++) {
            const __amdgpu_buffer_rsrc_t sr = rsrc(a.L[l].s + min(r, N), max(N - r, 0) * 2);
            if constexpr (EVEN) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b128(sr, 16 * h, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    sv[l][e] = v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    sv[l][e] = buf_u16(sr, 16 * h + 2 * e);
            }
        }
        asm volatile("" ::: "memory");
        load(r + 16, nxt);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const bool use = live && r + 8 * h + e < r1;
            float v, d;
            act_both<ACT>(cur.g[e / 4][e % 4], v, d);
            const float dh = h2f((uint16_t)(EVEN ? cur.d[e / 2] >> (16 * (e % 2)) : cur.d[e]));
            const float da = use ? dh * cur.u[e / 4][e % 4] * d : 0.0f, db = use ? dh * v : 0.0f;
            acc[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(da, h2f((uint16_t)cur.w[0][e]), acc[0], 0, 0, 0);
            acc[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(db, h2f((uint16_t)cur.w[1][e]), acc[1], 0, 0, 0);
            const uint32_t sa = EVEN ? sv[0][e / 2] >> (16 * (e % 2)) : sv[0][e];
            const uint32_t sb = EVEN ? sv[1][e / 2] >> (16 * (e % 2)) : sv[1][e];
            mx = fmaxf(mx, fmaxf(fabsf(h2f((uint16_t)sa) * da), fabsf(h2f((uint16_t)sb) * db)));
        }
    };
    TokRows ta, tb;
    load(r0, ta);
    for (int r = r0; r < r1; r += 32) {
        work(r, ta, tb);
        work(r + 16, tb, ta);
    }
    if (wt == 0) {
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        if (h == 0 && live)
            a.slabmax[(int64_t)m * a.slabs + slab] = mx;
    }
    const int kt = a.L[0].k + a.L[1].k;
#pragma unroll
    for (int l = 0; l < 2; l++)
        if (c < a.L[l].k)
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int t = tile * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
                if (t < a.M)
                    a.PW[((int64_t)slab * a.M + t) * kt + (l ? a.L[0].k : 0) + c] = acc[l][r];
            }
}

// blocks [0, work_blocks): waves over (token tile, slab); then (first row of the
// grid only) map_blocks: the map from columns to weak columns; then x at the weak
// columns, gathered once (launch 3 reads it once per 64 rows: gathers there would
// fetch a cache line per value each time)
template <int ACT, bool EVEN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_gated_tok(const GatedBwdArgs a)
{
    if ((int)blockIdx.x >= a.work_blocks + a.map_blocks) {
        const int kt = a.L[0].k + a.L[1].k;
        const int64_t e = (int64_t)((int)blockIdx.x - a.work_blocks - a.map_blocks) * 256 + threadIdx.x;
        if (blockIdx.y != 0 || e >= (int64_t)a.M * kt)
            return;
        const int64_t m = e / kt;
        const int c = (int)(e - m * kt);
        const int j = c < a.L[0].k ? a.L[0].idx[c] : a.L[1].idx[c - a.L[0].k];
        a.XW[e] = a.x[m * a.K + (j >= 0 && j < a.K ? j : 0)];
        return;
    }
    if ((int)blockIdx.x >= a.work_blocks) {
        const int j = ((int)blockIdx.x - a.work_blocks) * 256 + (int)threadIdx.x;
        if (blockIdx.y != 0 || j >= a.K)
            return;
        for (int l = 0; l < 2; l++) {
            int lo = 0, hi = a.L[l].k;  // first position whose column is >= j
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (a.L[l].idx[mid] < j)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            a.L[l].map[j] = lo < a.L[l].k && a.L[l].idx[lo] == j ? lo : -1;
        }
        return;
    }
    const int w = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tiles = (a.M + 31) >> 5;
    if (w >= tiles * a.slabs)
        return;
    const int slab = __builtin_amdgcn_readfirstlane(w / tiles);
    tok_slab<ACT, EVEN>(a, w - slab * tiles, slab, (int)blockIdx.y);
}

// ------------------------------------------------------------- launches 2 and 3
// A block: 64 rows (lane l: rows 2 (l % 32), + 1) x one slab of tokens, its 4
// waves taking four tokens in turn, two pairs (lane half h: token of the pair). The
// matrix cores' k index is the token: da of row 2 (l % 32) + e against x at weak
// column l % 32. The waves' sums are added in order in LDS.
constexpr int kTokFlight = 2;  // pairs of tokens whose loads are in flight together

__device__ __forceinline__ int scale_exp(float mx)
{
    return mx > 0.0f && mx < 0x1p120f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
}

__device__ __forceinline__ uint32_t swap_neighbours(uint32_t v)  // lane 2 i <-> 2 i + 1
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);  // quad_perm [1, 0, 3, 2]
}

template <int ACT, bool EVEN>
__device__ __forceinline__ void row_slab(const GatedBwdArgs& a, int tile, int slab, int wt, float* red)
{
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = slab * a.slab_tokens, t1 = min(a.M, t0 + a.slab_tokens);
    const int row = tile * 64 + 2 * l32;
    const bool conv = a.dx && wt == 0;  // this block writes A
    const bool on[2] = {a.L[0].dw && wt * 32 < a.L[0].k, a.L[1].dw && wt * 32 < a.L[1].k};
    const int rc[2] = {min(row, a.N - 1), min(row + 1, a.N - 1)};
    float sc[2][2];
    const int kt = a.L[0].k + a.L[1].k;
    int jw[2];  // this lane's weak columns in a row of XW
#pragma unroll
    for (int l = 0; l < 2; l++) {
        sc[l][0] = h2f(a.L[l].s[rc[0]]);
        sc[l][1] = h2f(a.L[l].s[rc[1]]);
        jw[l] = on[l] ? (l ? a.L[0].k : 0) + min(wt * 32 + l32, a.L[l].k - 1) : 0;
    }
    f32x16 acc[2][2] = {{zero16(), zero16()}, {zero16(), zero16()}};
    // kTokFlight pairs of tokens per step; the next step's loads are issued before
    // this one's arithmetic
    struct Pairs {
        uint32_t g[kTokFlight][2], u[kTokFlight][2];
        uint32_t d[kTokFlight][2], xw[kTokFlight][2];  // EVEN: d[v][0], both values
        int ex[kTokFlight];
    };
    const int po = h * a.N + row;  // this lane's element of a pair of tokens
    // Neighbouring lanes swap half of what they have for A, so that each stores four
    // rows of one token: odd lanes of the second pair, even lanes of the first. Four
    // tokens are then 64 bytes in a row and half the stores (84 -> 72 us at M = 2048
    // with rows of 11008 against 4 bytes per lane as computed)
    const int odd = lane & 1;
    int aoff[2];  // byte of those four rows in a tile of A, for the tile's first tokens
#pragma unroll
    for (int l = 0; l < 2; l++)
        aoff[l] = (int)a_offset(a.Np, 2 * odd + h, l * a.Np + row - 2 * odd) * 2;
    auto load = [&](int t, Pairs& q) {  // t uniform
#pragma unroll
        for (int v = 0; v < kTokFlight; v++) {
            const int tp = min(t + 2 * v, t1 - 1);  // the pair's first token; past the slab: not used
            const int64_t o = (int64_t)tp * a.N, n = (int64_t)min(2, a.M - tp) * a.N;
            const auto gv = __builtin_amdgcn_raw_buffer_load_b64(rsrc(a.g + o, n * 4), 4 * po, 0, 0);
            const auto uv = __builtin_amdgcn_raw_buffer_load_b64(rsrc(a.u + o, n * 4), 4 * po, 0, 0);
            q.g[v][0] = gv[0], q.g[v][1] = gv[1], q.u[v][0] = uv[0], q.u[v][1] = uv[1];
            const __amdgpu_buffer_rsrc_t dr = rsrc(a.dh + o, n * 2);
            if constexpr (EVEN) {
                q.d[v][0] = __builtin_amdgcn_raw_buffer_load_b32(dr, 2 * po, 0, 0);
            } else {
                q.d[v][0] = buf_u16(dr, 2 * po);
                q.d[v][1] = buf_u16(dr, 2 * po + 2);
            }
            const int64_t m = min(tp + h, a.M - 1);
#pragma unroll
            for (int l = 0; l < 2; l++)  // (workspace: readable also where not used)
                q.xw[v][l] = a.XW[m * kt + jw[l]];
            q.ex[v] = a.texp[m];
        }
    };
    auto work = [&](int tb, const Pairs& cur, Pairs& nxt) {
        load(tb + 8 * kTokFlight, nxt);
        uint32_t as[2][kTokFlight];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int v = 0; v < kTokFlight; v++) {
            const int t = tb + 2 * v + h;
            float dab[2][2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const bool use = t < t1 && row + e < a.N;
                float va, sl;
                act_both<ACT>(__builtin_bit_cast(float, cur.g[v][e]), va, sl);
                const float dh = h2f((uint16_t)(EVEN ? cur.d[v][0] >> (16 * e) : cur.d[v][e]));
                dab[0][e] = use ? dh * __builtin_bit_cast(float, cur.u[v][e]) * sl : 0.0f;
                dab[1][e] = use ? dh * va : 0.0f;
            }
            if (conv)  // uniform
#pragma unroll
                for (int l = 0; l < 2; l++)
                    as[l][v] = f2h(__builtin_amdgcn_ldexpf(dab[l][0] * sc[l][0], cur.ex[v])) |
                               (uint32_t)f2h(__builtin_amdgcn_ldexpf(dab[l][1] * sc[l][1], cur.ex[v])) << 16;
#pragma unroll
            for (int l = 0; l < 2; l++) {
                const float xv = h2f((uint16_t)cur.xw[v][l]);
#pragma unroll
                for (int e = 0; e < 2; e++)
                    acc[l][e] = __builtin_amdgcn_mfma_f32_32x32x2f32(dab[l][e], xv, acc[l][e], 0, 0, 0);
            }
        }
        if (conv) {
            // the four tokens are a quarter of a 32-token tile of A; lanes without
            // rows or token store out of range
            const __amdgpu_buffer_rsrc_t dst = rsrc(a.A + (int64_t)(tb >> 5) * 64 * a.Np, (int64_t)128 * a.Np);
            const int dead = tb + 2 * odd + h < t1 && row < a.Np ? 0 : 0x40000000;
#pragma unroll
            for (int l = 0; l < 2; l++) {
                const uint32_t mine = odd ? as[l][1] : as[l][0];
                const uint32_t got = swap_neighbours(odd ? as[l][0] : as[l][1]);
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                const u32x2 v = {odd ? got : mine, odd ? mine : got};
                __builtin_amdgcn_raw_buffer_store_b64(v, dst, (aoff[l] | dead) + (tb & 31) * 16, 0, 0);
            }
        }
    };
    Pairs pa, pb;
    const int first = t0 + 4 * wave;
    if (first < t1)
        load(first, pa);
    static_assert(kTokFlight == 2, "a step is four tokens");
    for (int t = first; t < t1; t += 16 * kTokFlight) {
        work(t, pa, pb);
        work(t + 8 * kTokFlight, pb, pa);
    }
    // D element r of lane l: row 2 (8 (r / 4) + 4 h + r % 4) + e, weak column l % 32
#pragma unroll
    for (int l = 0; l < 2; l++) {
        if (!on[l])
            continue;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            __syncthreads();
            if (wave > 0)
#pragma unroll
                for (int r = 0; r < 16; r++)
                    red[((wave - 1) * 16 + r) * 64 + lane] = acc[l][e][r];
            __syncthreads();
            if (wave == 0)
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const float v = ((acc[l][e][r] + red[r * 64 + lane]) + red[(16 + r) * 64 + lane]) +
                                    red[(32 + r) * 64 + lane];
                    const int i = tile * 64 + 2 * (8 * (r >> 2) + 4 * h + (r & 3)) + e;
                    const int c = wt * 32 + l32;
                    if (i < a.N && c < a.L[l].k) {
                        const int64_t at = (int64_t)i * a.L[l].k + c;
                        if (a.tslabs > 1)
                            a.L[l].PD[(int64_t)slab * a.N * a.L[l].k + at] = v;
                        else
                            a.L[l].dw[at] = v;
                    }
                }
        }
    }
}

template <int ACT, bool EVEN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void k_gated_rows(const GatedBwdArgs a)
{
    __shared__ float red[48 * 64];
    const int tiles = (a.Np + 63) / 64;
    const int slab = __builtin_amdgcn_readfirstlane((int)blockIdx.x / tiles);
    row_slab<ACT, EVEN>(a, (int)blockIdx.x - slab * tiles, slab, (int)blockIdx.y, red);
}

// Between the two: blocks [0, work_blocks): a wave per token, its exponent from the
// slabs' largest values; the rest: the slabs' weak sums added in order.
__global__ __launch_bounds__(256) void k_gated_sums(const GatedBwdArgs a)
{
    if ((int)blockIdx.x < a.work_blocks) {
        const int m = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        if (m >= a.M)
            return;
        float mx = 0.0f;
        for (int s = threadIdx.x & 63; s < a.slabs; s += 64)
            mx = fmaxf(mx, a.slabmax[(int64_t)m * a.slabs + s]);
        mx = wave_max_dpp(mx);
        if ((threadIdx.x & 63) == 0)
            a.texp[m] = scale_exp(mx);
        return;
    }
    // 64 values per block, a quarter of the slabs per wave, 8 loads in flight
    __shared__ float part[3][64];
    const int64_t n = (int64_t)a.M * (a.L[0].k + a.L[1].k);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t e = (int64_t)((int)blockIdx.x - a.work_blocks) * 64 + lane;
    const int64_t ec = e < n ? e : n - 1;
    const int per = (a.slabs + 3) >> 2, s1 = min(a.slabs, (wave + 1) * per);
    float t = 0.0f;
    for (int s = wave * per; s < s1; s += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = a.PW[min(s + i, s1 - 1) * n + ec];
#pragma unroll
        for (int i = 0; i < 8; i++)
            t += s + i < s1 ? v[i] : 0.0f;
    }
    if (wave > 0)
        part[wave - 1][lane] = t;
    __syncthreads();
    if (wave > 0 || e >= n)
        return;
    t = ((t + part[0][lane]) + part[1][lane]) + part[2][lane];
    a.PWs[e] = t;
}

// ------------------------------------------------------------------- launch 4
// dx: D[m][j] = sum over r < 2 Np of A[m][r] (q - z)[r][j], rows of gate, then of
// up. A block owns BM tokens x BN columns and steps of RS rows: thread t decodes
// one 32-column group of one row into the LDS tile [row][column] (exact fp16), one
// step ahead of the products; A goes from memory into the operand registers two
// steps ahead, as whole kilobytes in operand order: through LDS it would take a
// third of the LDS bandwidth, which bounds the step (397 -> 365 us at M = 2048,
// 2 x 11008 x 4096). v_mfma_f32_32x32x16_f16
// takes 8 consecutive rows per lane; for the decoded tile the transposing LDS read
// (ds_read_b64_tr_b16: in 16 lanes, lane i receives element i of four rows of 16
// columns) gives 4 rows of the lane's column. Tile rows are padded to 64 bytes past
// a multiple of 256, so the four rows of a read lie in distinct banks.
template <int FM, int FN, int WM, int WN, int RS>
struct DxTile {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    static constexpr int BROW = BN * 2 + 64;         // LDS bytes of a decoded row
    // The 16-byte pieces of group g of row r are stored at piece ^ b_swizzle: rows and
    // groups 64 bytes apart would put the 16 lanes of a write on 4 of the 16 places
    // that the banks hold (415 -> 395 us at M = 2048, 2 x 11008 x 4096). Constant over
    // a lane's reads: its rows agree modulo 4, a wave's groups share g / 4.
    static constexpr int GB = BN / 32;
    __device__ static __forceinline__ int b_swizzle(int g, int r)
    {
        return GB == 8 ? ((g >> 2) & 1) | ((r & 1) << 1) : r & 3;
    }
    static_assert((GB == 8 && FN == 4) || GB == 4, "a wave's groups must share their swizzle");
    static_assert(RS * GB == NT, "one group per thread and step");
    static_assert((BN * 2) % 256 == 0, "tile rows 64 bytes apart modulo the banks");
};

// four rows of this lane's column from each of two places in the decoded tile
__device__ __forceinline__ half8_t read_columns(const char* a, const char* b)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)b);
    return __builtin_bit_cast(half8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int FM, int FN, int WM, int WN, int RS>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2))) void k_gated_dx(const GatedBwdArgs a)
{
    using T = DxTile<FM, FN, WM, WN, RS>;
    __shared__ __attribute__((aligned(1024))) char bs[2][RS * T::BROW];

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int K = a.K, G = K >> 5, M = a.M, N = a.N, Np = a.Np;
    const int ctiles = (K + T::BN - 1) / T::BN;
    const int b = blockIdx.x;
    const int m0 = (b % a.mtiles) * T::BM;
    const int j0 = (b / a.mtiles % ctiles) * T::BN;
    const int sp = b / (a.mtiles * ctiles);
    const int steps = 2 * Np / RS;
    const int st0 = sp * a.split_steps, st1 = min(steps, st0 + a.split_steps);

    // A of this wave's 32-token tiles (tiles past M repeat the last: not stored);
    // steps past the end repeat the last
    constexpr int KS = RS / 16;
    __amdgpu_buffer_rsrc_t ar[FM];
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int tile = min((m0 >> 5) + wm * FM + i, (M - 1) >> 5);
        ar[i] = rsrc(a.A + (int64_t)tile * 64 * Np, (int64_t)128 * Np);
    }
    struct Tokens {
        half8_t v[KS][FM];
    };
    auto load_a = [&](int st, Tokens& t) {
        const int o = min(st, st1 - 1) * KS * 1024;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
            for (int i = 0; i < FM; i++)
                t.v[ks][i] = __builtin_bit_cast(
                    half8_t, __builtin_amdgcn_raw_buffer_load_b128(ar[i], lane * 16, o + ks * 1024, 0));
    };
    // codes: thread t decodes group t % (BN / 32) of row t / (BN / 32) of a step.
    // Rows past N and groups past K read valid ones (A is zero there, the columns
    // are not stored).
    constexpr int GB = T::GB;
    const int lrow = tid / GB, lg = tid % GB;
    const int gg = min(j0 / 32 + lg, G - 1);
    struct Codes {
        uint32_t w0, w1, w2, z;
    };
    auto load_q = [&](int st, Codes& c) {
        const int r = min(st, st1 - 1) * RS + lrow;
        const BwdLayer& L = r < Np ? a.L[0] : a.L[1];
        const int row = min(r < Np ? r : r - Np, N - 1);
        const uint32_t* src = L.q + ((int64_t)row * G + gg) * 3;
        c.w0 = src[0];
        c.w1 = src[1];
        c.w2 = src[2];
        c.z = L.z[row];
    };
    const Magic mg = make_magic();
    auto stage_b = [&](const Codes& c, char* tile) {
        uint32_t p[16];
        decode_group(c.w0, c.w1, c.w2, mg, make_zero_sub(c.z), p);
        uint4* dst = reinterpret_cast<uint4*>(tile + lrow * T::BROW + lg * 64);
        const int swz = T::b_swizzle(lg, lrow);
#pragma unroll
        for (int q4 = 0; q4 < 4; q4++)
            dst[q4 ^ swz] = make_uint4(p[4 * q4], p[4 * q4 + 1], p[4 * q4 + 2], p[4 * q4 + 3]);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
            acc[i][f] = zero16();

    // this lane's columns of 16-row step ks: decoded rows 16 ks + 8 h + 4 t + (l % 16)
    // / 4, columns of its 16-lane group
    const int brow = (lane & 15) >> 2, bpiece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int boff = (8 * h + brow) * T::BROW + wn * FN * 64 + ((bpiece ^ T::b_swizzle(wn * FN, brow)) << 4) + 8 * (lane & 1);

    // Step st computes on cur and tile st & 1; it starts the loads of step st + 2 and
    // decodes step st + 1 (its codes were loaded one step ago) into the other tile.
    auto step = [&](int st, const Tokens& cur, Tokens& nxt2, Codes& mine, Codes& next) {
        // closes the tile written in the last step, and the reads of the one that this
        // step overwrites; loads in flight stay in flight
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        load_a(st + 2, nxt2);
        load_q(st + 2, next);
        const char* tile = bs[(st - st0) & 1];
        if (st + 1 < st1)  // uniform
            stage_b(mine, bs[(st + 1 - st0) & 1]);
        if (st < st1) {
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
#pragma unroll
                for (int f = 0; f < FN; f++) {
                    const char* src = tile + boff + ks * 16 * T::BROW + f * 64;
                    const half8_t bv = read_columns(src, src + 4 * T::BROW);
#pragma unroll
                    for (int i = 0; i < FM; i++)
                        acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(cur.v[ks][i], bv, acc[i][f], 0, 0, 0);
                }
            }
        }
    };

    Codes qa, qb;
    Tokens ta, tb, tc;
    load_a(st0, ta);
    load_q(st0, qa);
    asm volatile("" ::: "memory");
    load_a(st0 + 1, tb);
    load_q(st0 + 1, qb);
    asm volatile("" ::: "memory");
    stage_b(qa, bs[0]);
    for (int st = st0; st < st1; st += 6) {
        step(st, ta, tc, qb, qa);
        step(st + 1, tb, ta, qa, qb);
        step(st + 2, tc, tb, qb, qa);
        step(st + 3, ta, tc, qa, qb);
        step(st + 4, tb, ta, qb, qa);
        step(st + 5, tc, tb, qa, qb);
    }

    // D element r of lane l: token 8 (r / 4) + 4 h + r % 4, column l % 32
    const int kt = a.L[0].k + a.L[1].k;
#pragma unroll
    for (int f = 0; f < FN; f++) {
        const int j = j0 + wn * 32 * FN + 32 * f + l32;
        if (j >= K)
            continue;
        if (a.split > 1) {
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int m = m0 + wm * 32 * FM + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                    if (m < M)
                        a.P[((int64_t)sp * M + m) * K + j] = acc[i][f][r];
                }
            continue;
        }
        const int wg = a.L[0].map[j], wu = a.L[1].map[j];
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int m = m0 + wm * 32 * FM + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                if (m < M) {
                    float v = __builtin_amdgcn_ldexpf(acc[i][f][r], -a.texp[m]);
                    if (wg >= 0)
                        v += a.PWs[(int64_t)m * kt + wg];
                    if (wu >= 0)
                        v += a.PWs[(int64_t)m * kt + a.L[0].k + wu];
                    a.dx[(int64_t)m * K + j] = f2h(v);
                }
            }
    }
}

// ------------------------------------------------------------------- launch 5
// blocks [0, work_blocks): dx, a thread per 4 columns; then dw of gate, of up
__global__ __launch_bounds__(256) void k_gated_fin(const GatedBwdArgs a, int blocks_g)
{
    const int64_t b = blockIdx.x;
    if (b < a.work_blocks) {
        const int64_t n = (int64_t)a.M * a.K;
        const int64_t e = (b * 256 + threadIdx.x) * 4;
        if (e >= n)
            return;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int s = 0;
        auto add = [&](auto count) {  // that many loads in flight, added in order
            constexpr int C = decltype(count)::value;
            for (; s + C <= a.split; s += C) {
                float4 v[C];
#pragma unroll
                for (int i = 0; i < C; i++)
                    v[i] = *reinterpret_cast<const float4*>(a.P + (s + i) * n + e);
#pragma unroll
                for (int i = 0; i < C; i++)
                    t.x += v[i].x, t.y += v[i].y, t.z += v[i].z, t.w += v[i].w;
            }
        };
        add(std::integral_constant<int, 8>{});
        add(std::integral_constant<int, 2>{});
        add(std::integral_constant<int, 1>{});
        const int64_t m = e / a.K;
        const int j = (int)(e - m * a.K);
        const int ex = -a.texp[m], kt = a.L[0].k + a.L[1].k;
        const float o[4] = {t.x, t.y, t.z, t.w};
        const int4 mg = *reinterpret_cast<const int4*>(a.L[0].map + j), mu = *reinterpret_cast<const int4*>(a.L[1].map + j);
        const int wg[4] = {mg.x, mg.y, mg.z, mg.w}, wu[4] = {mu.x, mu.y, mu.z, mu.w};
        uint32_t q[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            float v = __builtin_amdgcn_ldexpf(o[c], ex);
            if (wg[c] >= 0)
                v += a.PWs[m * kt + wg[c]];
            if (wu[c] >= 0)
                v += a.PWs[m * kt + a.L[0].k + wu[c]];
            q[c] = f2h(v);
        }
        uint16_t* dst = a.dx + e;
        if ((reinterpret_cast<uintptr_t>(a.dx) & 7) == 0) {  // uniform; dx may start at any even address
            *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        } else {
#pragma unroll
            for (int c = 0; c < 4; c++)
                dst[c] = (uint16_t)q[c];
        }
        return;
    }
    const int64_t c = b - a.work_blocks;
    const BwdLayer& L = c < blocks_g ? a.L[0] : a.L[1];
    const int64_t n = (int64_t)a.N * L.k;
    const int64_t e = (c < blocks_g ? c : c - blocks_g) * 256 + threadIdx.x;
    if (e >= n)
        return;
    float t = 0.0f;
    for (int s = 0; s < a.tslabs; s += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = L.PD[min(s + i, a.tslabs - 1) * n + e];
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (s + i < a.tslabs)  // uniform
                t += v[i];
    }
    L.dw[e] = t;
}

constexpr size_t al256(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t clampi(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : (v > hi ? hi : v); }

// tile of launch 4 for M tokens: tokens x columns, rows per step
struct DxShape {
    int bm, bn, rs;
};
DxShape dx_shape(int64_t M)
{
    if (M <= 32)
        return {32, 128, 64};
    if (M <= 64)
        return {64, 128, 64};
    return {128, 256, 32};
}

struct GatedBwdPlan {
    int64_t Np, slabs, slab_rows, tslabs, slab_tokens, split, split_steps;
    size_t off_texp, off_max, off_map, off_pw, off_pws, off_xw, off_a, off_pd, off_p, total;
};

GatedBwdPlan gated_bwd_plan(int64_t N, int64_t K, int64_t kt, int64_t M)
{
    GatedBwdPlan p;
    const size_t budget = (size_t)64 << 20;  // of each set of partial sums, unless one slab alone is larger
    p.Np = cdiv(N, 64) * 64;
    // launch 1: 2048 waves (what the GPU holds at two per SIMD) where the rows
    // allow slabs of 32 at least
    const int64_t tiles = cdiv(M, 32);
    p.slabs = clampi(2048 / tiles, 1, cdiv(N, 32));
    if (kt > 0)
        p.slabs = clampi((int64_t)(budget / ((size_t)M * kt * 4)), 1, p.slabs);
    p.slab_rows = cdiv(cdiv(N, p.slabs), 16) * 16;
    p.slabs = cdiv(N, p.slab_rows);
    // launch 3: blocks of 64 rows, as many as the GPU holds at once (1024, four
    // waves per SIMD), 32 tokens per slab at least
    const int64_t rtiles = p.Np / 64;
    p.tslabs = clampi(1024 / rtiles, 1, cdiv(M, 32));
    if (kt > 0)
        p.tslabs = clampi((int64_t)(budget / ((size_t)N * kt * 4)), 1, p.tslabs);
    p.slab_tokens = cdiv(cdiv(M, p.tslabs), 16) * 16;  // four tokens for each of four waves
    p.tslabs = cdiv(M, p.slab_tokens);
    // launch 4: 512 blocks, 4 steps each at least
    const DxShape d = dx_shape(M);
    const int64_t steps = 2 * p.Np / d.rs;
    p.split = clampi(cdiv(512, cdiv(M, d.bm) * cdiv(K, d.bn)), 1, cdiv(steps, 4));
    p.split_steps = cdiv(steps, p.split);
    p.split = cdiv(steps, p.split_steps);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += al256(bytes);
        return at;
    };
    p.off_texp = take((size_t)M * 4);
    p.off_max = take((size_t)p.slabs * M * 4);
    p.off_map = take((size_t)2 * K * 4);
    p.off_pw = take((size_t)p.slabs * M * kt * 4);
    p.off_pws = take((size_t)M * kt * 4);
    p.off_xw = take((size_t)M * kt * 2);
    p.off_a = take((size_t)cdiv(M, 32) * 32 * 2 * p.Np * 2);
    p.off_pd = take(p.tslabs > 1 ? (size_t)p.tslabs * N * kt * 4 : 0);
    p.off_p = take(p.split > 1 ? (size_t)p.split * M * K * 4 : 0);
    p.total = o;
    return p;
}

template <int FM, int FN, int WM, int WN, int RS>
hipError_t launch_dx(const GatedBwdArgs& a, int64_t blocks, hipStream_t s)
{
    using T = DxTile<FM, FN, WM, WN, RS>;
    static_assert(T::NT == 256, "the threads per block that the grids are checked with");
    hipLaunchKernelGGL((k_gated_dx<FM, FN, WM, WN, RS>), dim3((unsigned)blocks), dim3(T::NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t gated_bwd_workspace_bytes(int64_t N, int64_t K, int32_t kg, int32_t ku, int64_t M)
{
    return gated_bwd_plan(N, K, (int64_t)kg + ku, M).total;
}

hipError_t launch_gated_backward(const LinearDesc& gate, const LinearDesc& up, int64_t M, int act, const float* g,
                                 const float* u, const uint16_t* dh, uint16_t* dx, float* dw_gate, float* dw_up,
                                 void* ws, hipStream_t s)
{
    const int64_t N = gate.N, K = gate.K, kt = (int64_t)gate.k + up.k;
    const GatedBwdPlan p = gated_bwd_plan(N, K, kt, M);
    char* const w = static_cast<char*>(ws);
    GatedBwdArgs a{};
    const LinearDesc* d[2] = {&gate, &up};
    float* dw[2] = {gate.k > 0 ? dw_gate : nullptr, up.k > 0 ? dw_up : nullptr};
    for (int l = 0; l < 2; l++) {
        BwdLayer& L = a.L[l];
        L.q = d[l]->q, L.s = d[l]->s, L.z = d[l]->z, L.idx = d[l]->idx, L.ww = d[l]->ww, L.k = d[l]->k;
        L.dw = dw[l];
        L.PD = reinterpret_cast<float*>(w + p.off_pd) + (l ? p.tslabs * N * gate.k : 0);
        L.map = reinterpret_cast<int32_t*>(w + p.off_map) + l * K;
    }
    a.x = gate.x, a.g = g, a.u = u, a.dh = dh, a.dx = dx;
    a.texp = reinterpret_cast<int32_t*>(w + p.off_texp);
    a.slabmax = reinterpret_cast<float*>(w + p.off_max);
    a.PW = reinterpret_cast<float*>(w + p.off_pw);
    a.PWs = reinterpret_cast<float*>(w + p.off_pws);
    a.XW = reinterpret_cast<uint16_t*>(w + p.off_xw);
    a.A = reinterpret_cast<uint16_t*>(w + p.off_a);
    a.P = reinterpret_cast<float*>(w + p.off_p);
    a.M = (int32_t)M, a.N = (int32_t)N, a.K = (int32_t)K, a.Np = (int32_t)p.Np;
    a.slabs = (int32_t)p.slabs, a.slab_rows = (int32_t)p.slab_rows;
    a.tslabs = (int32_t)p.tslabs, a.slab_tokens = (int32_t)p.slab_tokens;
    a.split = (int32_t)p.split, a.split_steps = (int32_t)p.split_steps;
    const int kmax = gate.k > up.k ? gate.k : up.k;
    const unsigned wtiles = kmax > 0 ? (unsigned)cdiv(kmax, 32) : 1u;
    const bool any_dw = dw[0] || dw[1];
    const bool even = N % 2 == 0 && ((reinterpret_cast<uintptr_t>(dh) | reinterpret_cast<uintptr_t>(gate.s) |
                                      reinterpret_cast<uintptr_t>(up.s)) & 3) == 0;
    a.work_blocks = dx ? (int32_t)cdiv(cdiv(M, 32) * p.slabs, 4) : 0;
    a.map_blocks = dx ? (int32_t)cdiv(K, 256) : 0;
    // every launch's blocks (256 threads each), checked before the first
    const DxShape tile = dx_shape(M);
    a.mtiles = (int)cdiv(M, tile.bm);
    const int64_t first = a.work_blocks + a.map_blocks + (any_dw ? cdiv(M * kt, 256) : 0);
    const int64_t sums = cdiv(M, 4) + cdiv(M * kt, 64);
    const int64_t rows = p.Np / 64 * p.tslabs;
    const int64_t product = a.mtiles * cdiv(K, tile.bn) * p.split;
    const int64_t fin = dx && p.split > 1 ? cdiv(M * K, 1024) : 0;
    const int64_t bg = dw[0] && p.tslabs > 1 ? cdiv(N * gate.k, 256) : 0;
    const int64_t bu = dw[1] && p.tslabs > 1 ? cdiv(N * up.k, 256) : 0;
    for (const int64_t blocks : {first, dx ? sums : 1, rows, dx ? product : 1, fin + bg + bu + 1})
        if (!grid_fits(blocks, 256))
            return hipErrorInvalidConfiguration;
    {
        const dim3 grid((unsigned)first, wtiles);
        for_act(act, [&](auto c) {
            if (even)
                hipLaunchKernelGGL((k_gated_tok<decltype(c)::value, true>), grid, dim3(256), 0, s, a);
            else
                hipLaunchKernelGGL((k_gated_tok<decltype(c)::value, false>), grid, dim3(256), 0, s, a);
        });
    }
    if (dx) {
        a.work_blocks = (int32_t)cdiv(M, 4);
        hipLaunchKernelGGL(k_gated_sums, dim3((unsigned)sums), dim3(256), 0, s, a);
    }
    {
        const dim3 grid((unsigned)rows, any_dw ? wtiles : 1u);
        for_act(act, [&](auto c) {
            if (even)
                hipLaunchKernelGGL((k_gated_rows<decltype(c)::value, true>), grid, dim3(256), 0, s, a);
            else
                hipLaunchKernelGGL((k_gated_rows<decltype(c)::value, false>), grid, dim3(256), 0, s, a);
        });
    }
    hipError_t e = hipGetLastError();
    if (dx && e == hipSuccess) {
        if (M <= 32)
            e = launch_dx<1, 1, 1, 4, 64>(a, product, s);
        else if (M <= 64)
            e = launch_dx<2, 1, 1, 4, 64>(a, product, s);
        else
            e = launch_dx<2, 4, 2, 2, 32>(a, product, s);
    }
    if (e != hipSuccess)
        return e;
    a.work_blocks = (int32_t)fin;
    if (fin + bg + bu > 0)
        hipLaunchKernelGGL(k_gated_fin, dim3((unsigned)(fin + bg + bu)), dim3(256), 0, s, a, (int)bg);
    return hipGetLastError();
}

}  // namespace owq
