// gated.hip -- the gated half of a feed-forward block in one launch (gfx950):
//   g = x Wg^T,  u = x Wu^T,  h[m][i] = act(g[m][i]) u[m][i]
// Wg and Wu are packed layers of the same N and K, each with weak columns of its
// own; row i of both ends in the same wave, so the activation and the product run
// on the fp32 sums and h is rounded once; g and u never reach memory unless the
// caller keeps them (fp32, for the backward).
//
// The three kernels are the linear's three regimes with both layers' rows side by
// side (the decoded groups of two rows meet one read of x), chosen by the token
// count M as for the linear:
//   k_gated_gemv  M <= 2    a wave per RP rows of both layers, lanes split K;
//                           bound by the code stream from HBM
//   k_gated_mfv   M <= 16   a wave per 16 rows of both, v_mfma_f32_16x16x32_f16;
//                           code stream and register decode
//   k_gated_gemm  above     a tile of tokens x (rows of gate + rows of up),
//                           v_mfma_f32_32x32x16_f16; matrix cores and decode
// Products of fp16 x with the integers q - z are exact; sums are fp32.
//
// Measured, two layers of 11008 x 4096: M = 1 10.7 us (3.3 TB/s of codes and weak
// columns; 9.2 one after another in a graph), M = 2048 325 us (1.14 PFLOP/s, where a
// plain library product of 8192^3 reaches 1.16), 342 with g and u kept; 28672 x 8192 at
// M = 8 49 us (3.8 TB/s); 2048 x 768 at M = 1 4.4 us, launch and one memory latency.
#include <type_traits>

#include "owq_act.h"
#include "owq_decode.h"
#include "owq_device.h"
#include "owq_gemv.h"
#include "owq_launch.h"
#include "owq_pair_gemm.h"

namespace owq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct GatedArgs {
    PairLayer L[2];  // gate, up
    const uint16_t* x;
    uint16_t* h;
    float* g;  // NULL: not kept
    float* u;
    int32_t M, N, K, act;
    int32_t mblocks;  // token blocks of the GEMM form (the fastest-varying block index)
};

// ------------------------------------------------------------- one or two tokens
// The linear's decode kernel (gemv.hip) with R = 2 RP rows per wave: rows
// 0 .. RP - 1 of the wave are gate's, RP .. 2 RP - 1 the same rows of up.
template <int M, bool MMA, int RP>
__device__ __forceinline__ void gated_gemv_body(const GatedArgs& a)
{
    constexpr int R = 2 * RP;
    static_assert(R <= 4, "a wave's rows are reduced four at once");
    constexpr int TT = kChunkTiles;
    constexpr int GC = 64 * TT;  // groups per chunk
    extern __shared__ uint4 smem[];
    const uint16_t* __restrict__ X = a.x;
    const int N = a.N, K = a.K;
    const int G = K >> 5;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int brow = (int)blockIdx.x * 4 * RP;
    const int row0 = brow + wave * RP;
    const int nb = min(N - brow, 4 * RP);

    __amdgpu_buffer_rsrc_t qr[2];
#pragma unroll
    for (int l = 0; l < 2; l++)
        qr[l] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(a.L[l].q) + (int64_t)brow * G * 3, (short)0,
                                                  nb * G * 12, 0x00020000);
    int vrow[RP];
#pragma unroll
    for (int r = 0; r < RP; r++)
        vrow[r] = (wave * RP + r) * G * 12 + lane * 12;

    constexpr int PC = 4 * GC;
    constexpr int XP = M * PC / 256;
    uint4 xg[XP];
    u32x3 cw[R][TT];
    // every load unconditional (clamped): one under a branch would be waited for
    // at the branch's end
    auto issue_chunk = [&](int g0, int gc) {
#pragma unroll
        for (int t = 0; t < XP; t++) {
            const int i = tid + 256 * t;
            const int m = i / PC, pc = min(i % PC, 4 * gc - 1);
            xg[t] = *reinterpret_cast<const uint4*>(X + m * K + g0 * 32 + pc * 8);
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int u = 0; u < TT; u++)
                cw[r][u] = __builtin_amdgcn_raw_buffer_load_b96(qr[r / RP], vrow[r % RP] + (g0 + 64 * u) * 12, 0,
                                                                kNonTemporal);
    };

    uint32_t sv[R], zv[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = min(row0 + r % RP, N - 1);
        sv[r] = a.L[r / RP].s[row];
        zv[r] = a.L[r / RP].z[row];
    }
    const int kc[2] = {max(a.L[0].k, 1), max(a.L[1].k, 1)};  // with k == 0 the host passes valid dummy arrays
    int widx[2][2];
#pragma unroll
    for (int l = 0; l < 2; l++)
#pragma unroll
        for (int v = 0; v < 2; v++)
            widx[l][v] = a.L[l].idx[min(lane + 64 * v, kc[l] - 1)];
    asm volatile("" ::: "memory");
    issue_chunk(0, min(GC, G));
    float wwv[R][2], xw[2][M][2];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const PairLayer& L = a.L[r / RP];
        const int row = min(row0 + r % RP, N - 1);
#pragma unroll
        for (int v = 0; v < 2; v++) {
            const int c = lane + 64 * v;
            const float w = h2f(L.ww[(int64_t)row * L.k + min(c, kc[r / RP] - 1)]);
            wwv[r][v] = c < L.k ? w : 0.0f;
        }
    }
#pragma unroll
    for (int l = 0; l < 2; l++)
#pragma unroll
        for (int v = 0; v < 2; v++) {
            const int c = lane + 64 * v;
            int j = widx[l][v];
            j = (j >= 0 && j < K) ? j : 0;
#pragma unroll
            for (int m = 0; m < M; m++) {
                const float xv = h2f(X[(int64_t)m * K + j]);
                xw[l][m][v] = c < a.L[l].k ? xv : 0.0f;
            }
        }

    float sc[R];
    uint32_t zr[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        sc[r] = h2f((uint16_t)__builtin_amdgcn_readfirstlane((int)sv[r]));
        zr[r] = (uint32_t)__builtin_amdgcn_readfirstlane((int)zv[r]);
    }
    const Magic mg = make_magic();
    float acc[R][M];
    f32x4 macc[MMA ? R : 1][MMA ? M : 1];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int m = 0; m < M; m++) {
            acc[r][m] = 0.0f;
            if (MMA)
                macc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }

    for (int g0 = 0; g0 < G; g0 += GC) {
        const int gc = min(GC, G - g0);
        if (g0 > 0) {
            __syncthreads();
            issue_chunk(g0, gc);
        }
#pragma unroll
        for (int t = 0; t < XP; t++) {
            const int i = tid + 256 * t;
            const int pc = i % PC;
            const bool on = pc < 4 * gc;
            if (MMA)  // every slot is written: x, or zeros past the chunk's groups
                smem[xs_slot(i / PC, TT, pc >> 2, pc & 3)] =
                    make_uint4(on ? xg[t].x : 0u, on ? xg[t].y : 0u, on ? xg[t].z : 0u, on ? xg[t].w : 0u);
            else if (on)
                smem[xs_slot(i / PC, TT, pc >> 2, pc & 3)] = make_uint4(xg[t].x, xg[t].y, xg[t].z, xg[t].w);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < TT; u++) {
            const int g = (u << 6) + lane;
            if constexpr (MMA) {
                auto quad = [&](auto qdc) {
                    constexpr int qd = decltype(qdc)::value;
                    uint4 xv[M];
#pragma unroll
                    for (int m = 0; m < M; m++)
                        xv[m] = smem[xs_slot(m, TT, g, qd)];
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        uint32_t p[4];
                        decode_quad<qd>(cw[r][u].x, cw[r][u].y, cw[r][u].z, mg, make_zero_sub(zr[r]), p);
                        const half8_t bq = pair_h8(p[0], p[1], p[2], p[3]);
#pragma unroll
                        for (int m = 0; m < M; m++)
                            macc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, xv[m]), bq,
                                                                                macc[r][m], 0, 0, 0);
                    }
                };
                quad(std::integral_constant<int, 0>{});
                quad(std::integral_constant<int, 1>{});
                quad(std::integral_constant<int, 2>{});
                quad(std::integral_constant<int, 3>{});
            } else {
                uint4 xq[M][4];
#pragma unroll
                for (int m = 0; m < M; m++)
#pragma unroll
                    for (int qd = 0; qd < 4; qd++)
                        xq[m][qd] = smem[xs_slot(m, TT, g, qd)];
                if (g < gc) {
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        uint32_t p[16];
                        decode_group(cw[r][u].x, cw[r][u].y, cw[r][u].z, mg, make_zero_sub(zr[r]), p);
#pragma unroll
                        for (int m = 0; m < M; m++) {
                            float t = acc[r][m];
#pragma unroll
                            for (int qd = 0; qd < 4; qd++) {
                                t = dot2(p[4 * qd + 0], xq[m][qd].x, t);
                                t = dot2(p[4 * qd + 1], xq[m][qd].y, t);
                                t = dot2(p[4 * qd + 2], xq[m][qd].z, t);
                                t = dot2(p[4 * qd + 3], xq[m][qd].w, t);
                            }
                            acc[r][m] = t;
                        }
                    }
                }
            }
        }
    }

    if constexpr (MMA) {  // each lane's own products lie on the diagonal of the 16 x 16 results (see gemv.hip)
        const bool diag = (lane >> 4) == ((lane & 15) >> 2);
        const int e = lane & 3;
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int m = 0; m < M; m++) {
                const f32x4 c = macc[r][m];
                const float v = e == 0 ? c[0] : e == 1 ? c[1] : e == 2 ? c[2] : c[3];
                acc[r][m] = diag ? v : 0.0f;
            }
    }

#pragma unroll
    for (int m = 0; m < M; m++) {
        float part[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            part[r] = 0.0f;
            if (r < R) {
                part[r] = sc[r] * acc[r][m];
#pragma unroll
                for (int v = 0; v < 2; v++)
                    part[r] += wwv[r][v] * xw[r / RP][m][v];
            }
        }
        auto tail = [&](const PairLayer& L, int r, float& sum) {  // weak columns from the 129th, from global memory
            const int row = min(row0 + r, N - 1);
            for (int c = lane + 128; c < L.k; c += 64) {
                int j = L.idx[c];
                j = (j >= 0 && j < K) ? j : 0;
                sum += h2f(L.ww[(int64_t)row * L.k + c]) * h2f(X[(int64_t)m * K + j]);
            }
        };
#pragma unroll
        for (int r = 0; r < R; r++)
            tail(a.L[r / RP], r % RP, part[r]);
        reduce4(part);  // lanes 16 q .. 16 q + 15: the total of row reduced_index(q) = q
        const float gv = part[0], uv = __shfl(part[0], (lane + 16 * RP) & 63, 64);
        const int row = row0 + (lane >> 4);
        if ((lane & 15) == 0 && (lane >> 4) < RP && row < N) {
            const int64_t o = (int64_t)m * N + row;
            with_act(a.act, [&](auto act) { a.h[o] = f2h(act_value<decltype(act)::value>(gv) * uv); });
            if (a.g) {
                a.g[o] = gv;
                a.u[o] = uv;
            }
        }
    }
}

template <int M, bool MMA, int RP>
__global__ __launch_bounds__(256) void k_gated_gemv(const GatedArgs a)
{
    gated_gemv_body<M, MMA, RP>(a);
}

// ------------------------------------------------------------- up to 16 tokens
// The linear's matrix-core decode (mfv.hip) with a wave's 16 rows taken from both
// layers: each chunk's codes of gate, then of up, go through the wave's LDS rows
// (one after the other: LDS serves a wave in order), and both meet the same x
// operands. U, MC, W, S, D as there.
template <int U, int MC>
struct GatedShape {
    static constexpr int GC = 4 * U;
    static constexpr int RS = GC * 64 + 16;
    static constexpr int STAGE = MC * RS;
    static constexpr int PT = GC / 16;
    static constexpr int CRS = GC * 12 + 16;
    static constexpr int CQ = GC * 12 / 16;
    static constexpr int CL = 16 * CQ / 64;
    static_assert(GC % 16 == 0 && (16 * CQ) % 64 == 0 && CRS % 16 == 0, "codes and x must split evenly");
};

template <int U, int MC, int W, int S, int D>
__global__ __launch_bounds__(64 * W * S) void k_gated_mfv(const GatedArgs a)
{
    using SH = GatedShape<U, MC>;
    constexpr int GC = SH::GC, RS = SH::RS, STAGE = SH::STAGE, PT = SH::PT;
    constexpr int DPW = MC * PT / W;
    constexpr int kCodePolicy = MC >= 8 ? 2 : 0;
    static_assert((MC * PT) % W == 0, "x loads must split evenly over the waves");
    constexpr int CRS = SH::CRS, CQ = SH::CQ, CL = SH::CL;
    __shared__ __attribute__((aligned(1024))) char xs0[S][STAGE];
    __shared__ __attribute__((aligned(1024))) char xs1[S][STAGE];
    __shared__ __attribute__((aligned(1024))) char xs2[D == 2 ? S : 1][D == 2 ? STAGE : 16];
    __shared__ __attribute__((aligned(16))) char cs[W * S][16 * CRS];
    static_assert(S == 1 || (S - 1) * W * 2 * 64 * 16 <= STAGE * S, "partial sums must fit in one stage set");

    const int M = a.M, N = a.N, K = a.K;
    const int G = K >> 5;
    const int nch = (G + GC - 1) / GC;
    const int per = (nch + S - 1) / S;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = wid % W, kg = wid / W;
    const int c0 = kg * per, c1 = min(nch, c0 + per);
    const int l16 = lane & 15, qd = lane >> 4;
    const int brow = (int)blockIdx.x * 16 * W;
    const int nb = min(N - brow, 16 * W);
    const int rloc = min(wave * 16 + l16, nb - 1);

    __amdgpu_buffer_rsrc_t qr[2];
#pragma unroll
    for (int l = 0; l < 2; l++)
        qr[l] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(a.L[l].q) + (int64_t)brow * G * 3, (short)0,
                                                  nb * G * 12, 0x00020000);
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.x), (short)0, M * K * 2, 0x00020000);

    // chunks past the group's range and groups past K are read out of the buffers'
    // range, which gives zeros and fetches nothing
    auto dma = [&](int c, char* stage) {
        const int cc = min(c, c1 - 1);
        const int dead = c >= c1 ? 0x40000000 : 0;
#pragma unroll
        for (int t = 0; t < DPW; t++) {
            const int qi = wave * DPW + t;
            const int m = qi / PT, part = qi % PT;
            const int g = cc * GC + part * 16 + (lane >> 2);
            const int off = (min(m, M - 1) * K + g * 32) * 2 + (lane & 3) * 16;
            pair_dma(xr, stage + m * RS + part * 1024, off + (g >= G ? 0x40000000 : dead));
        }
    };
    typedef uint4 QRegs[2][CL];
    auto load_q = [&](int c, QRegs& cw) {
        const int cc = min(c, c1 - 1);
        const int dead = c >= c1 ? 0x40000000 : 0;
#pragma unroll
        for (int l = 0; l < 2; l++)
#pragma unroll
            for (int i = 0; i < CL; i++) {
                const int pc = 64 * i + lane;
                const int r = pc / CQ, o = (pc % CQ) * 16;
                cw[l][i] = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(qr[l], ((wave * 16 + r) * G + cc * GC) * 12 + o + dead,
                                                                 0, kCodePolicy));
            }
    };
    char* const crow = cs[wid];

    float sc[2];
    ZeroSub zs[2];
#pragma unroll
    for (int l = 0; l < 2; l++) {
        sc[l] = h2f(a.L[l].s[brow + rloc]);
        zs[l] = make_zero_sub((uint32_t)a.L[l].z[brow + rloc]);
    }
    const Magic mg = make_magic();
    constexpr int AU = U < 4 ? U : 4;  // accumulators per layer: the MFMAs of different groups do not wait for one another
    f32x4 accu[2][AU];
#pragma unroll
    for (int l = 0; l < 2; l++)
#pragma unroll
        for (int u = 0; u < AU; u++)
            accu[l][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int arow = min(l16, M - 1) * RS + qd * 64;
    auto step = [&](int c, const char* cur, char* nxt, const QRegs& qc, QRegs& qn) {
        // x of chunk c has arrived once at most the newer loads remain: codes of
        // c, then x and codes of c + 1 .. c + D - 1
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(D * 2 * CL + (D - 1) * DPW) : "memory");
        dma(c + D, nxt);
        load_q(c + D, qn);
        if (c < c1) {  // wave-uniform
#pragma unroll
            for (int l = 0; l < 2; l++) {
#pragma unroll
                for (int i = 0; i < CL; i++) {
                    const int pc = 64 * i + lane;
                    *reinterpret_cast<uint4*>(crow + (pc / CQ) * CRS + (pc % CQ) * 16) = qc[l][i];
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const uint32_t* gw = reinterpret_cast<const uint32_t*>(crow + l16 * CRS + (4 * u + qd) * 12);
                    uint32_t p[16];
                    decode_group(gw[0], gw[1], gw[2], mg, zs[l], p);
#pragma unroll
                    for (int st = 0; st < 4; st++) {
                        const half8_t av = __builtin_bit_cast(
                            half8_t, *reinterpret_cast<const uint4*>(cur + arow + 4 * u * 64 + st * 16));
                        accu[l][u % AU] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            av, pair_h8(p[4 * st], p[4 * st + 1], p[4 * st + 2], p[4 * st + 3]), accu[l][u % AU], 0, 0, 0);
                    }
                }
            }
        }
    };

    QRegs qa, qb, qc3;
    dma(c0, xs0[kg]);
    load_q(c0, qa);
    asm volatile("" ::: "memory");
    if constexpr (D == 2) {
        dma(c0 + 1, xs1[kg]);
        load_q(c0 + 1, qb);
        asm volatile("" ::: "memory");
        for (int c = c0; c < c0 + per; c += 3) {  // the same trip count in every group
            step(c, xs0[kg], xs2[kg], qa, qc3);
            step(c + 1, xs1[kg], xs0[kg], qb, qa);
            step(c + 2, xs2[kg], xs1[kg], qc3, qb);
        }
    } else {
        for (int c = c0; c < c0 + per; c += 2) {
            step(c, xs0[kg], xs1[kg], qa, qb);
            step(c + 1, xs1[kg], xs0[kg], qb, qa);
        }
    }
    // no x load may write LDS after this point (the stages are reused below)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    f32x4 acc[2];
#pragma unroll
    for (int l = 0; l < 2; l++) {
        acc[l] = accu[l][0];
#pragma unroll
        for (int u = 1; u < AU; u++)
            acc[l] += accu[l][u];
    }

    if constexpr (S > 1) {  // K groups 1 .. S - 1 hand their sums to group 0
        f32x4* part = reinterpret_cast<f32x4*>(&xs0[0][0]);
        __syncthreads();
        if (kg > 0)
#pragma unroll
            for (int l = 0; l < 2; l++)
                part[(((kg - 1) * W + wave) * 2 + l) * 64 + lane] = acc[l];
        __syncthreads();
        if (kg > 0)
            return;
#pragma unroll
        for (int g2 = 1; g2 < S; g2++)
#pragma unroll
            for (int l = 0; l < 2; l++)
                acc[l] += part[(((g2 - 1) * W + wave) * 2 + l) * 64 + lane];
    }

    // row steps, then the weak columns as 32-deep steps: B = w_weak, A = x gathered
    const uint16_t* xm = a.x + (int64_t)min(l16, M - 1) * K;
#pragma unroll
    for (int l = 0; l < 2; l++) {
        const PairLayer& L = a.L[l];
        acc[l] *= sc[l];
        const uint16_t* wr = L.ww + (int64_t)(brow + rloc) * L.k;
        for (int cs2 = 0; cs2 < L.k; cs2 += 32) {
            uint32_t bw[4], aw[4];
#pragma unroll
            for (int e2 = 0; e2 < 4; e2++) {
                uint32_t wv[2], xv[2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int c = cs2 + 8 * qd + 2 * e2 + h;
                    const bool on = c < L.k;
                    int j = L.idx[min(c, L.k - 1)];
                    j = (j >= 0 && j < K) ? j : 0;
                    wv[h] = on ? (uint32_t)wr[min(c, L.k - 1)] : 0u;
                    xv[h] = on ? (uint32_t)xm[j] : 0u;
                }
                bw[e2] = wv[0] | (wv[1] << 16);
                aw[e2] = xv[0] | (xv[1] << 16);
            }
            acc[l] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pair_h8(aw[0], aw[1], aw[2], aw[3]),
                                                           pair_h8(bw[0], bw[1], bw[2], bw[3]), acc[l], 0, 0, 0);
        }
    }

    // D element r of lane l: token 4 (l / 16) + r, row l % 16
    const int row = wave * 16 + l16;
    if (row < nb)
        with_act(a.act, [&](auto act) {
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int m = 4 * qd + r;
                if (m < M) {
                    const int64_t o = (int64_t)m * N + brow + row;
                    a.h[o] = f2h(act_value<decltype(act)::value>(acc[0][r]) * acc[1][r]);
                    if (a.g) {
                        a.g[o] = acc[0][r];
                        a.u[o] = acc[1][r];
                    }
                }
            }
        });
}

// ------------------------------------------------------------- prompts, training
// The pair product (owq_pair_gemm.h) with gate's rows as one set and up's as the
// other: a wave has the same tokens and rows of both.
template <int FM, int WN, int S>
__global__ __launch_bounds__(64 * WN * S) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_gated_gemm(const GatedArgs a)
{
    using T = PairTile<FM, WN, S>;
    const int M = a.M, N = a.N;
    const int m0 = ((int)blockIdx.x % a.mblocks) * T::BM;
    const int n0 = ((int)blockIdx.x / a.mblocks) * T::BN;
    const int rows[2] = {n0, n0};
    f32x16 acc[2][FM];
    if (!pair_gemm<FM, WN, S, false>(a.L, a.x, nullptr, M, N, a.K, m0, rows, acc))
        return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wid = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), kg = wid / WN;
    const int n = n0 + wid % WN * 32 + l32;
    // D element r of lane l: token 8 (r / 4) + 4 h + r % 4, row l % 32; of these the
    // waves hold their K group's share
    constexpr int REGS = S > 1 && T::SHARE == 1 ? 4 : 16;
    const int mt = m0 + 4 * h + kg * (REGS == 4 ? 8 : T::SHARE > 1 ? 32 * T::OWN : 0);
    with_act(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < T::OWN; i++)
#pragma unroll
            for (int r = 0; r < REGS; r++) {
                const int m = mt + 32 * i + 8 * (r >> 2) + (r & 3);
                if (m < M && n < N) {
                    const int64_t o = (int64_t)m * N + n;
                    const float gv = acc[0][i][r], uv = acc[1][i][r];
                    a.h[o] = f2h(act_value<decltype(act)::value>(gv) * uv);
                    if (a.g) {
                        a.g[o] = gv;
                        a.u[o] = uv;
                    }
                }
            }
    });
}

template <int M, bool MMA, int RP>
hipError_t gated_gemv(const GatedArgs& a, hipStream_t s)
{
    const int nblocks = (a.N + 4 * RP - 1) / (4 * RP);
    if (!grid_fits(nblocks, 256))
        return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)M * kChunkTiles * 4 * kQuadStride * 16;
    hipLaunchKernelGGL((k_gated_gemv<M, MMA, RP>), dim3(nblocks), dim3(256), lds, s, a);
    return hipGetLastError();
}

template <int U, int MC, int W, int S, int D>
hipError_t gated_mfv(const GatedArgs& a, hipStream_t s)
{
    const int nblocks = (a.N + 16 * W - 1) / (16 * W);
    if (!grid_fits(nblocks, 64 * W * S))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_gated_mfv<U, MC, W, S, D>), dim3(nblocks), dim3(64 * W * S), 0, s, a);
    return hipGetLastError();
}

template <int FM, int WN, int S>
hipError_t gated_gemm(GatedArgs a, hipStream_t s)
{
    using T = PairTile<FM, WN, S>;
    a.mblocks = (int)(((int64_t)a.M + T::BM - 1) / T::BM);
    const int64_t nblocks = (int64_t)a.mblocks * (((int64_t)a.N + T::BN - 1) / T::BN);
    if (!grid_fits(nblocks, T::NT))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_gated_gemm<FM, WN, S>), dim3((unsigned)nblocks), dim3(T::NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated(const LinearDesc& gate, const LinearDesc& up, int64_t M, int act, uint16_t* h, float* g,
                        float* u, hipStream_t s)
{
    GatedArgs a{{pair_layer(gate), pair_layer(up)}, gate.x, h, g, u, (int32_t)M, (int32_t)gate.N, (int32_t)gate.K, act, 1};
    // Enough rows for four per wave: 1024 blocks of 8 rows of each layer stay busy
    // longer than the launch takes to fill and drain. 28672 x 8192, us with four /
    // two rows: M = 1 42.9 / 47.7, M = 2 50.6 / 66.4; 11008 x 4096: 11.2 / 10.7 and
    // 14.5 / 14.3 (two rows of two tokens: v_dot2, 16.3 on the matrix cores)
    const bool many = gate.N >= 16384;
    if (M == 1)
        return many ? gated_gemv<1, false, 2>(a, s) : gated_gemv<1, false, 1>(a, s);
    if (M == 2)
        return many ? gated_gemv<2, true, 2>(a, s) : gated_gemv<2, false, 1>(a, s);
    // 4 row waves, or 2 x 2 K groups where the rows are few: us at M = 4, 28672 x
    // 8192 46.7 / 53.0, 11008 x 4096 18.0 / 16.1; M = 8 48.1 / 55.0, 17.3 / 18.3, 2731 x
    // 1056 10.1 / 8.7; M = 16 53.6 / 58.5, 18.2 / 20.4, 11.1 / 9.6 (codes two chunks
    // ahead leave one wave per SIMD: 63 at M = 8)
    if (M <= 4)
        return many ? gated_mfv<4, 4, 4, 1, 1>(a, s) : gated_mfv<4, 4, 2, 2, 1>(a, s);
    const bool few = gate.N < 8192;
    if (M <= 8)
        return few ? gated_mfv<4, 8, 2, 2, 1>(a, s) : gated_mfv<4, 8, 4, 1, 1>(a, s);
    if (M <= 16)
        return few ? gated_mfv<4, 16, 2, 2, 1>(a, s) : gated_mfv<4, 16, 4, 1, 1>(a, s);
    return pair_tile(M, gate.N, [&](auto fm, auto wn, auto sk) {
        return gated_gemm<decltype(fm)::value, decltype(wn)::value, decltype(sk)::value>(a, s);
    });
}

}  // namespace owq
