// api.cpp -- the C ABI of libowq.so: synchronous argument validation, then
// kernel dispatch on the caller's stream. Declarations and the contract of
// every entry point are in include/owq.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <utility>
#include <vector>

#include "../../include/owq.h"
#include "owq_launch.h"

namespace {

thread_local char g_err[512] = "";

owq_status fail(owq_status s, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

// The last error again, prefixed with "<what> <i>: " (the message is copied
// first: formatting a buffer into itself is undefined).
owq_status fail_at(owq_status s, const char* what, int i)
{
    char msg[sizeof g_err];
    snprintf(msg, sizeof msg, "%s", g_err);
    return fail(s, "%s %d: %s", what, i, msg);
}

owq_status hip_status(hipError_t e, const char* what)
{
    if (e == hipSuccess) {
        g_err[0] = '\0';
        return OWQ_OK;
    }
    return fail(OWQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Of a launcher that checks its grids before it launches anything
owq_status launch_status(hipError_t e, const char* what)
{
    if (e == hipErrorInvalidConfiguration)
        return fail(OWQ_ERR_SHAPE, "%s: these sizes need more threads than one launch counts (2^32)", what);
    return hip_status(e, what);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxK = 65536;
constexpr int32_t kMaxRank = 256;    // of a low-rank adapter
constexpr int64_t kMaxBlock = (int64_t)1 << 30;  // tokens and rows of the gated block and the adapted linear
constexpr int32_t kMaxGrads = 4096;  // tensors per owq_clip_grad_norm and owq_orthogonalize
constexpr int32_t kMaxNsSteps = 16;

owq_status check_k_dim(int64_t K)
{
    if (K < 32 || K > kMaxK || K % 32 != 0)
        return fail(OWQ_ERR_SHAPE, "K = %lld: need 32 <= K <= %lld and K %% 32 == 0", (long long)K,
                    (long long)kMaxK);
    return OWQ_OK;
}

bool check_enabled()
{
    static const bool on = [] {
        const char* e = getenv("OWQ_CHECK");
        return e && e[0] == '1';
    }();
    return on;
}

// Optional (OWQ_CHECK=1): synchronous copy of weak_idx and a host check that it
// is strictly ascending inside [0, K).
owq_status check_idx_on_host(const int32_t* idx, int32_t k, int64_t K, hipStream_t s)
{
    if (!check_enabled() || k == 0)
        return OWQ_OK;
    std::vector<int32_t> h((size_t)k);
    hipError_t e = hipMemcpyAsync(h.data(), idx, (size_t)k * sizeof(int32_t), hipMemcpyDeviceToHost, s);
    if (e == hipSuccess)
        e = hipStreamSynchronize(s);
    if (e != hipSuccess)
        return hip_status(e, "OWQ_CHECK copy of weak_idx");
    for (int32_t c = 0; c < k; c++) {
        if (h[c] < 0 || h[c] >= K || (c > 0 && h[c] <= h[c - 1]))
            return fail(OWQ_ERR_RANGE, "weak_idx[%d] = %d is not strictly ascending in [0, %lld)", c, h[c],
                        (long long)K);
    }
    return OWQ_OK;
}

owq_status check_layer(const owq_layer* L, int64_t M, const uint16_t* x, const uint16_t* y)
{
    if (!L)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    if (L->bits != 3)
        return fail(OWQ_ERR_UNSUPPORTED, "bits = %d: only 3-bit codes are supported", L->bits);
    if (L->N < 1 || L->N > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)L->N);
    owq_status st = check_k_dim(L->K);
    if (st != OWQ_OK)
        return st;
    if (M < 1 || M > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "M = %lld out of range", (long long)M);
    if (L->k < 0 || L->k > L->K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", L->k, (long long)L->K);
    if (!L->qcodes || !L->scales || !L->zeros || !x || !y)
        return fail(OWQ_ERR_NULL, "qcodes, scales, zeros, x and y must be non-NULL");
    if (L->k > 0 && (!L->weak_idx || !L->w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(x, 16) || !aligned(L->qcodes, 4) || !aligned(L->scales, 2) || !aligned(y, 2) ||
        (L->k > 0 && (!aligned(L->weak_idx, 4) || !aligned(L->w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (x: 16 B, qcodes/weak_idx: 4 B, fp16 arrays: 2 B)");
    return OWQ_OK;
}

owq::LinearDesc desc_of(const owq_layer* L, const uint16_t* x, uint16_t* y)
{
    owq::LinearDesc d;
    d.q = L->qcodes;
    d.s = L->scales;
    d.z = L->zeros;
    d.idx = L->k > 0 ? L->weak_idx : nullptr;
    d.ww = L->k > 0 ? L->w_weak : nullptr;
    d.x = x;
    d.y = y;
    d.N = L->N;
    d.K = L->K;
    d.k = L->k;
    return d;
}

// An array of a call, for the checks that none of its outputs lies over another array
struct Span {
    const char* name;
    const void* p;  // NULL: not given
    uint64_t bytes;
};

bool overlap(const Span& a, const Span& b)
{
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && (pa < pb ? a.bytes > pb - pa : b.bytes > pa - pb);
}

owq_status check_apart(const Span& out, std::initializer_list<Span> others)
{
    for (const Span& s : others)
        if (overlap(out, s))
            return fail(OWQ_ERR_RANGE, "%s overlaps %s", out.name, s.name);
    return OWQ_OK;
}

// One tensor of a list whose outputs are written beside each other: out may be its own
// g, and is otherwise disjoint from every g and every other out.
struct InOut {
    const void* g;
    const void* out;
    uint64_t bytes;
};
owq_status check_list_apart(const std::vector<InOut>& list)
{
    std::vector<std::pair<uintptr_t, uintptr_t>> outs;  // [begin, end) of the non-empty outputs
    outs.reserve(list.size());
    for (const InOut& t : list)
        if (t.bytes > 0)
            outs.emplace_back((uintptr_t)t.out, (uintptr_t)t.out + t.bytes);
    std::sort(outs.begin(), outs.end());
    for (size_t i = 1; i < outs.size(); i++)
        if (outs[i].first < outs[i - 1].second)
            return fail(OWQ_ERR_RANGE, "two outputs overlap (a tensor listed twice?)");
    for (size_t i = 0; i < list.size(); i++) {
        const InOut& t = list[i];
        if (t.bytes == 0)
            continue;
        // the one output that begins in or reaches into [b, e): the last that begins below e
        const uintptr_t b = (uintptr_t)t.g, e = b + t.bytes;
        auto o = std::lower_bound(outs.begin(), outs.end(), std::make_pair(e, (uintptr_t)0));
        const bool hit = o != outs.begin() && (o - 1)->second > b;
        if (hit && !(t.out == t.g && (o - 1)->first == b))
            return fail(OWQ_ERR_RANGE, "item %zu: g overlaps an output that is not its own", i);
    }
    return OWQ_OK;
}

// (a scale, zero point or index that lies under an output is as wrong as a code)
owq_status check_apart(const Span& out, const owq_layer* L)
{
    const uint64_t N = (uint64_t)L->N, K = (uint64_t)L->K, k = (uint64_t)L->k;
    return check_apart(out, {{"qcodes", L->qcodes, N * K / 8 * 3},
                             {"scales", L->scales, 2 * N},
                             {"zeros", L->zeros, N},
                             {"weak_idx", L->weak_idx, 4 * k},
                             {"w_weak", L->w_weak, 2 * N * k}});
}

// --- integer form

bool int8_sizes_ok(int64_t N, int64_t K, int32_t k, int64_t M)
{
    return N >= 1 && N <= kMaxBlock && K >= 32 && K <= kMaxK && K % 32 == 0 && k >= 0 && k <= K && M >= 1 &&
           M <= kMaxBlock && owq::int8_grid_fits(M, N, K);
}

owq_status check_int8_layer(const owq_integer_layer* L, int64_t M, const uint16_t* x, const uint16_t* y, hipStream_t s)
{
    if (!L)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    if (L->N < 1 || L->N > kMaxBlock)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)L->N);
    owq_status st = check_k_dim(L->K);
    if (st != OWQ_OK)
        return st;
    if (M < 1 || M > kMaxBlock)
        return fail(OWQ_ERR_SHAPE, "M = %lld out of range", (long long)M);
    if (L->k < 0 || L->k > L->K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", L->k, (long long)L->K);
    if (!L->codes || !L->scales || !x || !y)
        return fail(OWQ_ERR_NULL, "codes, scales, x and y must be non-NULL");
    if (L->k > 0 && (!L->weak_idx || !L->w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(x, 16) || !aligned(L->codes, 16) || !aligned(L->scales, 4) || !aligned(y, 2) ||
        (L->k > 0 && (!aligned(L->weak_idx, 4) || !aligned(L->w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (x, codes: 16 B, scales, weak_idx: 4 B, fp16 arrays: 2 B)");
    if (!owq::int8_grid_fits(M, L->N, L->K))
        return launch_status(hipErrorInvalidConfiguration, "integer form");
    return check_idx_on_host(L->weak_idx, L->k, L->K, s);
}

owq_status check_apart(const Span& out, const owq_integer_layer* L)
{
    const uint64_t N = (uint64_t)L->N, K = (uint64_t)L->K, k = (uint64_t)L->k;
    return check_apart(out, {{"codes", L->codes, N * K},
                             {"scales", L->scales, 4 * N},
                             {"weak_idx", L->weak_idx, 4 * k},
                             {"w_weak", L->w_weak, 2 * N * k}});
}

// y and the workspace of a product: large enough, and apart from everything read
owq_status check_int8_spans(const owq_integer_layer* L, const uint16_t* x, int64_t M, const uint16_t* y, const void* workspace,
                            size_t need, size_t have)
{
    if (need > 0 && !workspace)
        return fail(OWQ_ERR_NULL, "workspace must be non-NULL above %d tokens", owq::kInt8GemvMaxM);
    if (need > 0 && !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (workspace: 256 B)");
    if (have < need)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", have, need);
    const Span sx{"x", x, 2 * (uint64_t)M * (uint64_t)L->K}, sy{"y", y, 2 * (uint64_t)M * (uint64_t)L->N};
    const Span ws{"workspace", workspace, need};
    owq_status st = check_apart(sy, {sx, ws});
    st = st != OWQ_OK ? st : check_apart(ws, {sx});
    for (const Span* out : {&sy, &ws})
        st = st != OWQ_OK ? st : check_apart(*out, L);
    return st;
}

owq::Int8Desc int8_desc(const owq_integer_layer* L, const uint16_t* x, uint16_t* y)
{
    return owq::Int8Desc{L->codes, L->scales, L->k > 0 ? L->weak_idx : nullptr, L->k > 0 ? L->w_weak : nullptr, x, y,
                         L->N, L->K, L->k};
}

// The two layers of a gated block, its input and an fp16 output.
owq_status check_gated(const owq_layer* gate, const owq_layer* up, int64_t M, const uint16_t* x, const uint16_t* h,
                       int32_t act, hipStream_t s)
{
    owq_status st = check_layer(gate, M, x, h);
    if (st != OWQ_OK)
        return fail_at(st, "layer", 0);
    st = check_layer(up, M, x, h);
    if (st != OWQ_OK)
        return fail_at(st, "layer", 1);
    if (M > kMaxBlock || gate->N > kMaxBlock)
        return fail(OWQ_ERR_SHAPE, "M = %lld, N = %lld: need at most 2^30", (long long)M, (long long)gate->N);
    if (gate->N != up->N || gate->K != up->K)
        return fail(OWQ_ERR_SHAPE, "gate is %lld x %lld, up is %lld x %lld", (long long)gate->N, (long long)gate->K,
                    (long long)up->N, (long long)up->K);
    if (act < OWQ_ACT_SILU || act > OWQ_ACT_RELU)
        return fail(OWQ_ERR_UNSUPPORTED, "act = %d is not an owq_activation", act);
    st = check_idx_on_host(gate->weak_idx, gate->k, gate->K, s);
    return st != OWQ_OK ? st : check_idx_on_host(up->weak_idx, up->k, up->K, s);
}

}  // namespace

namespace owq {

hipError_t launch_linear_any(const LinearDesc& d, int64_t M, hipStream_t s)
{
    if (M >= gemm_min_m())
        return launch_gemm(d, M, s);
    // decode kernels, in token slices of the chosen kernel's capacity
    hipError_t e = hipSuccess;
    for (int64_t m0 = 0; m0 < M && e == hipSuccess;) {
        const bool mat = decode_on_matrix_cores(M - m0);
        const int64_t cap = mat ? kMfvMaxM : gemv_max_tokens(d.K);
        const int64_t mm = M - m0 < cap ? M - m0 : cap;
        LinearDesc dm = d;
        dm.x = d.x + m0 * d.K;
        dm.y = d.y + m0 * d.N;
        e = mat ? launch_mfv(&dm, 1, (int)mm, s) : launch_gemv(&dm, 1, (int)mm, s);
        m0 += mm;
    }
    return e;
}

}  // namespace owq

extern "C" {

const char* owq_status_string(owq_status s)
{
    switch (s) {
    case OWQ_OK: return "OWQ_OK";
    case OWQ_ERR_NULL: return "OWQ_ERR_NULL: a required pointer is NULL";
    case OWQ_ERR_SHAPE: return "OWQ_ERR_SHAPE: a dimension is out of range";
    case OWQ_ERR_RANGE: return "OWQ_ERR_RANGE: k or an index is out of range";
    case OWQ_ERR_ALIGN: return "OWQ_ERR_ALIGN: a device pointer is misaligned";
    case OWQ_ERR_UNSUPPORTED: return "OWQ_ERR_UNSUPPORTED: unsupported configuration";
    case OWQ_ERR_WORKSPACE: return "OWQ_ERR_WORKSPACE: workspace too small";
    case OWQ_ERR_HIP: return "OWQ_ERR_HIP: HIP runtime error";
    }
    return "unknown owq_status";
}

const char* owq_last_error(void) { return g_err; }

size_t owq_calibrate_workspace_bytes(int64_t N, int64_t K, int64_t T)
{
    if (N < 1 || T < 1 || K < 32 || K > kMaxK || K % 32 != 0 || N > INT32_MAX)
        return 0;
    return owq::calib_plan(N, K, T).total;
}

owq_status owq_calibrate_score(const uint16_t* W, int64_t N, int64_t K, const uint16_t* X, int64_t T,
                               double* lambda, double* score, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    if (!W || !X || !lambda || !score || !workspace)
        return fail(OWQ_ERR_NULL, "W, X, lambda, score and workspace must be non-NULL");
    if (N < 1 || N > INT32_MAX || T < 1)
        return fail(OWQ_ERR_SHAPE, "N = %lld, T = %lld: need N, T >= 1", (long long)N, (long long)T);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (!aligned(W, 16) || !aligned(X, 16) || !aligned(lambda, 8) || !aligned(score, 8) ||
        !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W, X: 16 B, lambda/score: 8 B, workspace: 256 B)");
    owq::CalibPlan p = owq::calib_plan(N, K, T);
    if (workspace_bytes < p.total)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, p.total);
    return hip_status(owq::launch_calibrate(W, N, K, X, T, lambda, score, workspace, p,
                                            (hipStream_t)stream),
                      "owq_calibrate_score launch");
}

size_t owq_calibrate_batched_workspace_bytes(const owq_calib_item* items, int32_t count)
{
    if (!items || count < 1 || count > 64)
        return 0;
    size_t total = 0;
    for (int32_t l = 0; l < count; l++) {
        const size_t b = owq_calibrate_workspace_bytes(items[l].N, items[l].K, items[l].T);
        if (b == 0)
            return 0;
        total += (b + 255) & ~(size_t)255;
    }
    return total;
}

owq_status owq_calibrate_score_batched(const owq_calib_item* items, int32_t count, void* workspace,
                                       size_t workspace_bytes, void* stream)
{
    if (!items || !workspace)
        return fail(OWQ_ERR_NULL, "items and workspace must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    if (!aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned workspace (256 B)");
    std::vector<owq::CalibItem> it((size_t)count);
    std::vector<owq::CalibPlan> plans((size_t)count);
    std::vector<void*> ws((size_t)count);
    size_t off = 0;
    for (int32_t l = 0; l < count; l++) {
        const owq_calib_item& c = items[l];
        if (!c.W || !c.X || !c.lambda || !c.score)
            return fail(OWQ_ERR_NULL, "item %d: W, X, lambda and score must be non-NULL", l);
        if (c.N < 1 || c.N > INT32_MAX || c.T < 1)
            return fail(OWQ_ERR_SHAPE, "item %d: N = %lld, T = %lld: need N, T >= 1", l, (long long)c.N,
                        (long long)c.T);
        owq_status st = check_k_dim(c.K);
        if (st != OWQ_OK)
            return fail_at(st, "item", l);
        if (!aligned(c.W, 16) || !aligned(c.X, 16) || !aligned(c.lambda, 8) || !aligned(c.score, 8))
            return fail(OWQ_ERR_ALIGN, "item %d: misaligned pointer (W, X: 16 B, lambda/score: 8 B)", l);
        it[l] = owq::CalibItem{c.W, c.N, c.K, c.X, c.T, c.lambda, c.score};
        plans[l] = owq::calib_plan(c.N, c.K, c.T);
        ws[l] = static_cast<char*>(workspace) + off;
        off += (plans[l].total + 255) & ~(size_t)255;
    }
    if (workspace_bytes < off)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, off);
    return hip_status(owq::launch_calibrate_batched(it.data(), count, ws.data(), plans.data(), (hipStream_t)stream),
                      "owq_calibrate_score_batched launch");
}

owq_status owq_calibrate_score_noalloc(const uint16_t* W, int64_t N, int64_t K, const uint16_t* X, int64_t T,
                                       double* lambda, double* score, void* stream)
{
    if (!W || !X || !lambda || !score)
        return fail(OWQ_ERR_NULL, "W, X, lambda and score must be non-NULL");
    if (N < 1 || N > INT32_MAX || T < 1)
        return fail(OWQ_ERR_SHAPE, "N = %lld, T = %lld: need N, T >= 1", (long long)N, (long long)T);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (!aligned(W, 16) || !aligned(X, 16) || !aligned(lambda, 8) || !aligned(score, 8))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W, X: 16 B, lambda/score: 8 B)");
    owq::CalibPlan p = owq::calib_plan(N, K, T);
    if (p.total > owq::kCalibScratchBytes)
        return fail(OWQ_ERR_WORKSPACE,
                    "N = %lld, K = %lld, T = %lld need %zu bytes of workspace; the library's own holds %zu "
                    "(use owq_calibrate_score with a caller workspace)",
                    (long long)N, (long long)K, (long long)T, p.total, owq::kCalibScratchBytes);
    void* ws = nullptr;
    hipError_t e = owq::calib_scratch(&ws);
    if (e != hipSuccess)
        return hip_status(e, "owq_calibrate_score_noalloc: scratch lookup");
    return hip_status(owq::launch_calibrate(W, N, K, X, T, lambda, score, ws, p, (hipStream_t)stream),
                      "owq_calibrate_score_noalloc launch");
}

size_t owq_calibrate_noalloc_max_workspace(void) { return owq::kCalibScratchBytes; }

owq_status owq_select_weak(const double* score, int64_t K, int32_t k, int32_t* weak_idx, void* stream)
{
    if (!score)
        return fail(OWQ_ERR_NULL, "score must be non-NULL");
    if (K < 1 || K > (int64_t)1 << 24)
        return fail(OWQ_ERR_SHAPE, "K = %lld: need 1 <= K <= 2^24", (long long)K);
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && !weak_idx)
        return fail(OWQ_ERR_NULL, "weak_idx must be non-NULL when k > 0");
    if (!aligned(score, 8) || (k > 0 && !aligned(weak_idx, 4)))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (score: 8 B, weak_idx: 4 B)");
    if (k == 0) {
        g_err[0] = '\0';
        return OWQ_OK;
    }
    return hip_status(owq::launch_select(score, K, k, weak_idx, (hipStream_t)stream),
                      "owq_select_weak launch");
}

owq_status owq_select_weak_batched(const double* const* scores, const int64_t* Ks, const int32_t* ks,
                                   int32_t* const* weak_idxs, int32_t count, void* stream)
{
    if (!scores || !Ks || !ks || !weak_idxs)
        return fail(OWQ_ERR_NULL, "scores, Ks, ks and weak_idxs must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    for (int32_t i = 0; i < count; i++) {
        const int64_t K = Ks[i];
        const int32_t k = ks[i];
        if (!scores[i])
            return fail(OWQ_ERR_NULL, "selection %d: score must be non-NULL", i);
        if (K < 1 || K > (int64_t)1 << 24)
            return fail(OWQ_ERR_SHAPE, "selection %d: K = %lld: need 1 <= K <= 2^24", i, (long long)K);
        if (k < 0 || k > K)
            return fail(OWQ_ERR_RANGE, "selection %d: k = %d outside [0, K = %lld]", i, k, (long long)K);
        if (k > 0 && !weak_idxs[i])
            return fail(OWQ_ERR_NULL, "selection %d: weak_idx must be non-NULL when k > 0", i);
        if (!aligned(scores[i], 8) || (k > 0 && !aligned(weak_idxs[i], 4)))
            return fail(OWQ_ERR_ALIGN, "selection %d: misaligned pointer (score: 8 B, weak_idx: 4 B)", i);
    }
    return hip_status(owq::launch_select_batched(scores, Ks, ks, weak_idxs, count, (hipStream_t)stream),
                      "owq_select_weak_batched launch");
}

owq_status owq_pack(const uint16_t* W, int64_t N, int64_t K, const int32_t* weak_idx, int32_t k,
                    uint32_t* qcodes, uint16_t* scales, uint8_t* zeros, uint16_t* w_weak, void* stream)
{
    if (!W || !qcodes || !scales || !zeros)
        return fail(OWQ_ERR_NULL, "W, qcodes, scales and zeros must be non-NULL");
    if (N < 1 || N > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)N);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && (!weak_idx || !w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(W, 16) || !aligned(qcodes, 4) || !aligned(scales, 2) ||
        (k > 0 && (!aligned(weak_idx, 4) || !aligned(w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W: 16 B, qcodes/weak_idx: 4 B, fp16: 2 B)");
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_pack(W, N, K, k > 0 ? weak_idx : nullptr, k, qcodes, scales, zeros,
                                       k > 0 ? w_weak : nullptr, (hipStream_t)stream),
                      "owq_pack launch");
}

owq_status owq_pack_batched(const owq_pack_item* items, int32_t count, void* stream)
{
    if (!items)
        return fail(OWQ_ERR_NULL, "items must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    std::vector<owq::PackItem> it((size_t)count);
    for (int32_t l = 0; l < count; l++) {
        const owq_pack_item& c = items[l];
        if (!c.W || !c.qcodes || !c.scales || !c.zeros)
            return fail(OWQ_ERR_NULL, "item %d: W, qcodes, scales and zeros must be non-NULL", l);
        if (c.N < 1 || c.N > INT32_MAX)
            return fail(OWQ_ERR_SHAPE, "item %d: N = %lld out of range", l, (long long)c.N);
        owq_status st = check_k_dim(c.K);
        if (st != OWQ_OK)
            return fail_at(st, "item", l);
        if (c.k < 0 || c.k > c.K)
            return fail(OWQ_ERR_RANGE, "item %d: k = %d outside [0, K = %lld]", l, c.k, (long long)c.K);
        if (c.k > 0 && (!c.weak_idx || !c.w_weak))
            return fail(OWQ_ERR_NULL, "item %d: weak_idx and w_weak must be non-NULL when k > 0", l);
        if (!aligned(c.W, 16) || !aligned(c.qcodes, 4) || !aligned(c.scales, 2) ||
            (c.k > 0 && (!aligned(c.weak_idx, 4) || !aligned(c.w_weak, 2))))
            return fail(OWQ_ERR_ALIGN, "item %d: misaligned pointer (W: 16 B, qcodes/weak_idx: 4 B, fp16: 2 B)", l);
        st = check_idx_on_host(c.weak_idx, c.k, c.K, (hipStream_t)stream);
        if (st != OWQ_OK)
            return fail_at(st, "item", l);
        it[l] = owq::PackItem{c.W, c.N, c.K, c.k > 0 ? c.weak_idx : nullptr, c.k, c.qcodes, c.scales, c.zeros,
                              c.k > 0 ? c.w_weak : nullptr};
    }
    return hip_status(owq::launch_pack_batched(it.data(), count, (hipStream_t)stream), "owq_pack_batched launch");
}

owq_status owq_pack_search(const uint16_t* W, int64_t N, int64_t K, const int32_t* weak_idx, int32_t k,
                           const double* lambda, uint32_t* qcodes, uint16_t* scales, uint8_t* zeros,
                           uint16_t* w_weak, void* stream)
{
    if (!W || !qcodes || !scales || !zeros)
        return fail(OWQ_ERR_NULL, "W, qcodes, scales and zeros must be non-NULL");
    if (N < 1 || N > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)N);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && (!weak_idx || !w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(W, 16) || !aligned(qcodes, 4) || !aligned(scales, 2) || !aligned(lambda, 8) ||
        (k > 0 && (!aligned(weak_idx, 4) || !aligned(w_weak, 2))))
        return fail(OWQ_ERR_ALIGN,
                    "misaligned pointer (W: 16 B, lambda: 8 B, qcodes/weak_idx: 4 B, fp16: 2 B)");
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    const int32_t* idx = k > 0 ? weak_idx : nullptr;
    hipError_t e = owq::launch_search(W, N, K, idx, k, lambda, scales, zeros, (hipStream_t)stream);
    if (e == hipSuccess)
        e = owq::launch_pack_given(W, N, K, idx, k, qcodes, scales, zeros, k > 0 ? w_weak : nullptr,
                                   (hipStream_t)stream);
    return hip_status(e, "owq_pack_search launch");
}

owq_status owq_pack_storage(const uint16_t* W, int64_t N, int64_t K, const int32_t* weak_idx, int32_t k,
                            uint32_t* qcodes, uint16_t* scales, uint8_t* zeros, uint16_t* w_weak, void* stream)
{
    if (!W || !scales || !zeros || (!qcodes && k < K))
        return fail(OWQ_ERR_NULL, "W, scales, zeros and (unless k == K) qcodes must be non-NULL");
    if (N < 1 || N > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)N);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && (!weak_idx || !w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(W, 16) || !aligned(qcodes, 4) || !aligned(scales, 2) ||
        (k > 0 && (!aligned(weak_idx, 4) || !aligned(w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W: 16 B, qcodes/weak_idx: 4 B, fp16: 2 B)");
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_pack_storage(W, N, K, k > 0 ? weak_idx : nullptr, k, qcodes, scales, zeros,
                                               k > 0 ? w_weak : nullptr, (hipStream_t)stream),
                      "owq_pack_storage launch");
}

size_t owq_linear_storage_workspace_bytes(int64_t K, int32_t k, int64_t M)
{
    if (K < 32 || K > kMaxK || K % 32 != 0 || k < 0 || k > K || M < 1 || M > INT32_MAX)
        return 0;
    return owq::storage_workspace_bytes(K, k, M);
}

owq_status owq_linear_storage(const owq_layer* L, const uint16_t* x, int64_t M, uint16_t* y, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    if (!L)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    if (L->k == L->K && L->K >= 32 && !L->qcodes) {  // every column weak: no codes are stored
        owq_layer tmp = *L;
        tmp.qcodes = reinterpret_cast<const uint32_t*>(L->scales);
        return owq_linear_storage(&tmp, x, M, y, workspace, workspace_bytes, stream);
    }
    owq_status st = check_layer(L, M, x, y);
    if (st != OWQ_OK)
        return st;
    if (!workspace)
        return fail(OWQ_ERR_NULL, "workspace must be non-NULL");
    if (!aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned workspace (256 B)");
    const size_t need = owq::storage_workspace_bytes(L->K, L->k, M);
    if (workspace_bytes < need)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
    st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_linear_storage(desc_of(L, x, y), M, workspace, (hipStream_t)stream),
                      "owq_linear_storage launch");
}

size_t owq_linear_storage_batched_workspace_bytes(const owq_layer* Ls, int32_t count, int64_t M)
{
    if (!Ls || count < 1 || count > 64)
        return 0;
    size_t total = 0;
    for (int32_t l = 0; l < count; l++) {
        const size_t b = owq_linear_storage_workspace_bytes(Ls[l].K, Ls[l].k, M);
        if (b == 0)
            return 0;
        total += (b + 255) & ~(size_t)255;
    }
    return total;
}

owq_status owq_linear_storage_batched(const owq_layer* Ls, const uint16_t* const* xs, uint16_t* const* ys,
                                      int32_t count, int64_t M, void* workspace, size_t workspace_bytes,
                                      void* stream)
{
    if (!Ls || !xs || !ys)
        return fail(OWQ_ERR_NULL, "Ls, xs and ys must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    if (!workspace)
        return fail(OWQ_ERR_NULL, "workspace must be non-NULL");
    if (!aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned workspace (256 B)");
    std::vector<owq::LinearDesc> d((size_t)count);
    std::vector<void*> ws((size_t)count);
    size_t off = 0;
    for (int32_t l = 0; l < count; l++) {
        owq_layer L = Ls[l];
        if (L.k == L.K && L.K >= 32 && !L.qcodes)  // every column weak: no codes are stored
            L.qcodes = reinterpret_cast<const uint32_t*>(L.scales);
        owq_status st = check_layer(&L, M, xs[l], ys[l]);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        st = check_idx_on_host(L.weak_idx, L.k, L.K, (hipStream_t)stream);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        d[l] = desc_of(&L, xs[l], ys[l]);
        ws[l] = static_cast<char*>(workspace) + off;
        off += (owq::storage_workspace_bytes(L.K, L.k, M) + 255) & ~(size_t)255;
    }
    if (workspace_bytes < off)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, off);
    return hip_status(owq::launch_linear_storage_batched(d.data(), count, M, ws.data(), (hipStream_t)stream),
                      "owq_linear_storage_batched launch");
}

size_t owq_pack_optq_workspace_bytes(int64_t N, int64_t K, int32_t k)
{
    if (N < 1 || N > INT32_MAX || K < 32 || K > kMaxK || K % 32 != 0 || k < 0 || k > K)
        return 0;
    return owq::optq_plan(N, K, k).total;
}

owq_status owq_pack_optq(const uint16_t* W, int64_t N, int64_t K, const uint16_t* X, int64_t T,
                         const int32_t* weak_idx, int32_t k, uint32_t* qcodes, uint16_t* scales, uint8_t* zeros,
                         uint16_t* w_weak, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!W || !X || !qcodes || !scales || !zeros || !workspace)
        return fail(OWQ_ERR_NULL, "W, X, qcodes, scales, zeros and workspace must be non-NULL");
    if (N < 1 || N > INT32_MAX || T < 1 || T > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld, T = %lld out of range", (long long)N, (long long)T);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && (!weak_idx || !w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(W, 16) || !aligned(X, 2) || !aligned(qcodes, 4) || !aligned(scales, 2) ||
        !aligned(workspace, 256) || (k > 0 && (!aligned(weak_idx, 4) || !aligned(w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W: 16 B, workspace: 256 B, qcodes/weak_idx: 4 B, fp16: 2 B)");
    const owq::OptqPlan p = owq::optq_plan(N, K, k);
    if (workspace_bytes < p.total)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, p.total);
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_pack_optq(W, N, K, X, T, k > 0 ? weak_idx : nullptr, k, qcodes, scales, zeros,
                                            k > 0 ? w_weak : nullptr, workspace, p, (hipStream_t)stream),
                      "owq_pack_optq launch");
}

size_t owq_linear_backward_workspace_bytes(int64_t N, int64_t K, int32_t k)
{
    if (N < 1 || N > INT32_MAX || K < 32 || K > kMaxK || K % 32 != 0 || k < 0 || k > K)
        return 0;
    return owq::bwd_plan(N, K, k).total;
}

owq_status owq_linear_backward(const owq_layer* L, const uint16_t* x, const uint16_t* dy, int64_t M, uint16_t* dx,
                               float* dw_weak, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!L || !dy)
        return fail(OWQ_ERR_NULL, "layer and dy must be non-NULL");
    // check_layer wants an x and a y: x is read only for dw_weak, y is not used
    owq_status st = check_layer(L, M, x ? x : dy, dy);
    if (st != OWQ_OK)
        return st;
    if (dw_weak && L->k > 0 && !x)
        return fail(OWQ_ERR_NULL, "x must be non-NULL for dw_weak");
    if ((dx && !aligned(dx, 2)) || (dw_weak && !aligned(dw_weak, 4)) || !aligned(dy, 2))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (dy, dx: 2 B, dw_weak: 4 B)");
    owq::BwdPlan p = owq::bwd_plan(L->N, L->K, L->k);
    if (dx) {
        if (!workspace)
            return fail(OWQ_ERR_NULL, "workspace must be non-NULL when dx is requested");
        if (!aligned(workspace, 256))
            return fail(OWQ_ERR_ALIGN, "misaligned workspace (256 B)");
        if (workspace_bytes < p.total)
            return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, p.total);
    }
    st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    owq::LinearDesc d = desc_of(L, x, nullptr);
    return hip_status(owq::launch_linear_backward(d, dy, M, dx, dw_weak, workspace, p, (hipStream_t)stream),
                      "owq_linear_backward launch");
}

size_t owq_linear_backward_batched_workspace_bytes(const owq_layer* Ls, int32_t count)
{
    if (!Ls || count < 1 || count > 64)
        return 0;
    size_t total = 0;
    for (int32_t l = 0; l < count; l++) {
        const size_t b = owq_linear_backward_workspace_bytes(Ls[l].N, Ls[l].K, Ls[l].k);
        if (b == 0)
            return 0;
        total += (b + 255) & ~(size_t)255;
    }
    return total;
}

owq_status owq_linear_backward_batched(const owq_layer* Ls, const uint16_t* const* xs, const uint16_t* const* dys,
                                       int32_t count, int64_t M, uint16_t* const* dxs, float* const* dws,
                                       void* workspace, size_t workspace_bytes, void* stream)
{
    if (!Ls || !dys)
        return fail(OWQ_ERR_NULL, "Ls and dys must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    std::vector<owq::LinearDesc> d((size_t)count);
    std::vector<owq::BwdPlan> plans((size_t)count);
    std::vector<const uint16_t*> dy((size_t)count);
    std::vector<uint16_t*> dx((size_t)count);
    std::vector<float*> dw((size_t)count);
    std::vector<void*> ws((size_t)count);
    size_t need = 0;
    for (int32_t l = 0; l < count; l++) {
        const owq_layer* L = &Ls[l];
        const uint16_t* x = xs ? xs[l] : nullptr;
        dy[l] = dys[l];
        dx[l] = dxs ? dxs[l] : nullptr;
        dw[l] = dws ? dws[l] : nullptr;
        if (!dy[l])
            return fail(OWQ_ERR_NULL, "layer %d: dy must be non-NULL", l);
        owq_status st = check_layer(L, M, x ? x : dy[l], dy[l]);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        if (dw[l] && L->k > 0 && !x)
            return fail(OWQ_ERR_NULL, "layer %d: x must be non-NULL for dw_weak", l);
        if ((dx[l] && !aligned(dx[l], 2)) || (dw[l] && !aligned(dw[l], 4)) || !aligned(dy[l], 2))
            return fail(OWQ_ERR_ALIGN, "layer %d: misaligned pointer (dy, dx: 2 B, dw_weak: 4 B)", l);
        st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
        if (st != OWQ_OK)
            return st;
        d[l] = desc_of(L, x, nullptr);
        plans[l] = owq::bwd_plan(L->N, L->K, L->k);
        ws[l] = nullptr;
        if (dx[l]) {
            ws[l] = reinterpret_cast<void*>(need);  // offset for now
            need += (plans[l].total + 255) & ~(size_t)255;
        }
    }
    if (need > 0) {
        if (!workspace)
            return fail(OWQ_ERR_NULL, "workspace must be non-NULL when dx is requested");
        if (!aligned(workspace, 256))
            return fail(OWQ_ERR_ALIGN, "misaligned workspace (256 B)");
        if (workspace_bytes < need)
            return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
        for (int32_t l = 0; l < count; l++)
            if (dx[l])
                ws[l] = static_cast<char*>(workspace) + reinterpret_cast<size_t>(ws[l]);
    }
    hipError_t e = hipSuccess;
    for (int32_t l0 = 0; l0 < count && e == hipSuccess; l0 += owq::kBwdMaxLayers) {
        const int n = count - l0 < owq::kBwdMaxLayers ? count - l0 : owq::kBwdMaxLayers;
        e = owq::launch_linear_backward_batched(d.data() + l0, dy.data() + l0, n, M, dx.data() + l0, dw.data() + l0,
                                                ws.data() + l0, plans.data() + l0, (hipStream_t)stream);
    }
    return hip_status(e, "owq_linear_backward_batched launch");
}

owq_status owq_pack_grouped(const uint16_t* W, int64_t N, int64_t K, const int32_t* weak_idx, int32_t k,
                            int64_t G, uint32_t* qcodes, uint16_t* scales, uint8_t* zeros, uint16_t* w_weak,
                            void* stream)
{
    if (!W || !qcodes || !scales || !zeros)
        return fail(OWQ_ERR_NULL, "W, qcodes, scales and zeros must be non-NULL");
    if (N < 1 || N > INT32_MAX)
        return fail(OWQ_ERR_SHAPE, "N = %lld out of range", (long long)N);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (!owq::grouped_size_supported(G, K))
        return fail(OWQ_ERR_UNSUPPORTED, "G = %lld: need a power of two in [32, 2048] dividing K = %lld",
                    (long long)G, (long long)K);
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (k > 0 && (!weak_idx || !w_weak))
        return fail(OWQ_ERR_NULL, "weak_idx and w_weak must be non-NULL when k > 0");
    if (!aligned(W, 16) || !aligned(qcodes, 4) || !aligned(scales, 2) ||
        (k > 0 && (!aligned(weak_idx, 4) || !aligned(w_weak, 2))))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W: 16 B, qcodes/weak_idx: 4 B, fp16: 2 B)");
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_pack_grouped(W, N, K, k > 0 ? weak_idx : nullptr, k, G, qcodes, scales, zeros,
                                               k > 0 ? w_weak : nullptr, (hipStream_t)stream),
                      "owq_pack_grouped launch");
}

owq_status owq_linear_grouped(const owq_grouped_layer* L, const uint16_t* x, int64_t M, uint16_t* y, void* stream)
{
    if (!L)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    owq_layer base{L->N, L->K, L->k, L->bits, L->qcodes, L->scales, L->zeros, L->weak_idx, L->w_weak};
    owq_status st = check_layer(&base, M, x, y);
    if (st != OWQ_OK)
        return st;
    if (!owq::grouped_size_supported(L->G, L->K))
        return fail(OWQ_ERR_UNSUPPORTED, "G = %lld: need a power of two in [32, 2048] dividing K = %lld",
                    (long long)L->G, (long long)L->K);
    st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    const owq::LinearDesc d = desc_of(&base, x, y);
    hipError_t e = hipSuccess;
    for (int64_t m0 = 0; m0 < M && e == hipSuccess; m0 += owq::kGemvMaxM) {  // token slices
        const int64_t mm = M - m0 < owq::kGemvMaxM ? M - m0 : owq::kGemvMaxM;
        owq::LinearDesc dm = d;
        dm.x = d.x + m0 * d.K;
        dm.y = d.y + m0 * d.N;
        e = owq::launch_gemv_grouped(&dm, &L->G, 1, (int)mm, (hipStream_t)stream);
    }
    return hip_status(e, "owq_linear_grouped launch");
}

owq_status owq_linear_grouped_batched(const owq_grouped_layer* Ls, const uint16_t* const* xs, uint16_t* const* ys,
                                      int32_t count, int64_t M, void* stream)
{
    if (!Ls || !xs || !ys)
        return fail(OWQ_ERR_NULL, "Ls, xs and ys must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    if (M < 1 || M > owq::kGemvMaxM)
        return fail(OWQ_ERR_UNSUPPORTED, "M = %lld: the batched group-wise launch needs 1 <= M <= %d",
                    (long long)M, owq::kGemvMaxM);
    std::vector<owq::LinearDesc> d((size_t)count);
    std::vector<int64_t> groups((size_t)count);
    for (int32_t l = 0; l < count; l++) {
        const owq_grouped_layer& g = Ls[l];
        owq_layer base{g.N, g.K, g.k, g.bits, g.qcodes, g.scales, g.zeros, g.weak_idx, g.w_weak};
        owq_status st = check_layer(&base, M, xs[l], ys[l]);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        if (!owq::grouped_size_supported(g.G, g.K))
            return fail(OWQ_ERR_UNSUPPORTED, "layer %d: G = %lld: need a power of two in [32, 2048] dividing K = %lld",
                        l, (long long)g.G, (long long)g.K);
        st = check_idx_on_host(g.weak_idx, g.k, g.K, (hipStream_t)stream);
        if (st != OWQ_OK)
            return st;
        d[l] = desc_of(&base, xs[l], ys[l]);
        groups[l] = g.G;
    }
    hipError_t e = hipSuccess;
    for (int32_t l0 = 0; l0 < count && e == hipSuccess; l0 += owq::kGemvMaxLayers) {
        const int n = count - l0 < owq::kGemvMaxLayers ? count - l0 : owq::kGemvMaxLayers;
        e = owq::launch_gemv_grouped(d.data() + l0, groups.data() + l0, n, (int)M, (hipStream_t)stream);
    }
    return hip_status(e, "owq_linear_grouped_batched launch");
}

owq_status owq_linear(const owq_layer* L, const uint16_t* x, int64_t M, uint16_t* y, void* stream)
{
    owq_status st = check_layer(L, M, x, y);
    if (st != OWQ_OK)
        return st;
    st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return hip_status(owq::launch_linear_any(desc_of(L, x, y), M, (hipStream_t)stream), "owq_linear launch");
}

owq_status owq_linear_batched(const owq_layer* Ls, const uint16_t* const* xs, uint16_t* const* ys,
                              int32_t count, int64_t M, void* stream)
{
    if (!Ls || !xs || !ys)
        return fail(OWQ_ERR_NULL, "Ls, xs and ys must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    if (M < 1 || M > owq::kMfvMaxM)
        return fail(OWQ_ERR_UNSUPPORTED, "M = %lld: the batched decode launch needs 1 <= M <= %d",
                    (long long)M, owq::kMfvMaxM);
    const bool mat = owq::decode_on_matrix_cores(M);
    std::vector<owq::LinearDesc> d((size_t)count);
    for (int32_t l = 0; l < count; l++) {
        owq_status st = check_layer(&Ls[l], M, xs[l], ys[l]);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        st = check_idx_on_host(Ls[l].weak_idx, Ls[l].k, Ls[l].K, (hipStream_t)stream);
        if (st != OWQ_OK)
            return st;
        if (mat ? !owq::mfv_fits(M, Ls[l].K) : !owq::gemv_fits(M, Ls[l].K))
            return fail(OWQ_ERR_UNSUPPORTED, "layer %d: M = %lld, K = %lld outside the batched decode limits", l,
                        (long long)M, (long long)Ls[l].K);
        d[l] = desc_of(&Ls[l], xs[l], ys[l]);
    }
    hipError_t e = hipSuccess;
    for (int32_t l0 = 0; l0 < count && e == hipSuccess; l0 += owq::kGemvMaxLayers) {
        int n = count - l0 < owq::kGemvMaxLayers ? count - l0 : owq::kGemvMaxLayers;
        e = mat ? owq::launch_mfv(d.data() + l0, n, (int)M, (hipStream_t)stream)
                : owq::launch_gemv(d.data() + l0, n, (int)M, (hipStream_t)stream);
    }
    return hip_status(e, "owq_linear_batched launch");
}

owq_status owq_gated(const owq_layer* gate, const owq_layer* up, const uint16_t* x, int64_t M, int32_t act,
                     uint16_t* h, float* g, float* u, void* stream)
{
    owq_status st = check_gated(gate, up, M, x, h, act, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    if (!g != !u)
        return fail(OWQ_ERR_NULL, "g and u must be given together");
    if (!aligned(g, 4) || !aligned(u, 4))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (g, u: 4 B)");
    const uint64_t n = (uint64_t)M * (uint64_t)gate->N;
    const Span in{"x", x, 2 * (uint64_t)M * (uint64_t)gate->K};
    const Span outs[3] = {{"h", h, 2 * n}, {"g", g, 4 * n}, {"u", u, 4 * n}};
    for (int i = 0; i < 3; i++) {
        st = check_apart(outs[i], {in, outs[(i + 1) % 3]});
        for (const owq_layer* L : {gate, up})
            st = st != OWQ_OK ? st : check_apart(outs[i], L);
        if (st != OWQ_OK)
            return st;
    }
    return launch_status(owq::launch_gated(desc_of(gate, x, nullptr), desc_of(up, x, nullptr), M, act, h, g, u,
                                           (hipStream_t)stream),
                         "owq_gated launch");
}

size_t owq_gated_backward_workspace_bytes(int64_t N, int64_t K, int32_t k_gate, int32_t k_up, int64_t M)
{
    if (N < 1 || N > owq::kGatedBwdMax || M < 1 || M > owq::kGatedBwdMax || K < 32 || K > kMaxK || K % 32 != 0 ||
        k_gate < 0 || k_gate > K || k_up < 0 || k_up > K)
        return 0;
    return owq::gated_bwd_workspace_bytes(N, K, k_gate, k_up, M);
}

owq_status owq_gated_backward(const owq_layer* gate, const owq_layer* up, const uint16_t* x, const float* g,
                              const float* u, const uint16_t* dh, int64_t M, int32_t act, uint16_t* dx,
                              float* dw_gate, float* dw_up, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!gate || !up)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    const bool need_x = (dw_gate && gate->k > 0) || (dw_up && up->k > 0);
    if (!g || !u || !dh || !workspace || (need_x && !x))
        return fail(OWQ_ERR_NULL, "g, u, dh and workspace (and x for the weak gradients) must be non-NULL");
    // check_layer wants an x and an output: x is checked below when it is read
    owq_status st = check_gated(gate, up, M, reinterpret_cast<const uint16_t*>(workspace), dh, act,
                                (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    if (M > owq::kGatedBwdMax || gate->N > owq::kGatedBwdMax)
        return fail(OWQ_ERR_SHAPE, "M = %lld, N = %lld: need at most 2^20", (long long)M, (long long)gate->N);
    if (!aligned(g, 4) || !aligned(u, 4) || !aligned(dh, 2) || !aligned(dx, 2) || !aligned(dw_gate, 4) ||
        !aligned(dw_up, 4) || (need_x && !aligned(x, 16)) || !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (x: 16 B, g, u, dw: 4 B, dh, dx: 2 B, workspace: 256 B)");
    const size_t need = owq::gated_bwd_workspace_bytes(gate->N, gate->K, gate->k, up->k, M);
    if (workspace_bytes < need)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
    if (!dx && !need_x) {  // nothing to compute
        g_err[0] = '\0';
        return OWQ_OK;
    }
    // dx is written after x, g, u and dh have been read; everything else stays apart
    const uint64_t n = (uint64_t)M * (uint64_t)gate->N, mk = 2 * (uint64_t)M * (uint64_t)gate->K;
    const Span sx{"x", need_x ? x : nullptr, mk}, sg{"g", g, 4 * n}, su{"u", u, 4 * n}, sh{"dh", dh, 2 * n};
    const Span sdx{"dx", dx, mk}, ws{"workspace", workspace, need};
    const Span dwg{"dw_gate", dw_gate, 4 * (uint64_t)gate->N * (uint64_t)gate->k};
    const Span dwu{"dw_up", dw_up, 4 * (uint64_t)up->N * (uint64_t)up->k};
    st = check_apart(sdx, {dwg, dwu, ws});
    st = st != OWQ_OK ? st : check_apart(dwg, {sx, sg, su, sh, dwu, ws});
    st = st != OWQ_OK ? st : check_apart(dwu, {sx, sg, su, sh, ws});
    st = st != OWQ_OK ? st : check_apart(ws, {sx, sg, su, sh});
    for (const Span* out : {&sdx, &dwg, &dwu, &ws})
        for (const owq_layer* L : {gate, up})
            st = st != OWQ_OK ? st : check_apart(*out, L);
    if (st != OWQ_OK)
        return st;
    return launch_status(owq::launch_gated_backward(desc_of(gate, x, nullptr), desc_of(up, x, nullptr), M, act, g, u,
                                                    dh, dx, dw_gate, dw_up, workspace, (hipStream_t)stream),
                         "owq_gated_backward launch");
}

size_t owq_linear_adapters_workspace_bytes(int32_t rank, int64_t M)
{
    if (rank < 1 || rank > kMaxRank || M < 1 || M > kMaxBlock || !owq::adapter_shrink_grid_fits(rank, M))
        return 0;
    return owq::adapter_workspace_bytes(rank, M);
}

owq_status owq_linear_adapters(const owq_layer* L, const owq_adapters* ad, const int32_t* which, const uint16_t* x,
                               int64_t M, uint16_t* y, void* workspace, size_t workspace_bytes, void* stream)
{
    owq_status st = check_layer(L, M, x, y);
    if (st != OWQ_OK)
        return st;
    if (M > kMaxBlock || L->N > kMaxBlock)
        return fail(OWQ_ERR_SHAPE, "M = %lld, N = %lld: need at most 2^30", (long long)M, (long long)L->N);
    if (!ad || !ad->A || !ad->B || !ad->alpha || !which || !workspace)
        return fail(OWQ_ERR_NULL, "adapters (A, B, alpha), which and workspace must be non-NULL");
    if (ad->rank < 1 || ad->rank > kMaxRank)
        return fail(OWQ_ERR_SHAPE, "rank = %d: need 1 <= rank <= %d", ad->rank, kMaxRank);
    if (ad->count < 1)
        return fail(OWQ_ERR_SHAPE, "count = %d: need at least one adapter", ad->count);
    const bool gemm = M > owq::kMfvMaxM, mat = !gemm && owq::decode_on_matrix_cores(M);
    if (!owq::adapter_shrink_grid_fits(ad->rank, M) ||
        !(gemm ? owq::adapter_gemm_grid_fits(M, L->N) : mat ? owq::mfv_grid_fits(M, L->N) : owq::gemv_grid_fits(L->N)))
        return launch_status(hipErrorInvalidConfiguration, "owq_linear_adapters launch");
    if (!aligned(ad->A, 16) || !aligned(ad->B, 16) || !aligned(ad->alpha, 4) || !aligned(which, 4) ||
        !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (A, B: 16 B, alpha, which: 4 B, workspace: 256 B)");
    if (workspace_bytes < owq::adapter_workspace_bytes(ad->rank, M))
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes,
                    owq::adapter_workspace_bytes(ad->rank, M));
    const uint64_t K = (uint64_t)L->K, N = (uint64_t)L->N, ranks = (uint64_t)ad->count * (uint64_t)ad->rank;
    const Span sy{"y", y, 2 * (uint64_t)M * N}, ws{"workspace", workspace, owq::adapter_workspace_bytes(ad->rank, M)};
    for (const Span* out : {&sy, &ws}) {
        st = check_apart(*out, {{"x", x, 2 * (uint64_t)M * K},
                                {"A", ad->A, 2 * ranks * K},
                                {"B", ad->B, 2 * ranks * N},
                                {"alpha", ad->alpha, 4 * (uint64_t)ad->count},
                                {"which", which, 4 * (uint64_t)M},
                                out == &sy ? ws : sy});
        st = st != OWQ_OK ? st : check_apart(*out, L);
        if (st != OWQ_OK)
            return st;
    }
    st = check_idx_on_host(L->weak_idx, L->k, L->K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    float* const t = static_cast<float*>(workspace);
    int32_t* const order = reinterpret_cast<int32_t*>(t + M * owq::adapter_rpad(ad->rank));
    const owq::AdapterDesc a{ad->A, ad->B, ad->alpha, which, t, order, ad->count, ad->rank};
    hipError_t e = owq::launch_adapter_shrink(a, x, M, L->K, (hipStream_t)stream);
    if (e == hipSuccess)
    {
        const owq::LinearDesc d = desc_of(L, x, y);
        if (gemm)
            e = owq::launch_adapter_gemm(d, a, M, (hipStream_t)stream);
        else if (mat)
            e = owq::launch_mfv(&d, 1, (int)M, (hipStream_t)stream, &a);
        else
            e = owq::launch_gemv(&d, 1, (int)M, (hipStream_t)stream, &a);
    }
    return launch_status(e, "owq_linear_adapters launch");
}

size_t owq_clip_grad_norm_workspace_bytes(int32_t count)
{
    if (count < 1 || count > kMaxGrads)
        return 0;
    return owq::clip_workspace_bytes(count);
}

owq_status owq_clip_grad_norm(const owq_grad* items, int32_t count, double max_norm, float* norm, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    if (!items || !norm || !workspace)
        return fail(OWQ_ERR_NULL, "items, norm and workspace must be non-NULL");
    if (count < 1 || count > kMaxGrads)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= %d", count, kMaxGrads);
    if (!(max_norm >= 0.0))
        return fail(OWQ_ERR_RANGE, "max_norm = %g: need max_norm >= 0", max_norm);
    if (!aligned(norm, 4) || !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (norm: 4 B, workspace: 256 B)");
    if (workspace_bytes < owq::clip_workspace_bytes(count))
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes,
                    owq::clip_workspace_bytes(count));
    owq_status st = OWQ_OK;
    try {
        std::vector<owq::ClipEntry> it((size_t)count);
        std::vector<InOut> list;
        list.reserve((size_t)count);
        for (int32_t i = 0; i < count; i++) {
            const owq_grad& g = items[i];
            if (g.n < 0 || g.n > (int64_t)1 << 40)
                return fail(OWQ_ERR_SHAPE, "item %d: n = %lld: need 0 <= n <= 2^40", i, (long long)g.n);
            if (g.type != 0 && g.type != 1)
                return fail(OWQ_ERR_UNSUPPORTED, "item %d: type = %d: need 0 (fp32) or 1 (fp16)", i, g.type);
            if (g.n > 0 && (!g.g || !g.out))
                return fail(OWQ_ERR_NULL, "item %d: g and out must be non-NULL when n > 0", i);
            const size_t size = g.type ? 2 : 4;
            if (g.n > 0 && (!aligned(g.g, size) || !aligned(g.out, size)))
                return fail(OWQ_ERR_ALIGN, "item %d: misaligned pointer (%zu B)", i, size);
            it[(size_t)i] = owq::ClipEntry{g.g, g.out, g.n, g.type};
            list.push_back(InOut{g.g, g.out, (uint64_t)g.n * size});
        }
        st = check_list_apart(list);
        if (st != OWQ_OK)
            return st;
        const Span sn{"norm", norm, 4}, ws{"workspace", workspace, owq::clip_workspace_bytes(count)};
        st = check_apart(sn, {ws});
        for (int32_t i = 0; i < count && st == OWQ_OK; i++) {
            const owq_grad& g = items[i];
            const uint64_t bytes = (uint64_t)g.n * (g.type ? 2 : 4);
            for (const Span* s : {&sn, &ws})
                st = st != OWQ_OK ? st : check_apart(*s, {{"a gradient", g.g, bytes}, {"an output", g.out, bytes}});
            if (st != OWQ_OK)
                return fail_at(st, "item", i);
        }
        if (st != OWQ_OK)
            return st;
        return launch_status(owq::launch_clip(it.data(), count, max_norm, norm, workspace, (hipStream_t)stream),
                             "owq_clip_grad_norm launch");
    } catch (const std::exception& ex) {
        return fail(OWQ_ERR_HIP, "owq_clip_grad_norm: host memory: %s", ex.what());
    }
}

// ---------------------------------------------------------------- integer form --

owq_status owq_pack_integer(const uint16_t* W, int64_t N, int64_t K, const int32_t* weak_idx, int32_t k, int8_t* codes,
                         float* scales, uint16_t* w_weak, void* stream)
{
    if (N < 1 || !owq::grid_fits(N, 256))
        return fail(OWQ_ERR_SHAPE, "N = %lld: need 1 <= N < 2^24", (long long)N);
    owq_status st = check_k_dim(K);
    if (st != OWQ_OK)
        return st;
    if (k < 0 || k > K)
        return fail(OWQ_ERR_RANGE, "k = %d outside [0, K = %lld]", k, (long long)K);
    if (!W || !codes || !scales || (k > 0 && (!weak_idx || !w_weak)))
        return fail(OWQ_ERR_NULL, "W, codes and scales (and weak_idx, w_weak when k > 0) must be non-NULL");
    if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(weak_idx, 4) || !aligned(w_weak, 2))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (W, codes: 16 B, scales, weak_idx: 4 B, w_weak: 2 B)");
    const uint64_t n = (uint64_t)N, nk = n * (uint64_t)K;
    const Span outs[3] = {{"codes", codes, nk}, {"scales", scales, 4 * n}, {"w_weak", w_weak, 2 * n * (uint64_t)k}};
    for (int i = 0; i < 3; i++) {
        st = check_apart(outs[i], {{"W", W, 2 * nk}, {"weak_idx", weak_idx, 4 * (uint64_t)k}, outs[(i + 1) % 3]});
        if (st != OWQ_OK)
            return st;
    }
    st = check_idx_on_host(weak_idx, k, K, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    return launch_status(owq::launch_pack_int8(W, N, K, weak_idx, k, codes, scales, w_weak, (hipStream_t)stream),
                         "owq_pack_integer launch");
}

size_t owq_linear_integer_workspace_bytes(int64_t N, int64_t K, int32_t k, int64_t M)
{
    if (!int8_sizes_ok(N, K, k, M))
        return 0;
    return owq::int8_plan(N, K, k, M).total;
}

size_t owq_linear_integer_batched_workspace_bytes(const owq_integer_layer* Ls, int32_t count, int64_t M)
{
    if (!Ls || count < 1 || count > 64 || M < 1 || M > owq::kInt8BatchMaxM)
        return 0;
    size_t total = 0;
    for (int32_t l = 0; l < count; l++) {
        if (!int8_sizes_ok(Ls[l].N, Ls[l].K, Ls[l].k, M))
            return 0;
        total += owq::int8_plan(Ls[l].N, Ls[l].K, Ls[l].k, M).total;
    }
    return total;
}

owq_status owq_linear_integer(const owq_integer_layer* L, const uint16_t* x, int64_t M, uint16_t* y, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    owq_status st = check_int8_layer(L, M, x, y, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    const size_t need = owq::int8_plan(L->N, L->K, L->k, M).total;
    st = check_int8_spans(L, x, M, y, workspace, need, workspace_bytes);
    if (st != OWQ_OK)
        return st;
    const owq::Int8Desc d = int8_desc(L, x, y);
    return launch_status(owq::launch_linear_int8(&d, 1, M, &workspace, (hipStream_t)stream), "owq_linear_integer launch");
}

owq_status owq_linear_integer_batched(const owq_integer_layer* Ls, const uint16_t* const* xs, uint16_t* const* ys,
                                   int32_t count, int64_t M, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!Ls || !xs || !ys)
        return fail(OWQ_ERR_NULL, "Ls, xs and ys must be non-NULL");
    if (count < 1 || count > 64)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= 64", count);
    if (M < 1 || M > owq::kInt8BatchMaxM)
        return fail(OWQ_ERR_UNSUPPORTED, "M = %lld: the batched launch needs 1 <= M <= %d", (long long)M,
                    owq::kInt8BatchMaxM);
    owq::Int8Desc d[64];
    void* ws[64];
    size_t need = 0;
    for (int32_t l = 0; l < count; l++) {
        owq_status st = check_int8_layer(&Ls[l], M, xs[l], ys[l], (hipStream_t)stream);
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
        ws[l] = static_cast<char*>(workspace) + need;
        need += owq::int8_plan(Ls[l].N, Ls[l].K, Ls[l].k, M).total;
        d[l] = int8_desc(&Ls[l], xs[l], ys[l]);
    }
    for (int32_t l = 0; l < count; l++) {
        owq_status st = check_int8_spans(&Ls[l], xs[l], M, ys[l], workspace, need, workspace_bytes);
        // an output also stays apart from the other layers, their inputs and outputs
        const Span out{"y", ys[l], 2 * (uint64_t)M * (uint64_t)Ls[l].N};
        for (int32_t o = 0; o < count && st == OWQ_OK; o++) {
            if (o == l)
                continue;
            st = check_apart(out, {{"another x", xs[o], 2 * (uint64_t)M * (uint64_t)Ls[o].K},
                                   {"another y", ys[o], 2 * (uint64_t)M * (uint64_t)Ls[o].N}});
            st = st != OWQ_OK ? st : check_apart(out, &Ls[o]);
        }
        if (st != OWQ_OK)
            return fail_at(st, "layer", l);
    }
    // the layers of a launch share its grid: every launch is checked before the first
    for (int32_t l0 = 0; l0 < count; l0 += owq::kInt8MaxLayers) {
        int64_t rows = 0;
        for (int32_t l = l0; l < count && l < l0 + owq::kInt8MaxLayers; l++)
            rows += (Ls[l].N + 15) / 16 * 16;
        if (!owq::int8_grid_fits(M, rows, Ls[l0].K))
            return launch_status(hipErrorInvalidConfiguration, "owq_linear_integer_batched launch");
    }
    hipError_t e = hipSuccess;
    for (int32_t l0 = 0; l0 < count && e == hipSuccess; l0 += owq::kInt8MaxLayers) {
        const int n = count - l0 < owq::kInt8MaxLayers ? count - l0 : owq::kInt8MaxLayers;
        e = owq::launch_linear_int8(d + l0, n, M, ws + l0, (hipStream_t)stream);
    }
    return launch_status(e, "owq_linear_integer_batched launch");
}

size_t owq_linear_integer_backward_workspace_bytes(int64_t N, int64_t K, int32_t k, int64_t M)
{
    if (!int8_sizes_ok(N, K, k, M) || N > owq::kInt8BwdMax || M > owq::kInt8BwdMax)
        return 0;
    return owq::int8_bwd_plan(N, K, k, M).total;
}

owq_status owq_linear_integer_backward(const owq_integer_layer* L, const uint16_t* x, const uint16_t* dy, int64_t M,
                                    uint16_t* dx, float* dw_weak, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!L)
        return fail(OWQ_ERR_NULL, "layer is NULL");
    const bool need_x = dw_weak && L->k > 0;
    if (!dy || !workspace || (need_x && !x))
        return fail(OWQ_ERR_NULL, "dy and workspace (and x for the weak gradient) must be non-NULL");
    // check_int8_layer wants an x and an output: x is checked below when it is read
    owq_status st = check_int8_layer(L, M, static_cast<const uint16_t*>(workspace), dy, (hipStream_t)stream);
    if (st != OWQ_OK)
        return st;
    if (M > owq::kInt8BwdMax || L->N > owq::kInt8BwdMax)
        return fail(OWQ_ERR_SHAPE, "M = %lld, N = %lld: need at most 2^20", (long long)M, (long long)L->N);
    if (!aligned(dx, 2) || !aligned(dw_weak, 4) || (need_x && !aligned(x, 16)) || !aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (x: 16 B, dw_weak: 4 B, dy, dx: 2 B, workspace: 256 B)");
    const owq::Int8BwdPlan p = owq::int8_bwd_plan(L->N, L->K, L->k, M);
    if (workspace_bytes < p.total)
        return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, p.total);
    if (!dx && !need_x) {  // nothing to compute
        g_err[0] = '\0';
        return OWQ_OK;
    }
    const uint64_t m = (uint64_t)M, N = (uint64_t)L->N, K = (uint64_t)L->K;
    const Span sx{"x", need_x ? x : nullptr, 2 * m * K}, sdy{"dy", dy, 2 * m * N}, sdx{"dx", dx, 2 * m * K};
    const Span sdw{"dw_weak", dw_weak, 4 * N * (uint64_t)L->k}, ws{"workspace", workspace, p.total};
    st = check_apart(sdx, {sx, sdy, sdw, ws});
    st = st != OWQ_OK ? st : check_apart(sdw, {sx, sdy, ws});
    st = st != OWQ_OK ? st : check_apart(ws, {sx, sdy});
    for (const Span* out : {&sdx, &sdw, &ws})
        st = st != OWQ_OK ? st : check_apart(*out, L);
    if (st != OWQ_OK)
        return st;
    return launch_status(owq::launch_linear_int8_backward(int8_desc(L, x, nullptr), dy, M, dx, need_x ? dw_weak : nullptr,
                                                          workspace, p, (hipStream_t)stream),
                         "owq_linear_integer_backward launch");
}

// ------------------------------------------------------- orthogonalised update --

size_t owq_orthogonalize_workspace_bytes(const owq_update* items, int32_t count)
{
    if (!items || count < 1 || count > kMaxGrads)
        return 0;
    try {
        std::vector<owq::OrthoEntry> it((size_t)count);
        for (int32_t i = 0; i < count; i++) {
            if (items[i].rows < 0 || items[i].cols < 0 || !owq::orthogonalize_fits(items[i].rows, items[i].cols))
                return 0;
            it[(size_t)i].rows = items[i].rows;
            it[(size_t)i].cols = items[i].cols;
        }
        return owq::orthogonalize_workspace_bytes(it.data(), count);
    } catch (const std::exception&) {
        return 0;
    }
}

owq_status owq_orthogonalize(const owq_update* items, int32_t count, int32_t steps, const double* coefficients,
                             double eps, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!items || !coefficients || !workspace)
        return fail(OWQ_ERR_NULL, "items, coefficients and workspace must be non-NULL");
    if (count < 1 || count > kMaxGrads)
        return fail(OWQ_ERR_UNSUPPORTED, "count = %d: need 1 <= count <= %d", count, kMaxGrads);
    if (steps < 1 || steps > kMaxNsSteps)
        return fail(OWQ_ERR_RANGE, "steps = %d: need 1 <= steps <= %d", steps, kMaxNsSteps);
    for (int i = 0; i < 3; i++)
        if (!std::isfinite(coefficients[i]))
            return fail(OWQ_ERR_RANGE, "coefficient %d is not finite", i);
    if (!(eps > 0.0) || !std::isfinite(eps))
        return fail(OWQ_ERR_RANGE, "eps = %g: need a finite eps > 0", eps);
    if (!aligned(workspace, 256))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (workspace: 256 B)");
    try {
        std::vector<owq::OrthoEntry> it((size_t)count);
        std::vector<InOut> list;
        list.reserve((size_t)count);
        for (int32_t i = 0; i < count; i++) {
            const owq_update& u = items[i];
            if (u.rows < 0 || u.cols < 0 || !owq::orthogonalize_fits(u.rows, u.cols))
                return fail(OWQ_ERR_SHAPE, "item %d: %lld x %lld: need at most 2^20 and, for the shorter side, %lld", i,
                            (long long)u.rows, (long long)u.cols, (long long)owq::kOrthoMaxShort);
            if (u.type != 0 && u.type != 1)
                return fail(OWQ_ERR_UNSUPPORTED, "item %d: type = %d: need 0 (fp32) or 1 (fp16)", i, u.type);
            if (!std::isfinite(u.scale))
                return fail(OWQ_ERR_RANGE, "item %d: the scale is not finite", i);
            const uint64_t n = (uint64_t)u.rows * (uint64_t)u.cols, size = u.type ? 2 : 4;
            if (n > 0 && (!u.g || !u.out))
                return fail(OWQ_ERR_NULL, "item %d: g and out must be non-NULL", i);
            if (n > 0 && (!aligned(u.g, size) || !aligned(u.out, size)))
                return fail(OWQ_ERR_ALIGN, "item %d: misaligned pointer (%d B)", i, (int)size);
            it[(size_t)i] = owq::OrthoEntry{u.g, u.out, u.rows, u.cols, u.scale, u.type};
            list.push_back(InOut{u.g, u.out, n * size});
        }
        const size_t need = owq::orthogonalize_workspace_bytes(it.data(), count);
        if (workspace_bytes < need)
            return fail(OWQ_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
        owq_status st = check_list_apart(list);
        const Span ws{"workspace", workspace, need};
        for (int32_t i = 0; i < count && st == OWQ_OK; i++) {
            const InOut& t = list[(size_t)i];
            st = check_apart(ws, {{"a matrix", t.g, t.bytes}, {"an output", t.out, t.bytes}});
            if (st != OWQ_OK)
                return fail_at(st, "item", i);
        }
        if (st != OWQ_OK)
            return st;
        return launch_status(owq::launch_orthogonalize(it.data(), count, coefficients[0], coefficients[1], coefficients[2],
                                                       eps, steps, workspace, (hipStream_t)stream),
                             "owq_orthogonalize launch");
    } catch (const std::exception& ex) {
        return fail(OWQ_ERR_HIP, "owq_orthogonalize: host memory: %s", ex.what());
    }
}

int64_t owq_stream_read_sink_words(int64_t bytes) { return bytes > 0 ? owq::stream_read_sink_words(bytes) : 0; }

owq_status owq_stream_read(const void* src, int64_t bytes, uint32_t* sink, int64_t sink_words, void* stream)
{
    if (!src || !sink)
        return fail(OWQ_ERR_NULL, "src and sink must be non-NULL");
    if (bytes < 12 || bytes % 12 != 0 || bytes > ((int64_t)1 << 40))
        return fail(OWQ_ERR_SHAPE, "bytes = %lld: need 12 <= bytes <= 2^40 and bytes %% 12 == 0", (long long)bytes);
    if (!aligned(src, 4) || !aligned(sink, 4))
        return fail(OWQ_ERR_ALIGN, "misaligned pointer (src and sink: 4 B)");
    if (sink_words < owq::stream_read_sink_words(bytes))
        return fail(OWQ_ERR_RANGE, "sink_words = %lld: need %lld", (long long)sink_words,
                    (long long)owq::stream_read_sink_words(bytes));
    return hip_status(owq::launch_stream_read(src, bytes, sink, (hipStream_t)stream), "owq_stream_read launch");
}

}  // extern "C"
