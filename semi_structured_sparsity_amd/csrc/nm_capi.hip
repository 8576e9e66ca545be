// C ABI of libnmsparse: argument validation, error reporting and dispatch to
// the kernels.  Nothing is enqueued unless every check passes.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "nm_check.h"

namespace nm {

static thread_local char g_err[512] = "";

nm_status set_error(nm_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return st;
}

nm_status check_launch(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return set_error(NM_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
    return NM_OK;
}

static bool dtype_ok(nm_dtype d) { return d == NM_F32 || d == NM_BF16 || d == NM_I8 || d == NM_I32 || d == NM_FP8; }

static nm_status check_pattern(int N, int M, const char* fn) {
    NM_REQ(M == 4 || M == 8, NM_ERR_PATTERN, "%s: M must be 4 or 8 (got %d)", fn, M);
    NM_REQ(N >= 1 && N < M, NM_ERR_PATTERN, "%s: need 1 <= N < M (got N=%d, M=%d)", fn, N, M);
    return NM_OK;
}

static int64_t idx_words_needed(int64_t K, int N, int M) { return (K / M * N * index_bits(M) + 31) / 32; }

static nm_status check_score_src(const void* W, nm_dtype sdt, int64_t ldsc, const float* H, int64_t ldh,
                                 nm_score_mode mode, int64_t R, int64_t K, const char* fn) {
    NM_REQ(W || R * K == 0, NM_ERR_NULL, "%s: score source is NULL", fn);
    NM_REQ(sdt == NM_F32 || sdt == NM_BF16, NM_ERR_DTYPE, "%s: score source must be f32 or bf16", fn);
    NM_REQ(ldsc >= K, NM_ERR_SHAPE, "%s: score leading dimension %lld < K %lld", fn, (long long)ldsc, (long long)K);
    NM_REQ(mode == NM_SCORE_HESSIAN || mode == NM_SCORE_MAGNITUDE, NM_ERR_SHAPE, "%s: unknown score mode", fn);
    if (mode == NM_SCORE_HESSIAN) {
        NM_REQ(H || R * K == 0, NM_ERR_NULL, "%s: H is NULL in HESSIAN mode", fn);
        NM_REQ(ldh == 0 || ldh >= K, NM_ERR_SHAPE, "%s: ldh must be 0 or >= K", fn);
    }
    return NM_OK;
}

}  // namespace nm

using namespace nm;

extern "C" {

int nm_abi_version(void) { return NM_ABI_VERSION; }

const char* nm_last_error(void) { return g_err; }

size_t nm_colsumsq_workspace(int64_t n, int64_t K) { return (n <= 0 || K <= 0) ? 0 : colsumsq_ws(n, K); }

nm_status nm_hdiag_colsumsq(const void* X, nm_dtype xdt, int64_t n, int64_t K, int64_t ldx, float* H, void* ws,
                            size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_hdiag_colsumsq";
    NM_REQ(n >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    if (K == 0) return NM_OK;
    NM_REQ(H, NM_ERR_NULL, "%s: H is NULL", fn);
    NM_REQ(X || n == 0, NM_ERR_NULL, "%s: X is NULL", fn);
    NM_REQ(xdt == NM_BF16 || xdt == NM_F32, NM_ERR_DTYPE, "%s: X must be bf16 or f32", fn);
    NM_REQ(ldx >= K, NM_ERR_SHAPE, "%s: ldx < K", fn);
    const int64_t vec = 16 / esize(xdt);
    NM_REQ(K % vec == 0 && ldx % vec == 0 && aligned16(X), NM_ERR_ALIGN,
           "%s: X must be 16-byte aligned with K and ldx multiples of %lld", fn, (long long)vec);
    const size_t need = nm_colsumsq_workspace(n, K);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(!overlap(span(H, 1, K, K, 4), span(X, n, K, ldx, esize(xdt))), NM_ERR_ALIAS, "%s: H overlaps X", fn);
    launch_colsumsq(X, xdt, n, K, ldx, H, ws, (hipStream_t)stream);
    return check_launch(fn);
}

size_t nm_hutchinson_workspace(int64_t n, int64_t K, int64_t R, int probes) {
    if (n <= 0 || K <= 0 || R <= 0 || probes <= 0) return 0;
    return hutch_ws(n, K, R, probes);
}

nm_status nm_hdiag_hutchinson(const void* X, int64_t n, int64_t K, int64_t ldx, int64_t R, int probes, uint64_t seed,
                              float* D, int64_t ldd, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_hdiag_hutchinson";
    NM_REQ(n >= 0 && K >= 0 && R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(probes >= 1, NM_ERR_SHAPE, "%s: probes must be >= 1", fn);
    if (R == 0 || K == 0) return NM_OK;
    NM_REQ(X && D, NM_ERR_NULL, "%s: NULL pointer", fn);
    NM_REQ(n >= 1, NM_ERR_SHAPE, "%s: need at least one calibration row", fn);
    NM_REQ(ldx >= K && ldd >= K, NM_ERR_SHAPE, "%s: leading dimension < K", fn);
    NM_REQ(K % 64 == 0 && n % 64 == 0 && ldx % 8 == 0 && aligned16(X), NM_ERR_ALIGN,
           "%s: need K %% 64 == 0, n %% 64 == 0, 16-byte aligned X with ldx %% 8 == 0", fn);
    NM_REQ((int64_t)probes * R < (1LL << 31) && (uint64_t)R * (uint64_t)(K / 64) < (1ull << 40), NM_ERR_SHAPE,
           "%s: too many probe rows", fn);
    const size_t need = hutch_ws(n, K, R, probes);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(!overlap(span(D, R, K, ldd, 4), span(X, n, K, ldx, 2)), NM_ERR_ALIAS, "%s: D overlaps X", fn);
    launch_hutchinson(X, n, K, ldx, R, probes, seed, D, ldd, ws, (hipStream_t)stream);
    return check_launch(fn);
}

size_t nm_hutchinson_score_workspace(int64_t n, int64_t K, int64_t R, int probes) {
    if (n <= 0 || K <= 0 || R <= 0 || probes <= 0) return 0;
    return hutch_score_ws(n, K, R, probes);
}

nm_status nm_hutchinson_score(const void* X, int64_t n, int64_t K, int64_t ldx, int64_t R, int probes, uint64_t seed,
                              const void* W, nm_dtype wdt, int64_t ldw, float eps, float* S, int64_t lds,
                              double* stats, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_hutchinson_score";
    NM_REQ(n >= 0 && K >= 0 && R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(probes >= 1, NM_ERR_SHAPE, "%s: probes must be >= 1", fn);
    NM_REQ(wdt == NM_BF16, NM_ERR_DTYPE, "%s: W must be bf16", fn);
    if (R == 0 || K == 0) return NM_OK;
    NM_REQ(X && W && S, NM_ERR_NULL, "%s: NULL pointer", fn);
    NM_REQ(n >= 1, NM_ERR_SHAPE, "%s: need at least one calibration row", fn);
    NM_REQ(ldx >= K && ldw >= K && lds >= K, NM_ERR_SHAPE, "%s: leading dimension < K", fn);
    NM_REQ(K % 64 == 0 && n % 64 == 0 && ldx % 8 == 0 && aligned16(X), NM_ERR_ALIGN,
           "%s: need K %% 64 == 0, n %% 64 == 0, 16-byte aligned X with ldx %% 8 == 0", fn);
    NM_REQ(((uintptr_t)W & 7u) == 0 && ldw % 4 == 0 && aligned16(S) && lds % 4 == 0 && aligned16(ws), NM_ERR_ALIGN,
           "%s: need 8-byte aligned W (ldw %% 4), 16-byte aligned S (lds %% 4) and workspace", fn);
    // the fused epilogue lives in the dense split ring: its 32-bit offsets must hold
    NM_REQ((int64_t)probes * R < (1LL << 31) && (uint64_t)R * (uint64_t)(K / 64) < (1ull << 40) &&
               (int64_t)probes * R * n * 2 < (1LL << 32) && K * n * 2 < (1LL << 32),
           NM_ERR_SHAPE, "%s: problem too large for the fused kernel (use nm_hdiag_hutchinson + nm_score)", fn);
    const size_t need = hutch_score_ws(n, K, R, probes);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    const Range rs = span(S, R, K, lds, 4), rw = Range{(uintptr_t)ws, (uintptr_t)ws + need};
    const Range rst = span(stats, 1, 2, 2, 8);
    NM_REQ(!overlap(rs, span(X, n, K, ldx, 2)) && !overlap(rs, span(W, R, K, ldw, 2)) && !overlap(rs, rw) &&
               !overlap(rst, rs) && !overlap(rst, rw) && !overlap(rst, span(X, n, K, ldx, 2)) &&
               !overlap(rst, span(W, R, K, ldw, 2)) && !overlap(rw, span(X, n, K, ldx, 2)) &&
               !overlap(rw, span(W, R, K, ldw, 2)),
           NM_ERR_ALIAS, "%s: an output or the workspace overlaps an input", fn);
    return launch_hutchinson_score(X, n, K, ldx, R, probes, seed, (const uint16_t*)W, ldw, eps, S, lds, stats, ws,
                                   (hipStream_t)stream);
}

nm_status nm_score(const void* W, nm_dtype wdt, int64_t R, int64_t K, int64_t ldw, const float* H, int64_t ldh,
                   float eps, nm_score_mode mode, float* S, int64_t lds, nm_stream_t stream) {
    const char* fn = "nm_score";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    if (R * K == 0) return NM_OK;
    nm_status st = check_score_src(W, wdt, ldw, H, ldh, mode, R, K, fn);
    if (st != NM_OK) return st;
    NM_REQ(S, NM_ERR_NULL, "%s: S is NULL", fn);
    NM_REQ(lds >= K, NM_ERR_SHAPE, "%s: lds < K", fn);
    const Range rs = span(S, R, K, lds, 4);
    NM_REQ(!overlap(rs, span(W, R, K, ldw, esize(wdt))), NM_ERR_ALIAS, "%s: S overlaps W", fn);
    if (mode == NM_SCORE_HESSIAN)
        NM_REQ(!overlap(rs, span(H, ldh ? R : 1, K, ldh ? ldh : K, 4)), NM_ERR_ALIAS, "%s: S overlaps H", fn);
    launch_score(W, wdt, R, K, ldw, H, ldh, eps, mode, S, lds, (hipStream_t)stream);
    return check_launch(fn);
}

size_t nm_stats_workspace(int64_t R, int64_t K) { return reduce_ws(R, K); }

nm_status nm_score_stats(const float* S, int64_t R, int64_t K, int64_t lds, double* stats, void* ws, size_t ws_bytes,
                         nm_stream_t stream) {
    const char* fn = "nm_score_stats";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(stats, NM_ERR_NULL, "%s: stats is NULL", fn);
    NM_REQ(S || R * K == 0, NM_ERR_NULL, "%s: S is NULL", fn);
    NM_REQ(lds >= K, NM_ERR_SHAPE, "%s: lds < K", fn);
    const size_t need = reduce_ws(R, K);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(!overlap(span(stats, 1, 2, 2, 8), span(S, R, K, lds, 4)), NM_ERR_ALIAS, "%s: stats overlaps S", fn);
    launch_stats(S, R, K, lds, stats, ws, (hipStream_t)stream);
    return check_launch(fn);
}

size_t nm_gate_workspace(int64_t R, int64_t K, int steps) { return gate_ws(R, K, steps); }

nm_status nm_gate(const float* S, int64_t R, int64_t K, int64_t lds, const double* stats, int N, int M, float T0,
                  float rho, int steps, int m_step, float* m, int64_t ldf, uint8_t* hard_mask, int64_t ldm,
                  double* lmid, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_gate";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    nm_status st = check_pattern(N, M, fn);
    if (st != NM_OK) return st;
    NM_REQ(K % M == 0, NM_ERR_SHAPE, "%s: K %% M != 0", fn);
    NM_REQ(steps >= 1 && steps <= 64, NM_ERR_SHAPE, "%s: steps must be in [1, 64]", fn);
    NM_REQ(!m || (m_step >= 0 && m_step < steps), NM_ERR_SHAPE, "%s: m_step must be in [0, steps)", fn);
    NM_REQ(T0 > 0.f && rho > 0.f, NM_ERR_SHAPE, "%s: T0 and rho must be positive", fn);
    NM_REQ(stats && lmid, NM_ERR_NULL, "%s: stats / lmid is NULL", fn);
    NM_REQ((S && hard_mask) || R * K == 0, NM_ERR_NULL, "%s: NULL pointer", fn);
    NM_REQ(lds >= K && ldm >= (K + 7) / 8 && (!m || ldf >= K), NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    const size_t need = gate_ws(R, K, steps);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    const Range rs = span(S, R, K, lds, 4), rh = span(hard_mask, R, (K + 7) / 8, ldm, 1), rm = span(m, R, K, ldf, 4);
    const Range rl = span(lmid, 1, steps, steps, 8), rw = Range{(uintptr_t)ws, (uintptr_t)ws + need};
    const Range ins[2] = {rs, span(stats, 1, 2, 2, 8)};
    for (const Range& x : ins)
        NM_REQ(!overlap(x, rh) && !overlap(x, rm) && !overlap(x, rl) && !overlap(x, rw), NM_ERR_ALIAS,
               "%s: an output or the workspace overlaps S or stats", fn);
    NM_REQ(!overlap(rh, rm) && !overlap(rh, rl) && !overlap(rm, rl), NM_ERR_ALIAS, "%s: outputs overlap", fn);
    launch_gate(S, R, K, lds, stats, N, M, T0, rho, steps, m ? m_step : -1, m, ldf, hard_mask, ldm, lmid, ws,
                (hipStream_t)stream);
    return check_launch(fn);
}

nm_status nm_mask(const float* S, int64_t R, int64_t K, int64_t lds, int N, int M, uint8_t* mask, int64_t ldm,
                  nm_stream_t stream) {
    const char* fn = "nm_mask";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    nm_status st = check_pattern(N, M, fn);
    if (st != NM_OK) return st;
    NM_REQ(K % M == 0, NM_ERR_SHAPE, "%s: K %% M != 0", fn);
    if (R * K == 0) return NM_OK;
    NM_REQ(S && mask, NM_ERR_NULL, "%s: NULL pointer", fn);
    NM_REQ(lds >= K && ldm >= (K + 7) / 8, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    NM_REQ(!overlap(span(mask, R, (K + 7) / 8, ldm, 1), span(S, R, K, lds, 4)), NM_ERR_ALIAS, "%s: mask overlaps S",
           fn);
    launch_mask(S, R, K, lds, N, M, mask, ldm, (hipStream_t)stream);
    return check_launch(fn);
}

static nm_status check_pack_out(const char* fn, nm_dtype wdt, nm_dtype vdt, int64_t R, int64_t K, int64_t slots,
                                int64_t words, const void* vals, int64_t ldv, const uint32_t* idx, int64_t ldi) {
    NM_REQ(dtype_ok(wdt) && dtype_ok(vdt), NM_ERR_DTYPE, "%s: unknown dtype", fn);
    NM_REQ(vdt == wdt || (wdt == NM_F32 && vdt == NM_BF16), NM_ERR_DTYPE,
           "%s: value dtype must equal the weight dtype (or f32 -> bf16)", fn);
    NM_REQ(vals && idx, NM_ERR_NULL, "%s: vals / idx is NULL", fn);
    NM_REQ(ldv >= slots && ldi >= words, NM_ERR_SHAPE, "%s: ldv/ldi too small (need %lld / %lld)", fn,
           (long long)slots, (long long)words);
    NM_REQ(!overlap(span(vals, R, slots, ldv, esize(vdt)), span(idx, R, words, ldi, 4)), NM_ERR_ALIAS,
           "%s: vals overlaps idx", fn);
    (void)K;
    return NM_OK;
}

// NM_FLAG_VALIDATE: count the mask's groups with more than cap bits (a stream
// synchronisation) and refuse to pack when there are any.
static nm_status validate_mask(const char* fn, unsigned flags, const uint8_t* mask, int64_t ldm, int64_t R, int64_t K,
                               int G, int cap, nm_stream_t stream) {
    if (!(flags & NM_FLAG_VALIDATE)) return NM_OK;
    int64_t bad = 0;
    const nm_status st = count_overfull(mask, ldm, R, K, G, cap, (hipStream_t)stream, &bad);
    if (st != NM_OK) return st;
    NM_REQ(bad == 0, NM_ERR_PATTERN, "%s: %lld groups of %d have more than %d mask bits", fn, (long long)bad, G, cap);
    return NM_OK;
}

nm_status nm_pack(const void* W, nm_dtype wdt, int64_t R, int64_t K, int64_t ldw, const uint8_t* mask, int64_t ldm,
                  int N, int M, nm_dtype vdt, void* vals, int64_t ldv, uint32_t* idx, int64_t ldi, unsigned flags,
                  nm_stream_t stream) {
    const char* fn = "nm_pack";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ((flags & ~NM_FLAG_VALIDATE) == 0, NM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, flags);
    nm_status st = check_pattern(N, M, fn);
    if (st != NM_OK) return st;
    NM_REQ(K % M == 0, NM_ERR_SHAPE, "%s: K %% M != 0", fn);
    if (R * K == 0) return NM_OK;
    NM_REQ(W && mask, NM_ERR_NULL, "%s: W / mask is NULL", fn);
    NM_REQ(ldw >= K && ldm >= (K + 7) / 8, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    const int64_t slots = K / M * N, words = idx_words_needed(K, N, M);
    st = check_pack_out(fn, wdt, vdt, R, K, slots, words, vals, ldv, idx, ldi);
    if (st != NM_OK) return st;
    const Range rv = span(vals, R, slots, ldv, esize(vdt)), ri = span(idx, R, words, ldi, 4);
    const Range rw = span(W, R, K, ldw, esize(wdt)), rm = span(mask, R, (K + 7) / 8, ldm, 1);
    NM_REQ(!overlap(rv, rw) && !overlap(rv, rm) && !overlap(ri, rw) && !overlap(ri, rm), NM_ERR_ALIAS,
           "%s: an output overlaps an input", fn);
    st = validate_mask(fn, flags, mask, ldm, R, K, M, N, stream);
    if (st != NM_OK) return st;
    launch_pack(W, wdt, R, K, ldw, mask, ldm, N, M, vdt, vals, ldv, idx, ldi, (hipStream_t)stream);
    return check_launch(fn);
}

nm_status nm_gate_pack(const float* S, int64_t R, int64_t K, int64_t lds, const double* stats, int N, int M,
                       float T0, float rho, int steps, int m_step, float* m, int64_t ldf, uint8_t* hard_mask,
                       int64_t ldm, double* lmid, const void* W, nm_dtype wdt, int64_t ldw, nm_dtype vdt, void* vals,
                       int64_t ldv, uint32_t* idx, int64_t ldi, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_gate_pack";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    nm_status st = check_pattern(N, M, fn);
    if (st != NM_OK) return st;
    NM_REQ(K % M == 0, NM_ERR_SHAPE, "%s: K %% M != 0", fn);
    NM_REQ(steps >= 1 && steps <= 64, NM_ERR_SHAPE, "%s: steps must be in [1, 64]", fn);
    NM_REQ(!m || (m_step >= 0 && m_step < steps), NM_ERR_SHAPE, "%s: m_step must be in [0, steps)", fn);
    NM_REQ(T0 > 0.f && rho > 0.f, NM_ERR_SHAPE, "%s: T0 and rho must be positive", fn);
    NM_REQ(stats && lmid, NM_ERR_NULL, "%s: stats / lmid is NULL", fn);
    NM_REQ((S && hard_mask && W) || R * K == 0, NM_ERR_NULL, "%s: NULL pointer", fn);
    NM_REQ(lds >= K && ldm >= (K + 7) / 8 && ldw >= K && (!m || ldf >= K), NM_ERR_SHAPE,
           "%s: leading dimension too small", fn);
    const size_t need = gate_ws(R, K, steps);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    const int64_t slots = K / M * N, words = idx_words_needed(K, N, M);
    if (R * K > 0) {
        st = check_pack_out(fn, wdt, vdt, R, K, slots, words, vals, ldv, idx, ldi);
        if (st != NM_OK) return st;
    }
    const Range outs[6] = {span(hard_mask, R, (K + 7) / 8, ldm, 1), span(m, R, K, ldf, 4),
                           span(lmid, 1, steps, steps, 8), span(vals, R, slots, ldv, esize(vdt)),
                           span(idx, R, words, ldi, 4), Range{(uintptr_t)ws, (uintptr_t)ws + need}};
    const Range ins[3] = {span(S, R, K, lds, 4), span(stats, 1, 2, 2, 8), span(W, R, K, ldw, esize(wdt))};
    for (const Range& x : ins)
        for (const Range& y : outs)
            NM_REQ(!overlap(x, y), NM_ERR_ALIAS, "%s: an output or the workspace overlaps an input", fn);
    for (int a = 0; a < 6; ++a)
        for (int b = a + 1; b < 6; ++b) NM_REQ(!overlap(outs[a], outs[b]), NM_ERR_ALIAS, "%s: outputs overlap", fn);
    const int ms = m ? m_step : -1;
    const bool fused = R * K > 0 && wdt == NM_BF16 && vdt == NM_BF16 &&
                       launch_gate_pack(S, R, K, lds, stats, N, M, T0, rho, steps, ms, m, ldf, hard_mask, ldm, lmid,
                                        (const uint16_t*)W, ldw, (uint16_t*)vals, ldv, idx, ldi, ws, (hipStream_t)stream);
    if (!fused) {
        // any other shape: the gate, then the pack of its hard mask on the same stream
        launch_gate(S, R, K, lds, stats, N, M, T0, rho, steps, ms, m, ldf, hard_mask, ldm, lmid, ws, (hipStream_t)stream);
        if (R * K > 0)
            launch_pack(W, wdt, R, K, ldw, hard_mask, ldm, N, M, vdt, vals, ldv, idx, ldi, (hipStream_t)stream);
    }
    return check_launch(fn);
}

nm_status nm_prune_pack(const void* Wsc, nm_dtype sdt, int64_t ldsc, const float* H, int64_t ldh, float eps,
                        nm_score_mode mode, const void* Wv, nm_dtype wdt, int64_t ldwv, int64_t R, int64_t K, int N,
                        int M, uint8_t* mask, int64_t ldm, nm_dtype vdt, void* vals, int64_t ldv, uint32_t* idx,
                        int64_t ldi, nm_stream_t stream) {
    const char* fn = "nm_prune_pack";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    nm_status st = check_pattern(N, M, fn);
    if (st != NM_OK) return st;
    NM_REQ(K % M == 0, NM_ERR_SHAPE, "%s: K %% M != 0", fn);
    if (R * K == 0) return NM_OK;
    st = check_score_src(Wsc, sdt, ldsc, H, ldh, mode, R, K, fn);
    if (st != NM_OK) return st;
    NM_REQ(Wv, NM_ERR_NULL, "%s: Wv is NULL", fn);
    NM_REQ(ldwv >= K, NM_ERR_SHAPE, "%s: ldwv < K", fn);
    NM_REQ(!mask || ldm >= (K + 7) / 8, NM_ERR_SHAPE, "%s: ldm too small", fn);
    const int64_t slots = K / M * N, words = idx_words_needed(K, N, M);
    st = check_pack_out(fn, wdt, vdt, R, K, slots, words, vals, ldv, idx, ldi);
    if (st != NM_OK) return st;
    // the fused 2:4 path reads 16-byte vectors and writes 8-byte value pairs
    if (N == 2 && M == 4 && Wsc == Wv && vdt == NM_BF16) {
        const int64_t vec = 16 / esize(wdt);
        NM_REQ(aligned16(Wv) && ldwv % vec == 0 && ((uintptr_t)vals & 7u) == 0 && ldv % 4 == 0 &&
                   (mode == NM_SCORE_MAGNITUDE || (aligned16(H) && ldh % 4 == 0)),
               NM_ERR_ALIGN, "%s: fused 2:4 path needs 16-byte aligned W (ld %% %lld), H (ldh %% 4) and vals (ldv %% 4)",
               fn, (long long)vec);
    }
    const Range rv = span(vals, R, slots, ldv, esize(vdt)), ri = span(idx, R, words, ldi, 4);
    const Range rm = span(mask, R, (K + 7) / 8, ldm, 1);
    const Range in[3] = {span(Wsc, R, K, ldsc, esize(sdt)), span(Wv, R, K, ldwv, esize(wdt)),
                         mode == NM_SCORE_HESSIAN ? span(H, ldh ? R : 1, K, ldh ? ldh : K, 4) : Range{0, 0}};
    for (const Range& x : in)
        NM_REQ(!overlap(rv, x) && !overlap(ri, x) && !overlap(rm, x), NM_ERR_ALIAS, "%s: an output overlaps an input",
               fn);
    NM_REQ(!overlap(rm, rv) && !overlap(rm, ri), NM_ERR_ALIAS, "%s: mask overlaps vals/idx", fn);
    launch_prune_pack(Wsc, sdt, ldsc, H, ldh, eps, mode, Wv, wdt, ldwv, R, K, N, M, mask, ldm, vdt, vals, ldv, idx, ldi,
                      (hipStream_t)stream);
    return check_launch(fn);
}

static nm_status slide_common(const char* fn, bool select, const void* Wsc, nm_dtype sdt, int64_t ldsc, const float* H,
                              int64_t ldh, float eps, nm_score_mode mode, const void* Wv, nm_dtype wdt, int64_t ldwv,
                              int64_t R, int64_t K, int Ns, const uint8_t* mask_in, uint8_t* mask_out, int64_t ldm,
                              nm_dtype vdt, void* vals, int64_t ldv, uint32_t* idx, int64_t ldi, unsigned flags,
                              nm_stream_t stream) {
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ((flags & ~NM_FLAG_VALIDATE) == 0, NM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, flags);
    NM_REQ(Ns >= 2 && Ns <= 8, NM_ERR_PATTERN, "%s: slide N must be in [2, 8] (got %d)", fn, Ns);
    NM_REQ(K % (2 * Ns) == 0, NM_ERR_SHAPE, "%s: K %% 2N != 0", fn);
    if (R * K == 0) return NM_OK;
    if (select) {
        nm_status st = check_score_src(Wsc, sdt, ldsc, H, ldh, mode, R, K, fn);
        if (st != NM_OK) return st;
        NM_REQ(!mask_out || ldm >= (K + 7) / 8, NM_ERR_SHAPE, "%s: ldm too small", fn);
    } else {
        NM_REQ(mask_in, NM_ERR_NULL, "%s: mask is NULL", fn);
        NM_REQ(ldm >= (K + 7) / 8, NM_ERR_SHAPE, "%s: ldm too small", fn);
    }
    NM_REQ(Wv, NM_ERR_NULL, "%s: W is NULL", fn);
    NM_REQ(ldwv >= K, NM_ERR_SHAPE, "%s: ldw < K", fn);
    const int64_t Kl = K / (2 * Ns) * 4 * (Ns - 1);
    const int64_t slots = Kl / 2, words = (Kl + 31) / 32;
    nm_status st = check_pack_out(fn, wdt, vdt, R, K, slots, words, vals, ldv, idx, ldi);
    if (st != NM_OK) return st;
    const Range rv = span(vals, R, slots, ldv, esize(vdt)), ri = span(idx, R, words, ldi, 4);
    const Range rm = select ? span(mask_out, R, (K + 7) / 8, ldm, 1) : Range{0, 0};
    const Range in[4] = {select ? span(Wsc, R, K, ldsc, esize(sdt)) : Range{0, 0}, span(Wv, R, K, ldwv, esize(wdt)),
                         (select && mode == NM_SCORE_HESSIAN) ? span(H, ldh ? R : 1, K, ldh ? ldh : K, 4) : Range{0, 0},
                         select ? Range{0, 0} : span(mask_in, R, (K + 7) / 8, ldm, 1)};
    for (const Range& x : in)
        NM_REQ(!overlap(rv, x) && !overlap(ri, x) && !overlap(rm, x), NM_ERR_ALIAS, "%s: an output overlaps an input",
               fn);
    NM_REQ(!overlap(rm, rv) && !overlap(rm, ri), NM_ERR_ALIAS, "%s: mask overlaps vals/idx", fn);
    if (!select) {
        st = validate_mask(fn, flags, mask_in, ldm, R, K, 2 * Ns, 2 * Ns - 2, stream);
        if (st != NM_OK) return st;
    }
    launch_slide(Wsc, sdt, ldsc, H, ldh, eps, mode, select, Wv, wdt, ldwv, R, K, Ns, mask_in, mask_out, ldm, vdt, vals,
                 ldv, idx, ldi, (hipStream_t)stream);
    return check_launch(fn);
}

nm_status nm_slide_decompose(const void* W, nm_dtype wdt, int64_t R, int64_t K, int64_t ldw, const uint8_t* mask,
                             int64_t ldm, int Ns, nm_dtype vdt, void* vals, int64_t ldv, uint32_t* idx, int64_t ldi,
                             unsigned flags, nm_stream_t stream) {
    return slide_common("nm_slide_decompose", false, nullptr, NM_F32, 0, nullptr, 0, 0.f, NM_SCORE_MAGNITUDE, W, wdt,
                        ldw, R, K, Ns, mask, nullptr, ldm, vdt, vals, ldv, idx, ldi, flags, stream);
}

nm_status nm_prune_slide(const void* Wsc, nm_dtype sdt, int64_t ldsc, const float* H, int64_t ldh, float eps,
                         nm_score_mode mode, const void* Wv, nm_dtype wdt, int64_t ldwv, int64_t R, int64_t K, int Ns,
                         uint8_t* mask, int64_t ldm, nm_dtype vdt, void* vals, int64_t ldv, uint32_t* idx,
                         int64_t ldi, nm_stream_t stream) {
    return slide_common("nm_prune_slide", true, Wsc, sdt, ldsc, H, ldh, eps, mode, Wv, wdt, ldwv, R, K, Ns, nullptr,
                        mask, ldm, vdt, vals, ldv, idx, ldi, 0u, stream);
}

nm_status nm_absmean(const void* W, nm_dtype wdt, int64_t R, int64_t K, int64_t ldw, float* alpha, void* ws,
                     size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_absmean";
    NM_REQ(R >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(alpha, NM_ERR_NULL, "%s: alpha is NULL", fn);
    NM_REQ(W || R * K == 0, NM_ERR_NULL, "%s: W is NULL", fn);
    NM_REQ(dtype_ok(wdt) && wdt != NM_FP8, NM_ERR_DTYPE, "%s: W must be f32, bf16, int8 or int32", fn);
    NM_REQ(ldw >= K, NM_ERR_SHAPE, "%s: ldw < K", fn);
    const size_t need = reduce_ws(R, K);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(!overlap(span(alpha, 1, 1, 1, 4), span(W, R, K, ldw, esize(wdt))), NM_ERR_ALIAS, "%s: alpha overlaps W",
           fn);
    launch_absmean(W, wdt, R, K, ldw, alpha, ws, (hipStream_t)stream);
    return check_launch(fn);
}

nm_status nm_quant_lift(const void* X, nm_dtype xdt, int64_t Mtok, int64_t K, int64_t ldx, int Ns, nm_dtype qdt,
                        void* Xq, int64_t ldq, float* x_scale, nm_stream_t stream) {
    const char* fn = "nm_quant_lift";
    NM_REQ(Mtok >= 0 && K >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(Ns == 0 || (Ns >= 3 && Ns <= 8), NM_ERR_PATTERN,
           "%s: supported: no lift (Ns=0) and the (2N-2):2N lift (3 <= Ns <= 8), got Ns=%d", fn, Ns);
    NM_REQ(xdt == NM_BF16 && (qdt == NM_I8 || qdt == NM_FP8), NM_ERR_DTYPE, "%s: X must be bf16, codes I8 or FP8",
           fn);
    NM_REQ(K % 8 == 0 && (Ns == 0 || K % (2 * Ns) == 0), NM_ERR_SHAPE, "%s: K must be a multiple of 8 and of 2N", fn);
    if (Mtok == 0 || K == 0) return NM_OK;
    NM_REQ(X && Xq && x_scale, NM_ERR_NULL, "%s: NULL argument", fn);
    const int64_t Kl = Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K;
    NM_REQ(ldx >= K && ldq >= Kl, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    NM_REQ(aligned16(X) && (ldx * 2) % 16 == 0 && ((uintptr_t)Xq & (Ns ? 3u : 7u)) == 0 && ldq % (Ns ? 4 : 8) == 0,
           NM_ERR_ALIGN, "%s: X needs 16-byte aligned rows, Xq 4-byte (lifted) or 8-byte aligned rows", fn);
    const Range rx = span(X, Mtok, K, ldx, 2), rq = span(Xq, Mtok, Kl, ldq, 1), rs = span(x_scale, 1, Mtok, Mtok, 4);
    NM_REQ(!overlap(rq, rx) && !overlap(rs, rx) && !overlap(rq, rs), NM_ERR_ALIAS, "%s: outputs overlap", fn);
    launch_quant_lift(X, Mtok, K, ldx, Ns, qdt, Xq, ldq, x_scale, (hipStream_t)stream);
    return check_launch(fn);
}

// Whether a product over K columns with pattern Ns exists; the queries answer 0 for the others, whose
// lifted width may be 0 (the call refuses them).
static bool product_shape_ok(int64_t K, int Ns) {
    return K > 0 && (Ns == 0 || (Ns >= 3 && Ns <= 8 && K % (2 * Ns) == 0));
}

size_t nm_spmm_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns, nm_dtype xdt) {
    if (Mtok <= 0 || R <= 0 || !product_shape_ok(K, Ns)) return 0;
    return spmm_ws(Mtok, K, R, Ns, xdt);
}

}  // extern "C"

// Argument checks of nm_spmm and nm_spmm_noalloc (everything but the workspace).  *run is
// false when there is nothing to compute.
static nm_status spmm_check(const char* fn, const void* X, nm_dtype xdt, int64_t Mtok, int64_t K, int64_t ldx,
                            const void* vals, nm_dtype vdt, const uint32_t* idx, int64_t R, int64_t ldv, int64_t ldi,
                            int Ns, const float* x_scale, void* Y, nm_dtype ydt, int64_t ldy, bool* run) {
    *run = false;
    NM_REQ(Mtok >= 0 && K >= 0 && R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(Ns == 0 || (Ns >= 3 && Ns <= 8), NM_ERR_PATTERN,
           "%s: supported patterns are plain 2:4 (Ns=0) and (2N-2):2N via slide (3 <= Ns <= 8), got Ns=%d", fn, Ns);
    NM_REQ((xdt == NM_BF16 && vdt == NM_BF16 && (ydt == NM_BF16 || ydt == NM_F32)) ||
               (xdt == NM_I8 && vdt == NM_I8 && (ydt == NM_I32 || ydt == NM_F32 || ydt == NM_BF16)) ||
               (xdt == NM_FP8 && vdt == NM_FP8 && (ydt == NM_F32 || ydt == NM_BF16)),
           NM_ERR_DTYPE, "%s: supported: bf16 x bf16 -> bf16/f32, int8 x int8 -> int32/f32/bf16, fp8 x fp8 -> f32/bf16",
           fn);
    // the 2:4 product runs over the lifted width K' = (2 - 2/N) K: K' a multiple of one sparse
    // instruction's half depth (16 bf16, 32 one-byte columns)
    const int64_t kmult = xdt == NM_BF16 ? 16 : 32;
    NM_REQ(Ns == 0 || K % (2 * Ns) == 0, NM_ERR_SHAPE, "%s: K must be a multiple of 2N = %d", fn, 2 * Ns);
    const int64_t Kl = Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K;
    NM_REQ(Kl % kmult == 0, NM_ERR_SHAPE, "%s: the (lifted) width %lld must be a multiple of %lld for this dtype", fn,
           (long long)Kl, (long long)kmult);
    if (xdt == NM_I8) NM_REQ(Kl * 127 * 127 < (1LL << 31), NM_ERR_SHAPE, "%s: int8 sum may overflow int32", fn);
    if (Mtok == 0 || R == 0) return NM_OK;
    NM_REQ(Y, NM_ERR_NULL, "%s: Y is NULL", fn);
    NM_REQ(ldy >= R, NM_ERR_SHAPE, "%s: ldy < R", fn);
    if (K == 0) return set_error(NM_ERR_SHAPE, "%s: K == 0", fn);
    NM_REQ(X && vals && idx, NM_ERR_NULL, "%s: NULL input", fn);
    const int64_t es = esize(xdt);
    const int64_t iw = (Kl + 31) / 32;   // index words per row
    NM_REQ(ldx >= K && ldv >= Kl / 2 && ldi >= iw, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    NM_REQ(aligned16(X) && aligned16(vals) && (ldx * es) % 16 == 0 && (ldv * es) % 16 == 0, NM_ERR_ALIGN,
           "%s: X and vals must be 16-byte aligned with 16-byte row strides", fn);
    NM_REQ(((uintptr_t)idx & 3u) == 0, NM_ERR_ALIGN, "%s: idx must be 4-byte aligned", fn);
    const Range ry = span(Y, Mtok, R, ldy, esize(ydt));
    NM_REQ(!overlap(ry, span(X, Mtok, K, ldx, es)) && !overlap(ry, span(vals, R, Kl / 2, ldv, es)) &&
               !overlap(ry, span(idx, R, iw, ldi, 4)) && !overlap(ry, span(x_scale, 1, Mtok, Mtok, 4)),
           NM_ERR_ALIAS, "%s: Y overlaps an input", fn);
    *run = true;
    return NM_OK;
}

// ------------------------------------------------------------------ the product's own scratch
// The workspace of nm_spmm_noalloc: a static device array of NM_SPMM_SCRATCH_BYTES, one copy per
// GPU, held until the process ends.  In host code `g_spmm_scratch` names a host-side stand-in;
// its device address on a GPU comes from hipGetSymbolAddress with that GPU current, looked up
// once per device and kept in g_scratch_dev[] -- only that address is ever handed to kernels.
static __device__ __align__(256) uint8_t g_spmm_scratch[NM_SPMM_SCRATCH_BYTES];

static nm_status scratch_for(nm_stream_t stream, void** out) {
    constexpr int kMaxDev = 64;
    static void* dev_ptr[kMaxDev] = {};
    static std::mutex mu;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return set_error(NM_ERR_DEVICE, "nm_spmm_noalloc: hipGetDevice: %s", hipGetErrorString(e));
    NM_REQ(dev >= 0 && dev < kMaxDev, NM_ERR_DEVICE, "nm_spmm_noalloc: device %d out of range", dev);
    if (stream) {
        hipDevice_t sdev = -1;
        e = hipStreamGetDevice((hipStream_t)stream, &sdev);
        if (e != hipSuccess)
            return set_error(NM_ERR_DEVICE, "nm_spmm_noalloc: hipStreamGetDevice: %s", hipGetErrorString(e));
        NM_REQ(sdev == dev, NM_ERR_DEVICE, "nm_spmm_noalloc: the stream belongs to device %d, the current device is %d",
               (int)sdev, dev);
    }
    std::lock_guard<std::mutex> lock(mu);
    if (!dev_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_spmm_scratch));
        if (e != hipSuccess || !p)
            return set_error(NM_ERR_DEVICE, "nm_spmm_noalloc: hipGetSymbolAddress of the scratch buffer: %s",
                             hipGetErrorString(e));
        dev_ptr[dev] = p;
    }
    *out = dev_ptr[dev];
    return NM_OK;
}

extern "C" {

nm_status nm_spmm(const void* X, nm_dtype xdt, int64_t Mtok, int64_t K, int64_t ldx, const void* vals, nm_dtype vdt,
                  const uint32_t* idx, int64_t R, int64_t ldv, int64_t ldi, int Ns, const float* x_scale,
                  float w_scale, void* Y, nm_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_spmm";
    bool run = false;
    nm_status st = spmm_check(fn, X, xdt, Mtok, K, ldx, vals, vdt, idx, R, ldv, ldi, Ns, x_scale, Y, ydt, ldy, &run);
    if (st != NM_OK || !run) return st;
    const Range ry = span(Y, Mtok, R, ldy, esize(ydt));
    const size_t need = spmm_ws(Mtok, K, R, Ns, xdt);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(need == 0 || aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    if (need) NM_REQ(!overlap(ry, Range{(uintptr_t)ws, (uintptr_t)ws + need}), NM_ERR_ALIAS, "%s: Y overlaps ws", fn);
    return launch_spmm(X, xdt, Mtok, K, ldx, vals, idx, R, ldv, ldi, Ns, x_scale, w_scale, Y, ydt, ldy, ws, ws_bytes,
                       (hipStream_t)stream);
}

nm_status nm_spmm_noalloc(const void* X, nm_dtype xdt, int64_t Mtok, int64_t K, int64_t ldx, const void* vals,
                          nm_dtype vdt, const uint32_t* idx, int64_t R, int64_t ldv, int64_t ldi, int Ns,
                          const float* x_scale, float w_scale, void* Y, nm_dtype ydt, int64_t ldy,
                          nm_stream_t stream) {
    const char* fn = "nm_spmm_noalloc";
    bool run = false;
    nm_status st = spmm_check(fn, X, xdt, Mtok, K, ldx, vals, vdt, idx, R, ldv, ldi, Ns, x_scale, Y, ydt, ldy, &run);
    if (st != NM_OK || !run) return st;
    const size_t need = spmm_ws(Mtok, K, R, Ns, xdt);
    NM_REQ(need <= NM_SPMM_SCRATCH_BYTES, NM_ERR_WORKSPACE,
           "%s: this product needs %zu bytes of workspace, more than the %zu-byte scratch buffer; use nm_spmm", fn,
           need, (size_t)NM_SPMM_SCRATCH_BYTES);
    void* ws = nullptr;
    if (need) {
        st = scratch_for(stream, &ws);
        if (st != NM_OK) return st;
    }
    return launch_spmm(X, xdt, Mtok, K, ldx, vals, idx, R, ldv, ldi, Ns, x_scale, w_scale, Y, ydt, ldy, ws, need,
                       (hipStream_t)stream);
}

nm_status nm_bitmap_encode(const void* W, nm_dtype wdt, int64_t R, int64_t K, int64_t ldw, const uint8_t* mask,
                           int64_t ldm, void* vals, int64_t ldv, int32_t* offs, int64_t ldo, nm_stream_t stream) {
    const char* fn = "nm_bitmap_encode";
    NM_REQ(R >= 0 && K >= 0 && ldv >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(wdt == NM_BF16, NM_ERR_DTYPE, "%s: W must be bf16", fn);
    NM_REQ(K % 64 == 0, NM_ERR_SHAPE, "%s: K must be a multiple of 64", fn);
    if (R == 0) return NM_OK;
    NM_REQ(W && mask && offs && (vals || ldv == 0), NM_ERR_NULL, "%s: NULL argument", fn);
    NM_REQ(ldw >= K && ldm >= K / 8 && ldo >= K / 64 + 1, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    NM_REQ(aligned16(W) && ldw % 8 == 0 && ((uintptr_t)mask & 7u) == 0 && ldm % 8 == 0 && ((uintptr_t)offs & 3u) == 0 &&
               ((uintptr_t)vals & 1u) == 0,
           NM_ERR_ALIGN, "%s: W needs 16-byte aligned rows, mask 8-byte aligned rows", fn);
    const Range rv = span(vals, R, ldv, ldv, 2), ro = span(offs, R, K / 64 + 1, ldo, 4);
    NM_REQ(!overlap(rv, ro) && !overlap(rv, span(W, R, K, ldw, 2)) && !overlap(ro, span(W, R, K, ldw, 2)) &&
               !overlap(rv, span(mask, R, K / 8, ldm, 1)) && !overlap(ro, span(mask, R, K / 8, ldm, 1)),
           NM_ERR_ALIAS, "%s: an output overlaps an input or the other output", fn);
    launch_bitmap_encode(W, R, K, ldw, mask, ldm, vals, ldv, offs, ldo, (hipStream_t)stream);
    return check_launch(fn);
}

size_t nm_spmm_bitmap_workspace(int64_t Mtok, int64_t K, int64_t R) { return bitmap_spmm_ws(Mtok, K, R); }

nm_status nm_spmm_bitmap(const void* X, int64_t Mtok, int64_t K, int64_t ldx, const void* vals, int64_t ldv,
                         const uint8_t* mask, int64_t ldm, const int32_t* offs, int64_t ldo, int64_t R, void* Y,
                         nm_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_spmm_bitmap";
    NM_REQ(Mtok >= 0 && K >= 0 && R >= 0 && ldv >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(ydt == NM_BF16 || ydt == NM_F32, NM_ERR_DTYPE, "%s: Y must be bf16 or f32", fn);
    NM_REQ(K % 64 == 0, NM_ERR_SHAPE, "%s: K must be a multiple of 64", fn);
    if (Mtok == 0 || R == 0) return NM_OK;
    NM_REQ(K > 0, NM_ERR_SHAPE, "%s: K == 0", fn);
    NM_REQ(X && mask && offs && Y && vals, NM_ERR_NULL, "%s: NULL argument", fn);
    NM_REQ(ldx >= K && ldm >= K / 8 && ldo >= K / 64 + 1 && ldy >= R && ldv >= 8, NM_ERR_SHAPE,
           "%s: leading dimension too small (ldv >= 8)", fn);
    NM_REQ(aligned16(X) && ldx % 8 == 0 && ((uintptr_t)mask & 7u) == 0 && ldm % 8 == 0 && ((uintptr_t)offs & 3u) == 0 &&
               aligned16(vals) && ldv % 8 == 0,
           NM_ERR_ALIGN, "%s: X and vals need 16-byte aligned rows, mask 8-byte aligned rows", fn);
    const Range ry = span(Y, Mtok, R, ldy, esize(ydt));
    NM_REQ(!overlap(ry, span(X, Mtok, K, ldx, 2)) && !overlap(ry, span(vals, R, ldv, ldv, 2)) &&
               !overlap(ry, span(mask, R, K / 8, ldm, 1)) && !overlap(ry, span(offs, R, K / 64 + 1, ldo, 4)),
           NM_ERR_ALIAS, "%s: Y overlaps an input", fn);
    const size_t need = bitmap_spmm_ws(Mtok, K, R);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    if (need) NM_REQ(!overlap(ry, Range{(uintptr_t)ws, (uintptr_t)ws + need}), NM_ERR_ALIAS, "%s: Y overlaps ws", fn);
    return launch_bitmap_spmm(X, Mtok, K, ldx, vals, ldv, mask, ldm, offs, ldo, R, Y, ydt, ldy, ws, ws_bytes,
                              (hipStream_t)stream);
}

size_t nm_spmm_lowrank_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns, int rank) {
    if (Mtok <= 0 || R <= 0 || rank <= 0 || !product_shape_ok(K, Ns)) return 0;
    return spmm_lowrank_ws(Mtok, K, R, Ns, rank);
}

nm_status nm_spmm_lowrank(const void* X, int64_t Mtok, int64_t K, int64_t ldx, const void* vals, const uint32_t* idx,
                          int64_t R, int64_t ldv, int64_t ldi, int Ns, const void* A, int64_t lda, const void* B,
                          int64_t ldb, int rank, void* Y, nm_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes,
                          nm_stream_t stream) {
    const char* fn = "nm_spmm_lowrank";
    NM_REQ(Mtok >= 0 && K >= 0 && R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(Ns == 0 || (Ns >= 3 && Ns <= 8), NM_ERR_PATTERN,
           "%s: supported patterns are plain 2:4 (Ns=0) and (2N-2):2N via slide (3 <= Ns <= 8), got Ns=%d", fn, Ns);
    NM_REQ(ydt == NM_BF16 || ydt == NM_F32, NM_ERR_DTYPE, "%s: Y must be bf16 or f32", fn);
    NM_REQ(rank >= 8 && rank <= 256 && rank % 8 == 0, NM_ERR_SHAPE, "%s: rank must be a multiple of 8 in [8, 256]", fn);
    NM_REQ(K % 16 == 0 && (Ns == 0 || K % (2 * Ns) == 0), NM_ERR_SHAPE, "%s: K must be a multiple of 16 and of 2N", fn);
    NM_REQ((Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K) % 16 == 0, NM_ERR_SHAPE,
           "%s: the lifted width must be a multiple of 16", fn);
    if (Mtok == 0 || R == 0) return NM_OK;
    NM_REQ(K > 0, NM_ERR_SHAPE, "%s: K == 0", fn);
    NM_REQ(X && vals && idx && A && B && Y, NM_ERR_NULL, "%s: NULL argument", fn);
    const int64_t Kl = Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K;
    const int64_t iw = (Kl + 31) / 32;
    NM_REQ(ldx >= K && ldv >= Kl / 2 && ldi >= iw && lda >= K && ldb >= rank && ldy >= R, NM_ERR_SHAPE,
           "%s: leading dimension too small", fn);
    NM_REQ(aligned16(X) && aligned16(vals) && aligned16(A) && aligned16(B) && aligned16(idx) && ldx % 8 == 0 &&
               ldv % 8 == 0 && lda % 8 == 0 && ldb % 8 == 0 && ldi % 4 == 0,
           NM_ERR_ALIGN, "%s: X, vals, idx, A and B need 16-byte aligned bases and row strides", fn);
    const Range ry = span(Y, Mtok, R, ldy, esize(ydt));
    NM_REQ(!overlap(ry, span(X, Mtok, K, ldx, 2)) && !overlap(ry, span(vals, R, Kl / 2, ldv, 2)) &&
               !overlap(ry, span(idx, R, iw, ldi, 4)) && !overlap(ry, span(A, rank, K, lda, 2)) &&
               !overlap(ry, span(B, R, rank, ldb, 2)),
           NM_ERR_ALIAS, "%s: Y overlaps an input", fn);
    const size_t need = spmm_lowrank_ws(Mtok, K, R, Ns, rank);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    NM_REQ(!overlap(ry, Range{(uintptr_t)ws, (uintptr_t)ws + need}), NM_ERR_ALIAS, "%s: Y overlaps ws", fn);
    const LowRankIn lr{(const uint16_t*)A, lda, (const uint16_t*)B, ldb, rank};
    return launch_spmm_lowrank(X, Mtok, K, ldx, vals, idx, R, ldv, ldi, Ns, lr, Y, ydt, ldy, ws, ws_bytes,
                               (hipStream_t)stream);
}

size_t nm_spmm_glu_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns, nm_dtype xdt) {
    if (Mtok <= 0 || R <= 0 || !product_shape_ok(K, Ns)) return 0;
    return glu_ws(Mtok, K, R, Ns, xdt);
}

static bool act_ok(nm_act a) { return a == NM_ACT_SILU || a == NM_ACT_GELU || a == NM_ACT_GELU_TANH || a == NM_ACT_RELU2; }

nm_status nm_spmm_glu(const void* X, nm_dtype xdt, int64_t Mtok, int64_t K, int64_t ldx, const void* vals_g,
                      const uint32_t* idx_g, const void* vals_u, const uint32_t* idx_u, nm_dtype vdt, int64_t R,
                      int64_t ldv, int64_t ldi, int Ns, const float* x_scale, float g_scale, float u_scale,
                      nm_act act, void* H, nm_dtype hdt, int64_t ldh, void* G, void* U, int64_t ldg, void* ws,
                      size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_spmm_glu";
    NM_REQ(act_ok(act), NM_ERR_SHAPE, "%s: unknown activation", fn);
    NM_REQ(hdt == NM_BF16 || hdt == NM_F32, NM_ERR_DTYPE, "%s: H must be bf16 or f32", fn);
    NM_REQ(!G == !U, NM_ERR_NULL, "%s: G and U are both given or both NULL", fn);
    // each projection is held to the checks of the plain product (its output: H)
    bool run = false;
    nm_status st = spmm_check(fn, X, xdt, Mtok, K, ldx, vals_g, vdt, idx_g, R, ldv, ldi, Ns, x_scale, H, hdt, ldh, &run);
    if (st != NM_OK) return st;
    st = spmm_check(fn, X, xdt, Mtok, K, ldx, vals_u, vdt, idx_u, R, ldv, ldi, Ns, x_scale, H, hdt, ldh, &run);
    if (st != NM_OK || !run) return st;
    NM_REQ(((uintptr_t)H & (uintptr_t)(esize(hdt) - 1)) == 0 && ((uintptr_t)G & 1u) == 0 && ((uintptr_t)U & 1u) == 0,
           NM_ERR_ALIGN, "%s: an output is not element-aligned", fn);
    const size_t need = glu_ws(Mtok, K, R, Ns, xdt);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(need == 0 || aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    const int64_t Kl = Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K, es = esize(xdt), iw = (Kl + 31) / 32;
    const Range in[] = {span(X, Mtok, K, ldx, es),       span(vals_g, R, Kl / 2, ldv, es), span(idx_g, R, iw, ldi, 4),
                        span(vals_u, R, Kl / 2, ldv, es), span(idx_u, R, iw, ldi, 4),       span(x_scale, 1, Mtok, Mtok, 4)};
    Range out[4] = {span(H, Mtok, R, ldh, esize(hdt)), {0, 0}, {0, 0}, {0, 0}};
    if (need) out[3] = Range{(uintptr_t)ws, (uintptr_t)ws + need};
    if (G) {
        NM_REQ(ldg >= R, NM_ERR_SHAPE, "%s: ldg < R", fn);
        out[1] = span(G, Mtok, R, ldg, 2);
        out[2] = span(U, Mtok, R, ldg, 2);
    }
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in) NM_REQ(!overlap(out[i], r), NM_ERR_ALIAS, "%s: an output or ws overlaps an input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(out[i], out[j]), NM_ERR_ALIAS, "%s: outputs or ws overlap", fn);
    }
    GluIn g{};
    g.X = X;
    g.xdt = xdt;
    g.Mtok = Mtok;
    g.K = K;
    g.ldx = ldx;
    g.vals[0] = vals_g;
    g.vals[1] = vals_u;
    g.idx[0] = idx_g;
    g.idx[1] = idx_u;
    g.R = R;
    g.ldv = ldv;
    g.ldi = ldi;
    g.Ns = Ns;
    g.x_scale = x_scale;
    g.scale[0] = g_scale;
    g.scale[1] = u_scale;
    g.act = act;
    g.H = H;
    g.hdt = hdt;
    g.ldh = ldh;
    g.G = G;
    g.U = U;
    g.ldg = ldg;
    return launch_glu(g, ws, (hipStream_t)stream);
}

constexpr int64_t kBackwardMost = 1 << 21;   // tokens, columns, rows

// Checks and launch of both backward calls; nmat 2: the gated block (G and U given).
static nm_status backward_impl(const char* fn, GradIn in, GradOut out, int nmat, void* ws, size_t ws_bytes,
                               nm_stream_t stream) {
    const int64_t M = in.M, K = in.K, R = in.R, most = kBackwardMost;
    NM_REQ(M >= 0 && K >= 0 && R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(M <= most && K <= most && R <= most, NM_ERR_SHAPE, "%s: sizes up to 2^21", fn);
    const int Ns = in.Ns;
    NM_REQ(Ns == 0 || (Ns >= 3 && Ns <= 8), NM_ERR_PATTERN,
           "%s: supported patterns are plain 2:4 (Ns=0) and (2N-2):2N via slide (3 <= Ns <= 8), got Ns=%d", fn, Ns);
    NM_REQ(Ns == 0 || K % (2 * Ns) == 0, NM_ERR_SHAPE, "%s: K must be a multiple of 2N = %d", fn, 2 * Ns);
    const int64_t Kl = Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K;
    NM_REQ(Kl % 16 == 0, NM_ERR_SHAPE, "%s: the (lifted) width %lld must be a multiple of 16", fn, (long long)Kl);
    const bool dv = out.dV[0] != nullptr;
    NM_REQ(nmat == 1 || !out.dV[0] == !out.dV[1], NM_ERR_NULL, "%s: dVg and dVu are both given or both NULL", fn);
    NM_REQ(!out.dX || out.dxdt == NM_BF16 || out.dxdt == NM_F32, NM_ERR_DTYPE, "%s: dX must be bf16 or f32", fn);
    NM_REQ(!dv || out.dvdt == NM_BF16 || out.dvdt == NM_F32, NM_ERR_DTYPE, "%s: dV must be bf16 or f32", fn);
    if (K == 0 || (!out.dX && !dv)) return NM_OK;
    // without tokens dV is zero, without rows dX is: nothing but the outputs is touched then
    const int64_t iw = (Kl + 31) / 32;
    if (M > 0 && R > 0) {
        NM_REQ(in.dY && (nmat == 1 || (in.G && in.U)) && (in.X || !dv), NM_ERR_NULL, "%s: NULL input", fn);
        for (int i = 0; i < nmat; ++i)
            NM_REQ(in.idx[i] && (in.vals[i] || !out.dX), NM_ERR_NULL, "%s: NULL weight", fn);
        NM_REQ(in.lddy >= R && (nmat == 1 || in.ldg >= R) && (!dv || in.ldx >= K) && (!out.dX || in.ldv >= Kl / 2) &&
                   in.ldi >= iw,
               NM_ERR_SHAPE, "%s: leading dimension too small", fn);
        NM_REQ(((uintptr_t)in.dY & 1u) == 0 && ((uintptr_t)in.G & 1u) == 0 && ((uintptr_t)in.U & 1u) == 0, NM_ERR_ALIGN,
               "%s: an input is not element-aligned", fn);
        NM_REQ(!dv || (aligned16(in.X) && in.ldx % 8 == 0), NM_ERR_ALIGN, "%s: X needs 16-byte aligned rows", fn);
        for (int i = 0; i < nmat; ++i)
            NM_REQ(((uintptr_t)in.idx[i] & 3u) == 0 && (!out.dX || (aligned16(in.vals[i]) && in.ldv % 8 == 0)),
                   NM_ERR_ALIGN, "%s: vals need 16-byte aligned rows, idx 4-byte alignment", fn);
    }
    const int64_t vs = dv ? esize(out.dvdt) : 2, xs = out.dX ? esize(out.dxdt) : 2;
    NM_REQ(!out.dX || (out.lddx >= K && ((uintptr_t)out.dX & (uintptr_t)(xs - 1)) == 0), NM_ERR_SHAPE,
           "%s: lddx < K, or dX not element-aligned", fn);
    for (int i = 0; dv && i < nmat; ++i)
        NM_REQ(out.lddv >= Kl / 2 && aligned16(out.dV[i]) && (out.lddv * vs) % 16 == 0, NM_ERR_ALIGN,
               "%s: dV needs lddv >= K'/2 and 16-byte aligned rows", fn);
    const size_t need = grad_ws(M, K, R, Ns, nmat);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(need == 0 || aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    const Range rin[] = {span(in.dY, M, R, in.lddy, 2),         span(in.G, M, R, in.ldg, 2),
                         span(in.U, M, R, in.ldg, 2),           span(in.X, M, K, in.ldx, 2),
                         span(in.vals[0], R, Kl / 2, in.ldv, 2), span(in.vals[1], R, Kl / 2, in.ldv, 2),
                         span(in.idx[0], R, iw, in.ldi, 4),     span(in.idx[1], R, iw, in.ldi, 4)};
    Range rout[4] = {span(out.dX, M, K, out.lddx, xs), span(out.dV[0], R, Kl / 2, out.lddv, vs),
                     span(out.dV[1], R, Kl / 2, out.lddv, vs), {0, 0}};
    if (need) rout[3] = Range{(uintptr_t)ws, (uintptr_t)ws + need};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : rin) NM_REQ(!overlap(rout[i], r), NM_ERR_ALIAS, "%s: an output or ws overlaps an input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(rout[i], rout[j]), NM_ERR_ALIAS, "%s: outputs or ws overlap", fn);
    }
    return launch_grad(in, out, nmat, ws, (hipStream_t)stream);
}

static size_t backward_ws(int64_t Mtok, int64_t K, int64_t R, int Ns, int nmat) {
    // the call refuses the others
    const bool ok = product_shape_ok(K, Ns) && Mtok <= kBackwardMost && K <= kBackwardMost && R <= kBackwardMost;
    return ok ? grad_ws(Mtok, K, R, Ns, nmat) : 0;
}

size_t nm_spmm_backward_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns) { return backward_ws(Mtok, K, R, Ns, 1); }

nm_status nm_spmm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, int64_t Mtok, int64_t K,
                           const void* vals, const uint32_t* idx, int64_t R, int64_t ldv, int64_t ldi, int Ns, void* dX,
                           nm_dtype dxdt, int64_t lddx, void* dV, nm_dtype dvdt, int64_t lddv, void* ws,
                           size_t ws_bytes, nm_stream_t stream) {
    GradIn in{};
    in.dY = (const uint16_t*)dY;
    in.lddy = lddy;
    in.X = (const uint16_t*)X;
    in.ldx = ldx;
    in.M = Mtok;
    in.K = K;
    in.R = R;
    in.vals[0] = (const uint16_t*)vals;
    in.idx[0] = idx;
    in.ldv = ldv;
    in.ldi = ldi;
    in.Ns = Ns;
    GradOut out{dX, dxdt, lddx, {dV, nullptr}, dvdt, lddv};
    return backward_impl("nm_spmm_backward", in, out, 1, ws, ws_bytes, stream);
}

size_t nm_spmm_glu_backward_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns) {
    return backward_ws(Mtok, K, R, Ns, 2);
}

nm_status nm_spmm_glu_backward(const void* dH, int64_t lddh, const void* G, const void* U, int64_t ldg, nm_act act,
                               const void* X, int64_t ldx, int64_t Mtok, int64_t K, const void* vals_g,
                               const uint32_t* idx_g, const void* vals_u, const uint32_t* idx_u, int64_t R,
                               int64_t ldv, int64_t ldi, int Ns, void* dX, nm_dtype dxdt, int64_t lddx, void* dVg,
                               void* dVu, nm_dtype dvdt, int64_t lddv, void* ws, size_t ws_bytes, nm_stream_t stream) {
    NM_REQ(act_ok(act), NM_ERR_SHAPE, "nm_spmm_glu_backward: unknown activation");
    GradIn in{};
    in.dY = (const uint16_t*)dH;
    in.lddy = lddh;
    in.G = (const uint16_t*)G;
    in.U = (const uint16_t*)U;
    in.ldg = ldg;
    in.act = act;
    in.X = (const uint16_t*)X;
    in.ldx = ldx;
    in.M = Mtok;
    in.K = K;
    in.R = R;
    in.vals[0] = (const uint16_t*)vals_g;
    in.vals[1] = (const uint16_t*)vals_u;
    in.idx[0] = idx_g;
    in.idx[1] = idx_u;
    in.ldv = ldv;
    in.ldi = ldi;
    in.Ns = Ns;
    GradOut out{dX, dxdt, lddx, {dVg, dVu}, dvdt, lddv};
    return backward_impl("nm_spmm_glu_backward", in, out, 2, ws, ws_bytes, stream);
}

static nm_status adamw_impl(const char* fn, const nm_adamw_tensor* tensors, int count, nm_dtype sdt, double lr, double beta1,
                            double beta2, double eps, int64_t step, const uint64_t* seed, const float* grad_scale,
                            nm_stream_t stream) {
    NM_REQ(count >= 0, NM_ERR_SHAPE, "%s: negative count", fn);
    NM_REQ(sdt == NM_F32 || sdt == NM_FP8, NM_ERR_DTYPE, "%s: states must be f32 or fp8 codes", fn);
    NM_REQ(step >= 1, NM_ERR_SHAPE, "%s: step counts from 1", fn);
    NM_REQ(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps >= 0.0 && lr >= 0.0, NM_ERR_SHAPE,
           "%s: need 0 <= beta < 1, eps >= 0, lr >= 0", fn);
    if (count == 0) return NM_OK;
    NM_REQ(tensors, NM_ERR_NULL, "%s: tensors is NULL", fn);
    NM_REQ(((uintptr_t)grad_scale & 3u) == 0, NM_ERR_ALIGN, "%s: grad_scale is not element-aligned", fn);
    const bool s8 = sdt == NM_FP8;
    for (int i = 0; i < count; ++i) {
        const nm_adamw_tensor& t = tensors[i];
        NM_REQ(t.n >= 0 && t.n < (1LL << 40), NM_ERR_SHAPE, "%s: tensor %d has a size out of range", fn, i);
        NM_REQ((t.pdt == NM_F32 || t.pdt == NM_BF16) && (t.gdt == NM_F32 || t.gdt == NM_BF16), NM_ERR_DTYPE,
               "%s: tensor %d: p and g must be f32 or bf16", fn, i);
        if (t.n == 0) continue;
        NM_REQ(t.p && t.g && t.m && t.v && (!s8 || (t.m_scale && t.v_scale)), NM_ERR_NULL, "%s: tensor %d: NULL pointer",
               fn, i);
        const int64_t ps = esize(t.pdt), gs = esize(t.gdt), ss = s8 ? 1 : 4, nb = (t.n + 255) / 256;
        NM_REQ(((uintptr_t)t.p % ps) == 0 && ((uintptr_t)t.g % gs) == 0 && ((uintptr_t)t.m % ss) == 0 &&
                   ((uintptr_t)t.v % ss) == 0 && ((uintptr_t)t.copy & 1u) == 0 &&
                   (!s8 || (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) & 3u) == 0),
               NM_ERR_ALIGN, "%s: tensor %d: a pointer is not element-aligned", fn, i);
        const Range r[] = {span(t.p, 1, t.n, t.n, ps),
                           span(t.m, 1, t.n, t.n, ss),
                           span(t.v, 1, t.n, t.n, ss),
                           span(t.copy, 1, t.n, t.n, 2),
                           span(s8 ? t.m_scale : nullptr, 1, nb, nb, 4),
                           span(s8 ? t.v_scale : nullptr, 1, nb, nb, 4),
                           span(t.g, 1, t.n, t.n, gs),
                           span(grad_scale, 1, 1, 1, 4)};
        for (int a = 0; a < 6; ++a)
            for (int b = a + 1; b < 8; ++b)
                NM_REQ(!overlap(r[a], r[b]), NM_ERR_ALIAS, "%s: tensor %d: its arrays overlap", fn, i);
    }
    return launch_adamw(tensors, count, sdt, lr, beta1, beta2, eps, step, seed, grad_scale, (hipStream_t)stream);
}

nm_status nm_adamw(const nm_adamw_tensor* tensors, int count, nm_dtype sdt, double lr, double beta1, double beta2,
                   double eps, int64_t step, const float* grad_scale, nm_stream_t stream) {
    return adamw_impl("nm_adamw", tensors, count, sdt, lr, beta1, beta2, eps, step, nullptr, grad_scale, stream);
}

nm_status nm_adamw_unbiased(const nm_adamw_tensor* tensors, int count, double lr, double beta1, double beta2, double eps,
                            int64_t step, uint64_t seed, const float* grad_scale, nm_stream_t stream) {
    return adamw_impl("nm_adamw_unbiased", tensors, count, NM_FP8, lr, beta1, beta2, eps, step, &seed, grad_scale, stream);
}

}  // extern "C"
