// C ABI of include/nmsparse_layers.h: argument validation and dispatch, as in nm_capi.hip.
// Nothing is enqueued unless every check passes.
#include "nm_check.h"

using namespace nm;

namespace {

bool known_act(nm_act a) { return a == NM_ACT_SILU || a == NM_ACT_GELU || a == NM_ACT_GELU_TANH || a == NM_ACT_RELU2; }
bool code4(nm_dtype d) { return d == NM_I4 || d == NM_FP4; }
bool group_ok(int g) { return g == 64 || g == 128 || g == 256; }
int64_t lifted(int64_t K, int Ns) { return Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K; }

constexpr int64_t kMost = (int64_t)1 << 24;   // tokens, columns, rows of one call
constexpr int64_t kW4MostTokens = (int64_t)1 << 20;
constexpr int64_t kQuantMost = (int64_t)1 << 21;   // rows of the quantiser
constexpr int64_t kNormMost = 32768;           // columns of a norm
constexpr int64_t kMoeMostTokens = 64;
constexpr int kMoeMostExperts = 512, kMoeMostTopk = 16;

// the checks of a 4-bit product; nw: 1, or 2 weights (gated block)
nm_status w4_check(const char* fn, const W4In& in, int nw, const void* ws, size_t ws_bytes, bool* run) {
    *run = false;
    NM_REQ(in.Mtok >= 0 && in.K >= 0 && in.R >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(in.Mtok <= kW4MostTokens && in.K <= kMost && in.R <= kMost, NM_ERR_SHAPE, "%s: up to 2^20 tokens, widths and rows up to 2^24",
           fn);
    NM_REQ(in.Ns == 0 || (in.Ns >= 3 && in.Ns <= 8), NM_ERR_PATTERN,
           "%s: supported patterns are plain 2:4 (Ns=0) and (2N-2):2N via slide (3 <= Ns <= 8), got Ns=%d", fn, in.Ns);
    NM_REQ(code4(in.qdt), NM_ERR_DTYPE, "%s: codes are NM_I4 or NM_FP4", fn);
    NM_REQ(in.ydt == NM_BF16 || in.ydt == NM_F32, NM_ERR_DTYPE, "%s: the output must be bf16 or f32", fn);
    NM_REQ(group_ok(in.group), NM_ERR_SHAPE, "%s: group must be 64, 128 or 256 (got %d)", fn, in.group);
    NM_REQ(in.Ns == 0 || in.K % (2 * in.Ns) == 0, NM_ERR_SHAPE, "%s: K must be a multiple of 2N = %d", fn, 2 * in.Ns);
    const int64_t Kl = lifted(in.K, in.Ns);
    NM_REQ(Kl % 16 == 0, NM_ERR_SHAPE, "%s: the (lifted) width %lld must be a multiple of 16", fn, (long long)Kl);
    if (in.Mtok == 0 || in.R == 0) return NM_OK;
    NM_REQ(in.K > 0, NM_ERR_SHAPE, "%s: K == 0", fn);
    NM_REQ(in.X && in.Y, NM_ERR_NULL, "%s: NULL argument", fn);
    const int64_t iw = (Kl + 31) / 32, groups = ceil_div(Kl, in.group);
    NM_REQ(in.ldx >= in.K && in.ldc >= Kl / 4 && in.ldi >= iw && in.lds >= in.R && in.ldy >= in.R, NM_ERR_SHAPE,
           "%s: leading dimension too small", fn);
    NM_REQ(in.ldc < (1 << 26) && in.ldi < (1 << 24), NM_ERR_SHAPE, "%s: leading dimension of the weight too large", fn);
    NM_REQ(aligned16(in.X) && in.ldx % 8 == 0 && in.ldc % 16 == 0, NM_ERR_ALIGN,
           "%s: X and codes need 16-byte aligned bases and row strides", fn);
    NM_REQ(aligned_to(in.Y, esize(in.ydt)), NM_ERR_ALIGN, "%s: the output is not element-aligned", fn);
    NM_REQ(in.lds % 4 == 0, NM_ERR_ALIGN, "%s: lds must be a multiple of 4", fn);
    const size_t need = w4_ws(in.Mtok, Kl, in.R, nw == 2);
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(need == 0 || aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    const Range y = span(in.Y, in.Mtok, in.R, in.ldy, esize(in.ydt));
    const Range w = need ? Range{(uintptr_t)ws, (uintptr_t)ws + need} : Range{0, 0}, x = span(in.X, in.Mtok, in.K, in.ldx, 2);
    NM_REQ(!overlap(y, x) && !overlap(w, x) && !overlap(y, w), NM_ERR_ALIAS, "%s: the output, X and ws overlap", fn);
    for (int m = 0; m < nw; ++m) {
        NM_REQ(in.codes[m] && in.idx[m] && in.scales[m], NM_ERR_NULL, "%s: NULL weight", fn);
        NM_REQ(aligned16(in.codes[m]), NM_ERR_ALIGN, "%s: X and codes need 16-byte aligned bases and row strides", fn);
        NM_REQ(aligned_to(in.idx[m], 4), NM_ERR_ALIGN, "%s: idx must be 4-byte aligned", fn);
        NM_REQ(aligned_to(in.scales[m], 8), NM_ERR_ALIGN, "%s: scales must be 8-byte aligned", fn);
        for (const Range& r : {span(in.codes[m], in.R, Kl / 4, in.ldc, 1), span(in.idx[m], in.R, iw, in.ldi, 4),
                               span(in.scales[m], groups, in.R, in.lds, 2)})
            NM_REQ(!overlap(y, r) && !overlap(w, r), NM_ERR_ALIAS, "%s: the output or ws overlaps a weight", fn);
    }
    *run = true;
    return NM_OK;
}

}  // namespace

extern "C" {

nm_status nm_quant_w4(const void* vals, nm_dtype vdt, int64_t R, int64_t slots, int64_t ldv, nm_dtype qdt, int group,
                      void* codes, int64_t ldc, void* scales, int64_t lds, void* values, int64_t ldo,
                      nm_stream_t stream) {
    const char* fn = "nm_quant_w4";
    NM_REQ(R >= 0 && slots >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(R <= kQuantMost && slots <= kMost, NM_ERR_SHAPE, "%s: up to 2^21 rows of 2^24 values", fn);
    NM_REQ(vdt == NM_BF16 || vdt == NM_F32, NM_ERR_DTYPE, "%s: values must be bf16 or f32", fn);
    NM_REQ(code4(qdt), NM_ERR_DTYPE, "%s: codes are NM_I4 or NM_FP4", fn);
    NM_REQ(group_ok(group), NM_ERR_SHAPE, "%s: group must be 64, 128 or 256 (got %d)", fn, group);
    NM_REQ(slots % 8 == 0, NM_ERR_SHAPE, "%s: slots must be a multiple of 8", fn);
    if (R == 0 || slots == 0) return NM_OK;
    NM_REQ(vals && codes && scales, NM_ERR_NULL, "%s: NULL argument", fn);
    const int64_t es = esize(vdt), groups = ceil_div(2 * slots, group), row16 = (slots / 2 + 15) / 16 * 16;
    const int64_t codes_row = row16 < ldc ? row16 : ldc;
    NM_REQ(ldv >= slots && ldc >= slots / 2 && lds >= R && (!values || ldo >= slots), NM_ERR_SHAPE,
           "%s: leading dimension too small", fn);
    NM_REQ(aligned16(vals) && ldv * es % 16 == 0 && (!values || (aligned16(values) && ldo * es % 16 == 0)), NM_ERR_ALIGN,
           "%s: values need 16-byte aligned bases and row strides", fn);
    NM_REQ(aligned_to(codes, 4) && ldc % 4 == 0 && aligned_to(scales, 2), NM_ERR_ALIGN,
           "%s: codes need 4-byte aligned rows, scales 2-byte alignment", fn);
    const Range in = span(vals, R, slots, ldv, es), out[] = {span(codes, R, codes_row, ldc, 1), span(scales, groups, R, lds, 2),
                                                              span(values, R, slots, ldo, es)};
    for (int i = 0; i < 3; ++i) {
        NM_REQ(!overlap(out[i], in), NM_ERR_ALIAS, "%s: an output overlaps the input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(out[i], out[j]), NM_ERR_ALIAS, "%s: outputs overlap", fn);
    }
    return launch_quant_w4(vals, vdt, R, slots, ldv, qdt, group, codes, ldc, scales, lds, values, ldo, (hipStream_t)stream);
}

static size_t w4_query(int64_t Mtok, int64_t K, int64_t R, int Ns, bool glu) {
    if (Mtok <= 0 || Mtok > kW4MostTokens || K <= 0 || K > kMost || R <= 0 || R > kMost || !(Ns == 0 || (Ns >= 3 && Ns <= 8)) ||
        (Ns && K % (2 * Ns)) || lifted(K, Ns) % 16)
        return 0;
    return w4_ws(Mtok, lifted(K, Ns), R, glu);
}

size_t nm_spmm_w4_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns) { return w4_query(Mtok, K, R, Ns, false); }

size_t nm_spmm_glu_w4_workspace(int64_t Mtok, int64_t K, int64_t R, int Ns) { return w4_query(Mtok, K, R, Ns, true); }

nm_status nm_spmm_w4(const void* X, int64_t Mtok, int64_t K, int64_t ldx, const void* codes, nm_dtype qdt,
                     const uint32_t* idx, const void* scales, int64_t R, int64_t ldc, int64_t ldi, int64_t lds,
                     int group, int Ns, void* Y, nm_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const W4In in{(const uint16_t*)X, Mtok, K, ldx, {codes, nullptr}, {idx, nullptr}, {scales, nullptr}, qdt, R, ldc, ldi,
                  lds, group, Ns, NM_ACT_SILU, Y, ydt, ldy};
    bool run = false;
    const nm_status st = w4_check("nm_spmm_w4", in, 1, ws, ws_bytes, &run);
    return st != NM_OK || !run ? st : launch_w4(in, ws, (hipStream_t)stream);
}

nm_status nm_spmm_glu_w4(const void* X, int64_t Mtok, int64_t K, int64_t ldx, const void* codes_g,
                         const uint32_t* idx_g, const void* scales_g, const void* codes_u, const uint32_t* idx_u,
                         const void* scales_u, nm_dtype qdt, int64_t R, int64_t ldc, int64_t ldi, int64_t lds, int group,
                         int Ns, nm_act act, void* H, nm_dtype hdt, int64_t ldh, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_spmm_glu_w4";
    NM_REQ(known_act(act), NM_ERR_SHAPE, "%s: unknown activation", fn);
    const W4In in{(const uint16_t*)X, Mtok, K, ldx, {codes_g, codes_u}, {idx_g, idx_u}, {scales_g, scales_u}, qdt, R, ldc,
                  ldi, lds, group, Ns, act, H, hdt, ldh};
    bool run = false;
    const nm_status st = w4_check(fn, in, 2, ws, ws_bytes, &run);
    return st != NM_OK || !run ? st : launch_w4(in, ws, (hipStream_t)stream);
}

size_t nm_moe_workspace(int64_t Mtok, int64_t K, int64_t F, int E, int topk) {
    if (Mtok <= 0 || Mtok > kMoeMostTokens || K <= 0 || F <= 0 || K > kMost || F > kMost || E <= 0 || E > kMoeMostExperts || topk <= 0 ||
        topk > E || topk > kMoeMostTopk)
        return 0;
    return moe_ws(Mtok, K, F, E, topk);
}

nm_status nm_moe(const void* X, int64_t Mtok, int64_t K, int64_t ldx, const void* router, int64_t ldr, const float* bias,
                 int E, int topk, nm_route route, int renorm, float route_scale, const nm_experts* gate,
                 const nm_experts* up, const nm_experts* down, nm_dtype vdt, int group, int64_t F, int Ns, nm_act act,
                 void* Y, nm_dtype ydt, int64_t ldy, int32_t* sel, float* wts, void* ws, size_t ws_bytes,
                 nm_stream_t stream) {
    const char* fn = "nm_moe";
    NM_REQ(Mtok >= 0 && K >= 0 && F >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(Mtok <= kMoeMostTokens, NM_ERR_SHAPE, "%s: made for up to %lld tokens (got %lld)", fn, (long long)kMoeMostTokens,
           (long long)Mtok);
    NM_REQ(K <= kMost && F <= kMost, NM_ERR_SHAPE, "%s: widths up to 2^24", fn);
    NM_REQ(E >= 1 && E <= kMoeMostExperts && topk >= 1 && topk <= E && topk <= kMoeMostTopk, NM_ERR_SHAPE,
           "%s: need 1 <= topk <= min(E, 16), E <= 512 (got %d of %d)", fn, topk, E);
    NM_REQ(route == NM_ROUTE_SOFTMAX || route == NM_ROUTE_SIGMOID, NM_ERR_SHAPE, "%s: unknown route", fn);
    NM_REQ(known_act(act), NM_ERR_SHAPE, "%s: unknown activation", fn);
    NM_REQ(Ns == 0 || (Ns >= 3 && Ns <= 8), NM_ERR_PATTERN,
           "%s: supported patterns are plain 2:4 (Ns=0) and (2N-2):2N via slide (3 <= Ns <= 8), got Ns=%d", fn, Ns);
    NM_REQ(vdt == NM_BF16 || code4(vdt), NM_ERR_DTYPE, "%s: weights are bf16 values or NM_I4 / NM_FP4 codes", fn);
    NM_REQ(ydt == NM_BF16 || ydt == NM_F32, NM_ERR_DTYPE, "%s: Y must be bf16 or f32", fn);
    NM_REQ(vdt == NM_BF16 || group_ok(group), NM_ERR_SHAPE, "%s: group must be 64, 128 or 256 (got %d)", fn, group);
    NM_REQ(K % 16 == 0 && F % 16 == 0 && (Ns == 0 || (K % (2 * Ns) == 0 && F % (2 * Ns) == 0)), NM_ERR_SHAPE,
           "%s: K and F must be multiples of 16 and of 2N", fn);
    const int64_t Kl = lifted(K, Ns), Fl = lifted(F, Ns);
    NM_REQ(Kl % 16 == 0 && Fl % 16 == 0, NM_ERR_SHAPE, "%s: the lifted widths must be multiples of 16", fn);
    if (Mtok == 0) return NM_OK;
    NM_REQ(K > 0 && F > 0, NM_ERR_SHAPE, "%s: K == 0 or F == 0", fn);
    NM_REQ(X && router && Y && gate && up && down, NM_ERR_NULL, "%s: NULL argument", fn);
    NM_REQ(ldx >= K && ldr >= K && ldy >= K, NM_ERR_SHAPE, "%s: leading dimension too small", fn);
    NM_REQ(aligned16(X) && aligned16(router) && ldx % 8 == 0 && ldr % 8 == 0, NM_ERR_ALIGN,
           "%s: X and router need 16-byte aligned bases and row strides", fn);
    NM_REQ(aligned_to(Y, esize(ydt)) && aligned_to(sel, 4) && aligned_to(wts, 4) && aligned_to(bias, 4), NM_ERR_ALIGN,
           "%s: an argument is not element-aligned", fn);
    const size_t need = moe_ws(Mtok, K, F, E, topk);
    NM_REQ(ws && ws_bytes >= need, NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    const Range out[] = {span(Y, Mtok, K, ldy, esize(ydt)), span(sel, Mtok, topk, topk, 4), span(wts, Mtok, topk, topk, 4),
                         Range{(uintptr_t)ws, (uintptr_t)ws + need}};
    const Range in[] = {span(X, Mtok, K, ldx, 2), span(router, E, K, ldr, 2), span(bias, 1, E, E, 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in) NM_REQ(!overlap(out[i], r), NM_ERR_ALIAS, "%s: an output or ws overlaps an input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(out[i], out[j]), NM_ERR_ALIAS, "%s: outputs or ws overlap", fn);
    }
    MoeIn m{};
    const nm_experts* w[3] = {gate, up, down};
    for (int i = 0; i < 3; ++i) {
        const nm_experts& e = *w[i];
        const int64_t rows = i == 2 ? K : F, width = i == 2 ? Fl : Kl, iw = (width + 31) / 32;
        const bool bf = vdt == NM_BF16;
        const int64_t vbytes = bf ? width : width / 4, es = bf ? 2 : 1, groups = bf ? 1 : ceil_div(width, group);
        NM_REQ(e.vals && e.idx && (bf || e.scales), NM_ERR_NULL, "%s: NULL weight", fn);
        NM_REQ(e.ld_vals * es >= vbytes && e.ld_idx >= iw && (bf || e.ld_scales >= rows), NM_ERR_SHAPE,
               "%s: a weight's leading dimension is too small", fn);
        NM_REQ(e.ld_vals * es < (1 << 26) && e.ld_idx < (1 << 24), NM_ERR_SHAPE, "%s: a weight's leading dimension is too large",
               fn);
        NM_REQ(e.es_vals >= 0 && e.es_idx >= 0 && (bf || e.es_scales >= 0), NM_ERR_SHAPE, "%s: negative expert stride", fn);
        NM_REQ(aligned16(e.vals) && e.ld_vals * es % 16 == 0 && e.es_vals * es % 16 == 0 && aligned_to(e.idx, 4) &&
                   (bf || (aligned_to(e.scales, 8) && e.ld_scales % 4 == 0 && e.es_scales % 4 == 0)),
               NM_ERR_ALIGN, "%s: a weight is not aligned (values 16 bytes, idx 4, scales 8)", fn);
        for (const Range& o : out) {
            Range v = span(e.vals, rows, vbytes, e.ld_vals * es, 1), x = span(e.idx, rows, iw, e.ld_idx, 4);
            Range sc = bf ? Range{0, 0} : span(e.scales, groups, rows, e.ld_scales, 2);
            v.hi += (uintptr_t)((E - 1) * e.es_vals * es);
            x.hi += (uintptr_t)((E - 1) * e.es_idx * 4);
            if (!bf) sc.hi += (uintptr_t)((E - 1) * e.es_scales * 2);
            NM_REQ(!overlap(o, v) && !overlap(o, x) && !overlap(o, sc), NM_ERR_ALIAS, "%s: an output or ws overlaps a weight", fn);
        }
        m.w[i] = e;
    }
    m.X = X;
    m.Mtok = Mtok;
    m.K = K;
    m.ldx = ldx;
    m.router = router;
    m.ldr = ldr;
    m.bias = bias;
    m.E = E;
    m.topk = topk;
    m.route = route;
    m.renorm = renorm != 0;
    m.route_scale = route_scale;
    m.vdt = vdt;
    m.group = group;
    m.F = F;
    m.Ns = Ns;
    m.act = act;
    m.Y = Y;
    m.ydt = ydt;
    m.ldy = ldy;
    m.sel = sel;
    m.wts = wts;
    return launch_moe(m, ws, (hipStream_t)stream);
}

// what both directions of the norms check: kinds, types, the side inputs
static nm_status norm_check(const char* fn, int64_t Mtok, int64_t C, nm_dtype xdt, nm_dtype wdt, const void* Y,
                            const void* gate, int64_t ldg, int64_t gate_rows, nm_norm post, const void* w_post,
                            const void* b_post, nm_norm pre, const void* w_pre, const void* b_pre, float eps) {
    NM_REQ(Mtok >= 0 && C >= 0, NM_ERR_SHAPE, "%s: negative size", fn);
    NM_REQ(Mtok <= kMost && C <= kNormMost, NM_ERR_SHAPE, "%s: up to 2^24 tokens of 32768 columns", fn);
    NM_REQ(C >= 1 || Mtok == 0, NM_ERR_SHAPE, "%s: C == 0", fn);
    NM_REQ(xdt == NM_BF16 || xdt == NM_F32, NM_ERR_DTYPE, "%s: the residual stream must be bf16 or f32", fn);
    NM_REQ(wdt == NM_BF16 || wdt == NM_F32, NM_ERR_DTYPE, "%s: weights and gate must be bf16 or f32", fn);
    for (nm_norm k : {post, pre})
        NM_REQ(k == NM_NORM_NONE || k == NM_NORM_RMS || k == NM_NORM_LAYER, NM_ERR_SHAPE, "%s: unknown norm", fn);
    NM_REQ(post != NM_NORM_NONE || (!w_post && !b_post), NM_ERR_SHAPE, "%s: w_post and b_post belong to a norm", fn);
    NM_REQ(pre != NM_NORM_NONE || (!w_pre && !b_pre), NM_ERR_SHAPE, "%s: w_pre and b_pre belong to a norm", fn);
    NM_REQ(Mtok == 0 || Y || (!gate && post == NM_NORM_NONE), NM_ERR_NULL, "%s: a gate and norm_post need Y", fn);
    NM_REQ(gate_rows >= 0, NM_ERR_SHAPE, "%s: negative gate_rows", fn);
    NM_REQ(!gate || ldg >= C, NM_ERR_SHAPE, "%s: ldg < C", fn);
    NM_REQ(eps >= 0.0f, NM_ERR_SHAPE, "%s: eps must not be negative", fn);
    const int64_t ws = esize(wdt);
    for (const void* p : {gate, w_post, b_post, w_pre, b_pre})
        NM_REQ(aligned_to(p, ws), NM_ERR_ALIGN, "%s: a weight is not element-aligned", fn);
    return NM_OK;
}

static int64_t gate_count(int64_t Mtok, int64_t gate_rows) {
    return gate_rows > 0 && Mtok > 0 ? ceil_div(Mtok, gate_rows) : 1;
}

nm_status nm_block_norm(const void* X, nm_dtype xdt, int64_t Mtok, int64_t C, int64_t ldx, float res_scale,
                        const void* Y, int64_t ldyb, const void* gate, int64_t ldg, int64_t gate_rows, nm_norm post,
                        const void* w_post, const void* b_post, nm_norm pre, const void* w_pre, const void* b_pre,
                        nm_dtype wdt, float eps, void* Z, int64_t ldz, void* Nout, nm_dtype ndt, int Ns, int64_t ldn,
                        float* n_scale, nm_stream_t stream) {
    const char* fn = "nm_block_norm";
    const nm_status st = norm_check(fn, Mtok, C, xdt, wdt, Y, gate, ldg, gate_rows, post, w_post, b_post, pre, w_pre, b_pre, eps);
    if (st != NM_OK) return st;
    const bool code = ndt == NM_I8 || ndt == NM_FP8;
    NM_REQ(ndt == NM_BF16 || ndt == NM_F32 || code, NM_ERR_DTYPE, "%s: N must be bf16, f32, int8 or FP8", fn);
    NM_REQ(Ns == 0 || (code && Ns >= 3 && Ns <= 8), NM_ERR_PATTERN, "%s: Ns is 0, or 3 to 8 for codes (got %d)", fn, Ns);
    if (Mtok == 0) return NM_OK;
    NM_REQ(X, NM_ERR_NULL, "%s: X is NULL", fn);
    NM_REQ(!Nout == (pre == NM_NORM_NONE), NM_ERR_NULL, "%s: N is given exactly with a norm_pre", fn);
    NM_REQ(!Nout || !code || n_scale, NM_ERR_NULL, "%s: codes need n_scale", fn);
    const int64_t xs = esize(xdt), ns = esize(ndt), width = lifted(C, Ns);
    NM_REQ(!code || (C % 8 == 0 && (Ns == 0 || C % (2 * Ns) == 0)), NM_ERR_SHAPE,
           "%s: codes need C a multiple of 8 and of 2N", fn);
    NM_REQ(ldx >= C && (!Y || ldyb >= C) && (!Z || ldz >= C) && (!Nout || ldn >= width), NM_ERR_SHAPE,
           "%s: leading dimension too small", fn);
    NM_REQ(aligned_to(X, xs) && aligned_to(Y, 2) && aligned_to(Z, xs) && aligned_to(Nout, code ? 4 : ns) &&
               (!code || ldn % 4 == 0) && aligned_to(n_scale, 4),
           NM_ERR_ALIGN, "%s: an argument is not aligned (elements; codes: rows of 4 bytes)", fn);
    // codes are made of whole vectors of 8 columns
    if (code && Nout)
        NM_REQ(aligned16(X) && ldx * xs % 16 == 0 && (!Y || (aligned16(Y) && ldyb % 8 == 0)) && (!Z || (aligned16(Z) && ldz * xs % 16 == 0)) &&
                   (!gate || (aligned16(gate) && ldg * esize(wdt) % 16 == 0)) && aligned16(w_post) && aligned16(b_post) &&
                   aligned16(w_pre) && aligned16(b_pre),
               NM_ERR_ALIGN, "%s: codes need 16-byte aligned rows of every other argument", fn);
    const int64_t gates = gate_count(Mtok, gate_rows), wsz = esize(wdt);
    const Range rx = span(X, Mtok, C, ldx, xs);
    const Range in[] = {span(Y, Mtok, C, ldyb, 2),      span(gate, gates, C, ldg, wsz), span(w_post, 1, C, C, wsz),
                        span(b_post, 1, C, C, wsz), span(w_pre, 1, C, C, wsz),      span(b_pre, 1, C, C, wsz)};
    const Range out[] = {span(Z, Mtok, C, ldz, xs), span(Nout, Mtok, width, ldn, ns),
                         code && Nout ? span(n_scale, 1, Mtok, Mtok, 4) : Range{0, 0}};
    const bool in_place = Z == X && ldz == ldx;
    for (int i = 0; i < 3; ++i) {
        NM_REQ((i == 0 && in_place) || !overlap(out[i], rx), NM_ERR_ALIAS, "%s: an output overlaps X (Z may be X itself)", fn);
        for (const Range& r : in) NM_REQ(!overlap(out[i], r), NM_ERR_ALIAS, "%s: an output overlaps an input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(out[i], out[j]), NM_ERR_ALIAS, "%s: outputs overlap", fn);
    }
    if (!Z && !Nout) return NM_OK;
    const NormIn n{X,    xdt,    Mtok,   C,   ldx,   res_scale, Y,   ldyb, gate, ldg, gate_rows, post,    w_post,
                   b_post, pre, w_pre, b_pre, wdt, eps, Z, ldz, Nout, ndt, Ns, ldn, n_scale};
    return launch_block_norm(n, (hipStream_t)stream);
}

size_t nm_block_norm_backward_workspace(int64_t Mtok, int64_t C, int64_t gate_rows) {
    if (Mtok <= 0 || Mtok > kMost || C <= 0 || C > kNormMost || gate_rows < 0) return 0;
    return block_norm_bwd_ws(Mtok, C, gate_rows);
}

nm_status nm_block_norm_backward(const void* Z, nm_dtype xdt, int64_t Mtok, int64_t C, int64_t ldz, const void* dZ,
                                 int64_t lddz, const void* dN, nm_dtype dndt, int64_t lddn, float res_scale,
                                 const void* Y, int64_t ldyb, const void* gate, int64_t ldg, int64_t gate_rows, nm_norm post,
                                 const void* w_post, const void* b_post, nm_norm pre, const void* w_pre, nm_dtype wdt, float eps,
                                 void* dX, int64_t lddx, void* dY, int64_t lddy, float* dw_pre, float* db_pre, float* dw_post,
                                 float* db_post, float* dgate, void* ws, size_t ws_bytes, nm_stream_t stream) {
    const char* fn = "nm_block_norm_backward";
    const nm_status st = norm_check(fn, Mtok, C, xdt, wdt, Y, gate, ldg, gate_rows, post, w_post, b_post, pre, w_pre, nullptr, eps);
    if (st != NM_OK) return st;
    NM_REQ(dndt == NM_BF16 || dndt == NM_F32, NM_ERR_DTYPE, "%s: dN must be bf16 or f32", fn);
    const bool some = Mtok > 0;
    NM_REQ(pre != NM_NORM_NONE || (!dN && !dw_pre && !db_pre), NM_ERR_NULL, "%s: dN, dw_pre and db_pre belong to a norm_pre", fn);
    NM_REQ(!some || dN || (!dw_pre && !db_pre), NM_ERR_NULL, "%s: dw_pre and db_pre need dN", fn);
    NM_REQ(post != NM_NORM_NONE || (!dw_post && !db_post), NM_ERR_NULL, "%s: dw_post and db_post belong to a norm_post", fn);
    NM_REQ(!some || Y || !dY, NM_ERR_NULL, "%s: dY needs Y", fn);
    NM_REQ(!some || gate || !dgate, NM_ERR_NULL, "%s: dgate needs a gate", fn);
    if (C == 0) return NM_OK;
    float* sums[5] = {dw_pre, db_pre, dw_post, db_post, dgate};
    const int64_t xs = esize(xdt), ns = esize(dndt), wsz = esize(wdt), gates = gate_count(Mtok, gate_rows);
    bool any = false;
    for (float* p : sums) {
        any |= p != nullptr;
        NM_REQ(aligned_to(p, 4), NM_ERR_ALIGN, "%s: a parameter gradient is not element-aligned", fn);
    }
    if (some) {
        NM_REQ(Z || !dN, NM_ERR_NULL, "%s: dN needs Z", fn);
        NM_REQ((!Z || ldz >= C) && (!dZ || lddz >= C) && (!dN || lddn >= C) && (!Y || ldyb >= C) && (!dX || lddx >= C) &&
                   (!dY || lddy >= C),
               NM_ERR_SHAPE, "%s: leading dimension too small", fn);
        NM_REQ(aligned_to(Z, xs) && aligned_to(dZ, xs) && aligned_to(dN, ns) && aligned_to(Y, 2) && aligned_to(dX, xs) &&
                   aligned_to(dY, 2),
               NM_ERR_ALIGN, "%s: an argument is not element-aligned", fn);
    }
    const size_t need = any && some ? block_norm_bwd_ws(Mtok, C, gate_rows) : 0;
    NM_REQ(need == 0 || (ws && ws_bytes >= need), NM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
    NM_REQ(need == 0 || aligned16(ws), NM_ERR_ALIGN, "%s: ws must be 16-byte aligned", fn);
    const Range rdz = span(dZ, Mtok, C, lddz, xs);
    const Range in[] = {span(Z, Mtok, C, ldz, xs),   span(dN, Mtok, C, lddn, ns),  span(Y, Mtok, C, ldyb, 2),  span(gate, gates, C, ldg, wsz),
                        span(w_post, 1, C, C, wsz), span(b_post, 1, C, C, wsz), span(w_pre, 1, C, C, wsz)};
    Range out[8] = {span(dX, Mtok, C, lddx, xs), span(dY, Mtok, C, lddy, 2)};
    for (int i = 0; i < 5; ++i) out[2 + i] = span(sums[i], i == 4 ? gates : 1, C, C, 4);
    if (need) out[7] = Range{(uintptr_t)ws, (uintptr_t)ws + need};
    const bool in_place = dX == dZ && lddx == lddz;
    for (int i = 0; i < 8; ++i) {
        NM_REQ((i == 0 && in_place) || !overlap(out[i], rdz), NM_ERR_ALIAS, "%s: an output or ws overlaps dZ (dX may be dZ itself)", fn);
        for (const Range& r : in) NM_REQ(!overlap(out[i], r), NM_ERR_ALIAS, "%s: an output or ws overlaps an input", fn);
        for (int j = 0; j < i; ++j) NM_REQ(!overlap(out[i], out[j]), NM_ERR_ALIAS, "%s: outputs or ws overlap", fn);
    }
    if (!any && (!some || (!dX && !dY))) return NM_OK;
    NormBwdIn n{Z,   xdt, Mtok, C,   ldz, dZ,   lddz,   dN,     dndt, lddn,  res_scale, Y,   ldyb, gate, ldg, gate_rows,
                post, w_post, b_post, pre, w_pre, wdt, eps, dX, lddx, dY, lddy, {}};
    for (int i = 0; i < 5; ++i) n.sums[i] = sums[i];
    return launch_block_norm_bwd(n, ws, (hipStream_t)stream);
}

}  // extern "C"
