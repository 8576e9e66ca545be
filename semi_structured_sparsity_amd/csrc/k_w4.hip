// 4-bit packed weights: the quantiser, and Y = X W^T and the gated block H = act(X Wg^T) . (X Wu^T)
// for few tokens (nm_few.h has the operands' layout and the inner product).
#include "nm_codes.h"
#include "nm_few.h"

namespace nm {

// ------------------------------------------------------------------ quantiser
// One thread takes 8 consecutive values; the group / 16 threads of a group share its maximum by
// lane moves.  s = bf16(top / 7 or 6), code = nearest to v / s.
// Bound by memory: bf16 values of 11008 x 4096 to FP4, with the values they stand for, 22.5 us (4.5 TB/s).  A
// division a value and comparisons for its nearest code took 33 (vector issue); the quotient by a corrected
// reciprocal gives the same bits.  A block takes 64 rows by 128 values, so that the scales, whose rows run along
// the weight's rows, leave as whole lines.
template <bool F32, bool FP4>
__global__ __launch_bounds__(1024) void quant_w4_kernel(const void* __restrict__ vals, int64_t ldv, int64_t R, int chunks,
                                                        int glanes, uint8_t* __restrict__ codes, int64_t ldc,
                                                        uint16_t* __restrict__ scales, int64_t lds, void* __restrict__ values,
                                                        int64_t ldo) {
    __shared__ uint16_t sc[4][64];
    const int tid = threadIdx.x, row = tid >> 4;
    const int64_t r = (int64_t)blockIdx.y * 64 + row;
    const int c = blockIdx.x * 16 + (tid & 15);
    const bool in = r < R && c < chunks;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (in) {
        if constexpr (F32) {
            const float4* p = (const float4*)((const float*)vals + r * ldv + 8 * c);
            const float4 a = p[0], b = p[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *(const uint4*)((const uint16_t*)vals + r * ldv + 8 * c);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
    // the maximum as bits: of magnitudes their order is that of the numbers, and a NaN or an infinity is
    // at the top
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    for (int off = 1; off < glanes; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    const bool bad = top >= 0x7f800000u;
    const uint32_t sb = bad ? 0x7fc0u : f32_to_bf16_bits(__fdiv_rn(__uint_as_float(top), FP4 ? 6.0f : 7.0f));
    const float s = bf16_bits_to_f32(sb);
    if ((tid & 15) % glanes == 0) sc[(tid & 15) / glanes][row] = (uint16_t)sb;
    __syncthreads();
    const int groups = 16 / glanes, all = (chunks + glanes - 1) / glanes;
    if (tid < groups * 64) {
        const int g = blockIdx.x * groups + (tid >> 6);
        const int64_t at = (int64_t)blockIdx.y * 64 + (tid & 63);
        if (g < all && at < R) scales[(int64_t)g * lds + at] = sc[tid >> 6][tid & 63];
    }
    if (!in) {   // the row's bytes up to the next 16
        if (r < R && c < (chunks + 3) / 4 * 4 && 4 * (int64_t)c < ldc) *(uint32_t*)(codes + r * ldc + 4 * c) = 0;
        return;
    }
    uint32_t word = 0;
    float o[8];
    const bool none = bad || s == 0.0f;
    const RowDiv rd = row_div(none ? 1.0f : s);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = none ? 0.0f : row_quot(v[i], rd);
    if constexpr (FP4) {
        // the conversion instructions round to the nearest code, ties to even, and hold to 6; a zero's
        // sign goes
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[0], q[1], 1.0f, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[2], q[3], 1.0f, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[4], q[5], 1.0f, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[6], q[7], 1.0f, 3);
        const uint32_t some = (word | word >> 1 | word >> 2) & 0x11111111u;
        word = (word & 0x77777777u) | (word & some << 3);
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 1);
        const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 3);
        o[0] = p0[0], o[1] = p0[1], o[2] = p1[0], o[3] = p1[1], o[4] = p2[0], o[5] = p2[1], o[6] = p3[0], o[7] = p3[1];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = __builtin_fminf(__builtin_fmaxf(rintf(q[i]), -7.0f), 7.0f) + 0.0f;   // (-0 + 0 is +0)
            const uint32_t m = (uint32_t)__builtin_fabsf(o[i]), neg = __float_as_uint(o[i]) >> 31;
            word |= (m | neg << 3) << (4 * i);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= s;
    *(uint32_t*)(codes + r * ldc + 4 * c) = word;
    if (!values) return;
    if constexpr (F32) {
        float4* p = (float4*)((float*)values + r * ldo + 8 * c);
        p[0] = make_float4(o[0], o[1], o[2], o[3]);
        p[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
        *(uint4*)((uint16_t*)values + r * ldo + 8 * c) =
            make_uint4(f32_to_bf16_pair(o[0], o[1]), f32_to_bf16_pair(o[2], o[3]), f32_to_bf16_pair(o[4], o[5]),
                       f32_to_bf16_pair(o[6], o[7]));
    }
}

nm_status launch_quant_w4(const void* vals, nm_dtype vdt, int64_t R, int64_t slots, int64_t ldv, nm_dtype qdt, int group,
                          void* codes, int64_t ldc, void* scales, int64_t lds, void* values, int64_t ldo, hipStream_t s) {
    const int chunks = (int)(slots / 8), glanes = group / 16;
    // columns (and the bytes up to the next 16 of a row of codes) by rows
    const dim3 grid((unsigned)ceil_div((chunks + 3) / 4 * 4, 16), (unsigned)ceil_div(R, 64));
    if (grid.y > 65535u) return set_error(NM_ERR_SHAPE, "nm_quant_w4: weight too large for one launch");
#define NM_Q(F32, FP4)                                                                                                   \
    hipLaunchKernelGGL((quant_w4_kernel<F32, FP4>), grid, dim3(1024), 0, s, vals, ldv, R, chunks, glanes, (uint8_t*)codes, ldc, \
                       (uint16_t*)scales, lds, values, ldo)
    if (vdt == NM_F32 && qdt == NM_FP4) NM_Q(true, true);
    else if (vdt == NM_F32) NM_Q(true, false);
    else if (qdt == NM_FP4) NM_Q(false, true);
    else NM_Q(false, false);
#undef NM_Q
    return check_launch("nm_quant_w4");
}

// ------------------------------------------------------------------ products
struct W4Args {
    const uint16_t* X;
    int64_t ldx;
    int Mtok, width, gshift;
    FewLift lift;
    const uint8_t* codes[2];
    const uint32_t* idx[2];
    const uint16_t* scales[2];
    int64_t ldc, ldi, lds, R;
    void* Y;
    int64_t ldy;
    int y32, act;
    float* part;      // [splits][1 or 2][Mtok][R] where the units are split over blocks (grid.z), else null
};

__device__ __forceinline__ void w4_store(const W4Args& a, int64_t tok, int64_t r, float v) {
    if (a.y32) ((float*)a.Y)[tok * a.ldy + r] = v;
    else ((uint16_t*)a.Y)[tok * a.ldy + r] = (uint16_t)f32_to_bf16_bits(v);
}

// Bound by the stream of the weight and by its latency: one token of 11008 x 4096 (16.9 MB of codes and positions)
// 8.5 us in a graph, of which the smallest launch takes 3.5; gated, twice that weight, 13.6.
// A block of NW waves owns RT tiles of 16 rows (GLU: RT / 2 tiles of 16 features, gate and up
// beside each other) and 16 CT tokens.  Its waves take units of 256 columns in turn and their sums
// meet in LDS, added in wave order; splits of the units over blocks leave partial sums for
// w4_join_kernel.  XL: the tokens (16 at most) in LDS.
template <int VT, int SPG, bool GLU, int RT, int CT, int NW, bool XL, bool LIFT>
__global__ __launch_bounds__(NW * 64) void w4_kernel(W4Args a) {
    static_assert(!GLU || RT % 2 == 0, "gate and up tiles in pairs");
    static_assert(!XL || CT == 1, "one tile of tokens in LDS");
    constexpr int TR = GLU ? RT / 2 : RT;
    __shared__ __attribute__((aligned(16))) float red[NW][RT][256];
    extern __shared__ __attribute__((aligned(16))) uint8_t xlds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t f0 = (int64_t)blockIdx.x * (16 * TR);
    const int64_t t0 = (int64_t)blockIdx.y * (16 * CT);
    const int nu = (a.width + 255) / 256, first = XL ? wave : (int)blockIdx.z * NW + wave, step = XL ? NW : NW * (int)gridDim.z;
    FewRows w[RT];
    FewUnit<VT, SPG> cur[RT];
    FewStage<NW * 64> stage;
    if constexpr (XL) stage.load(a.X, a.ldx, a.Mtok, a.width, a.lift, xlds, tid);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int m = GLU ? i & 1 : 0;
        int64_t r0 = f0 + 16 * (GLU ? i / 2 : i);
        // a tile past the last row re-reads the block's first one (its sums are not stored)
        r0 = r0 < a.R ? r0 : f0;
        w[i] = few_rows(a.codes[m], a.idx[m], a.scales[m], a.ldc, a.ldi, a.lds, r0, a.R, lane);
        cur[i].load(w[i], first < nu ? first : 0, a.width, a.gshift, lane);
    }
    few_f32x4 acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = few_f32x4{0, 0, 0, 0};
    if constexpr (XL) {
        const int stride = few_lds_row(a.width);
        stage.store(a.Mtok, a.width, xlds, tid);
        __syncthreads();
        const int t = (lane & 15) < a.Mtok ? lane & 15 : a.Mtok - 1;
        const FewXLds x{xlds + t * stride};
        few_product<VT, SPG, RT, CT>(cur, w, x, first, step, nu, a.width, a.gshift, a.lift, lane, acc);
    } else {
        FewXDirect<CT, LIFT> x;
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int64_t t = t0 + 16 * j + (lane & 15);
            x.row[j] = a.X + (t < a.Mtok ? t : a.Mtok - 1) * a.ldx;
        }
        few_product<VT, SPG, RT, CT>(cur, w, x, first, step, nu, a.width, a.gshift, a.lift, lane, acc);
    }

#pragma unroll
    for (int j = 0; j < CT; ++j) {
        if (t0 + 16 * j >= a.Mtok) break;
        if (j) __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; ++i) *(few_f32x4*)&red[wave][i][lane * 4] = acc[i][j];
        __syncthreads();
        // output e of a tile: lane e / 4's accumulator e % 4
        for (int e = tid; e < TR * 256; e += NW * 64) {
            const int tile = e >> 8, k = e & 255;
            const int64_t tok = t0 + 16 * j + ((k >> 2) & 15), r = f0 + 16 * tile + 4 * (k >> 6) + (k & 3);
            if (tok >= a.Mtok || r >= a.R) continue;
            float v = 0.0f, up = 0.0f;
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                v += red[n][GLU ? 2 * tile : tile][k];
                if constexpr (GLU) up += red[n][2 * tile + 1][k];
            }
            if (!XL && a.part) {
                float* p = a.part + ((int64_t)blockIdx.z * (GLU ? 2 : 1) * a.Mtok + tok) * a.R + r;
                p[0] = v;
                if constexpr (GLU) p[(int64_t)a.Mtok * a.R] = up;
                continue;
            }
            if constexpr (GLU) v = few_act(a.act, v) * up;
            w4_store(a, tok, r, v);
        }
    }
}

// The splits' partial sums added in order, and what follows a sum.
template <bool GLU>
__global__ __launch_bounds__(256) void w4_join_kernel(W4Args a, int splits) {
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x, tok = blockIdx.y;
    if (r >= a.R) return;
    const int64_t all = (int64_t)a.Mtok * a.R;
    const float* p = a.part + tok * a.R + r;
    float v = split_sum(p, splits, (GLU ? 2 : 1) * all);
    if constexpr (GLU) v = few_act(a.act, v) * split_sum(p + all, splits, 2 * all);
    w4_store(a, tok, r, v);
}

template <int VT, int SPG, bool GLU, int RT, int CT, int NW, bool XL, bool LIFT>
static void w4_go(const W4Args& a, hipStream_t s, int splits = 1) {
    constexpr int rows = 16 * (GLU ? RT / 2 : RT);
    const dim3 grid((unsigned)ceil_div(a.R, rows), (unsigned)ceil_div(a.Mtok, 16 * CT), (unsigned)splits);
    const size_t lds = XL ? (size_t)a.Mtok * few_lds_row(a.width) : 0;
    hipLaunchKernelGGL((w4_kernel<VT, SPG, GLU, RT, CT, NW, XL, LIFT>), grid, dim3(NW * 64), lds, s, a);
    if (splits > 1)
        hipLaunchKernelGGL((w4_join_kernel<GLU>), dim3((unsigned)ceil_div(a.R, 256), (unsigned)a.Mtok), dim3(256), 0, s, a, splits);
}

// How a product of more than 16 tokens is cut up: tiles of 16 tokens a wave, and blocks that share a block's units
// (their sums go through the workspace).  Splits pay where the rows alone leave the chip short of waves and a
// wave is left at least a unit: 33 tokens of 4096 x 11008 29.7 us without, 21.8 with 8; 32 of 4096 x 4096 13.1
// and 11.3 with 4; 20 of 1024 x 2048 7.0 and 9.0 with 2.
struct W4Plan {
    int ct, splits;
};
static W4Plan w4_plan(int64_t Mtok, int64_t width, int64_t R, bool glu) {
    W4Plan p{2, 1};
    if (Mtok <= 16) return p;
    const int ct = Mtok > 32 && Mtok <= 48 ? 3 : 2;
    const int64_t nu = ceil_div(width, 256), base = ceil_div(R, glu ? 32 : 64) * ceil_div(Mtok, 16 * ct);
    int64_t splits = nu / 4 < 512 / base ? nu / 4 : 512 / base;
    if (nu >= 16 && splits >= 2) p = W4Plan{ct, (int)splits};
    return p;
}
size_t w4_ws(int64_t Mtok, int64_t width, int64_t R, bool glu) {
    const W4Plan p = w4_plan(Mtok, width, R, glu);
    return p.splits > 1 ? (size_t)p.splits * (glu ? 2 : 1) * (size_t)Mtok * (size_t)R * 4 : 0;
}

// Up to four tokens whose rows fit 32 KB of LDS: one tile (or gate and up pair) a block, waves by the number of
// tiles (one token of 11008 x 4096: 4 waves 8.4 us, 8 waves 8.8; of 4096 x 4096: 5.9 and 5.3).
// Up to 16 tokens: from memory; lifted ones with two tiles a block, which share the lifting's arithmetic
// (16 tokens of 6912 x 2560 6:8 gated: 15.5 us against 21.6), plain ones with one (of 11008 x 4096 gated: 23.5
// against 25.5).
// More: split as planned; else 32 at a time, four tiles a block where that still gives the chip blocks (32 tokens
// of 11008 x 4096: 17.8 us against 24.3 with two), two where not.
template <int VT, int SPG, bool GLU, bool LIFT>
static void w4_tokens(const W4Args& a, const W4Plan& p, hipStream_t s) {
    constexpr int W = GLU ? 2 : 1;
    if (a.Mtok <= 16) {
        w4_go<VT, SPG, GLU, LIFT ? 2 * W : W, 1, 8, false, LIFT>(a, s);
    } else if (p.splits > 1 && p.ct == 3) {
        w4_go<VT, SPG, GLU, 4, 3, 4, false, LIFT>(a, s, p.splits);
    } else if (p.splits > 1 || ceil_div(a.R, 64 / W) * ceil_div(a.Mtok, 32) >= 160) {
        w4_go<VT, SPG, GLU, 4, 2, 4, false, LIFT>(a, s, p.splits);
    } else {
        w4_go<VT, SPG, GLU, 2, 2, 8, false, LIFT>(a, s);
    }
}

template <int VT, int SPG, bool GLU>
static void w4_lift(const W4Args& a, const W4Plan& p, hipStream_t s) {
    constexpr int W = GLU ? 2 : 1;
    if (a.Mtok <= 4 && (int64_t)a.Mtok * few_lds_row(a.width) <= 32 * 1024) {
        if (a.R >= 512 * 16) w4_go<VT, SPG, GLU, W, 1, 4, true, false>(a, s);
        else w4_go<VT, SPG, GLU, W, 1, 8, true, false>(a, s);
    } else if (a.lift.Ns) {
        w4_tokens<VT, SPG, GLU, true>(a, p, s);
    } else {
        w4_tokens<VT, SPG, GLU, false>(a, p, s);
    }
}

template <int VT, bool GLU>
static void w4_group(const W4Args& a, const W4Plan& p, hipStream_t s) {
    if (a.gshift == 6) w4_lift<VT, 1, GLU>(a, p, s);
    else w4_lift<VT, 2, GLU>(a, p, s);
}

nm_status launch_w4(const W4In& in, void* ws, hipStream_t s) {
    W4Args a{};
    a.X = in.X;
    a.ldx = in.ldx;
    a.Mtok = (int)in.Mtok;
    a.lift = few_lift(in.Ns);
    a.width = (int)(in.Ns ? in.K / (2 * in.Ns) * 4 * (in.Ns - 1) : in.K);
    a.gshift = in.group == 64 ? 6 : in.group == 128 ? 7 : 8;
    for (int m = 0; m < 2; ++m) {
        a.codes[m] = (const uint8_t*)in.codes[m];
        a.idx[m] = in.idx[m];
        a.scales[m] = (const uint16_t*)in.scales[m];
    }
    a.ldc = in.ldc;
    a.ldi = in.ldi;
    a.lds = in.lds;
    a.R = in.R;
    a.Y = in.Y;
    a.ldy = in.ldy;
    a.y32 = in.ydt == NM_F32;
    a.act = in.act;
    const bool glu = in.codes[1] != nullptr;
    const W4Plan p = w4_plan(in.Mtok, a.width, in.R, glu);
    a.part = p.splits > 1 ? (float*)ws : nullptr;
    if (in.qdt == NM_FP4) {
        if (glu) w4_group<kFewFP4, true>(a, p, s);
        else w4_group<kFewFP4, false>(a, p, s);
    } else {
        if (glu) w4_group<kFewI4, true>(a, p, s);
        else w4_group<kFewI4, false>(a, p, s);
    }
    return check_launch(glu ? "nm_spmm_glu_w4" : "nm_spmm_w4");
}

}  // namespace nm
