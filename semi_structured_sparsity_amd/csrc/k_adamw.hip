// One AdamW step over many tensors (decoupled weight decay):
//   g' = g * grad_scale,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p  = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps),
// all in f32.  m, v and r = sqrt(v) take one rounding per operation in the order written, with
// no contraction, as does the quotient that picks a code below: codes are decided by them, so
// every correct evaluation of this order gives the same codes.  The parameter's update takes the
// denominator as fma(r, 1 / sqrt(1 - b2^t), eps) and the hardware's reciprocal of it (about 1e-7 relative).
//
// States in 8 bits: m and r = sqrt(v) are e4m3 codes with one f32 scale per 256 consecutive
// elements, scale = max |x| * (1 / 448), code = the e4m3 value nearest x * (448 * (1 / max)).  e4m3
// spans 18 binades below the scale's maximum, and r halves the binades v needs.  A nonzero r
// keeps at least the smallest code: an r that became zero beside an m that did not would
// divide m by eps.  The parameter update uses m and v before they are rounded to codes.
// A block whose maximum is below 2^-118 (its reciprocal would overflow) stores zeros.  NaN and
// infinite elements store the NaN code and do not enter the block's scale.
//
// Nearest codes lose a change below half a unit (3-6%) in every step, and a step takes at most
// 1 - sqrt(b2) off r: 2.5% at b2 0.95.  Only the scale's own fluctuation then moves r at an element that does
// not hold its block's maximum.  Half of a block's gradients tenfold smaller from step 1000 on, r thousands
// of steps later over the f32 one: normal gradients 1.01, 1.05, 13 and 7 at b2 0.9, 0.95, 0.99 and 0.999,
// uniform ones 1.00, 13 at 0.9, 0.95, a mean with 10% noise 1.03-1.12, 8 there, constant size 6, 10.
// The unbiased form (UNB) takes one of the two neighbouring codes with the probability that gives x on
// average: 1.00-1.02 for all of these.  Its random bits are a function of seed, step, tensor and
// element (88.8 M f32 masters 264 -> 266 us, 14.3 M bf16 parameters 34 -> 40).
//
// The step is bound by HBM: per parameter 8 B (f32 p read and written) or 4 B (bf16), the
// gradient's 2 or 4 B, 16 B of f32 states or 4 + 4/128 B of codes and scales, 2 B of the
// bf16 copy.  Descriptors travel as kernel arguments (no table upload, graph capture
// safe), kMaxTensors a launch, a tensor that passes a launch's most blocks in pieces; a block
// finds its tensor by a binary search over the tensors' first block numbers, in scalar registers.
#include <math.h>

#include "nm_adamw_pieces.h"
#include "nm_internal.h"

namespace nm {

constexpr int kMaxTensors = 44;     // descriptors per launch: kernel arguments stay below 4 KB
constexpr int kPerThread = 8;       // consecutive elements of a thread: 32 lanes hold a 256-element block
// Elements of a block.  Two passes a block with their loads issued together were 2% slower at
// 88 M parameters and 18% slower on nine small tensors (5.8 -> 7.0 us).
constexpr int kChunk = 256 * kPerThread;

enum : uint32_t { kPBf16 = 1, kGBf16 = 2, kVec = 4, kFlagBits = 3 };

struct AdamWDesc {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    uint16_t* c;
    int64_t n;
    float alpha;    // lr / (1 - b1^t)
    float decay;    // 1 - lr wd
    uint32_t flags;   // and from bit kFlagBits on the first chunk of the tensor that the piece holds
    uint32_t tensor;  // its number in the step
};
struct AdamWArgs {
    AdamWDesc t[kMaxTensors];
    uint32_t first[kMaxTensors + 1];
    int32_t count;
    const float* grad_scale;
    uint64_t seed;          // of the step (unbiased codes)
    float b1, c1, b2, c2;   // betas and 1 - beta
    float rbc2;             // 1 / sqrt(1 - b2^t)
    float eps;
};
static_assert(sizeof(AdamWArgs) <= 4096, "kernel arguments");

__device__ __forceinline__ float fin_abs(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;   // NaN compares false
}

// max over the 32 lanes of a half-wave: pairs, quads, eights and sixteens by DPP moves (lane i meets
// i ^ 1, i ^ 2, 7 - i of its eight and 15 - i of its row), then the two rows of the half
template <int CTRL>
__device__ __forceinline__ float dpp_max(float x) {
    return __builtin_fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 15, 15, true)));
}
__device__ __forceinline__ float half_max(float x) {
    x = dpp_max<0x0b1>(x);   // quad_perm [1, 0, 3, 2]
    x = dpp_max<0x04e>(x);   // quad_perm [2, 3, 0, 1]
    x = dpp_max<0x141>(x);   // row_half_mirror
    x = dpp_max<0x140>(x);   // row_mirror
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// e4m3 codes of x[0..7] * inv, packed; LEAST (x >= 0): nonzero values keep at least 2^-9 (code 1);
// nonfinite: some value may be NaN or infinite.  UNB: unbiased, by 16 random bits a value (of u[],
// from bit SHIFT on): the f32 value's 20 bits below a code's unit are carried into it by them; below the
// smallest normal 2^-6, whose unit is the one of [2^-6, 2^-5), the value is moved there and back.
template <bool LEAST, bool UNB, int SHIFT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv, bool nonfinite, const uint32_t (&u)[8]) {
    uint32_t w[2];
    const float least = inv > 0.0f ? 0x1p-9f : 0.0f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float y[4];
        uint32_t bad = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x[4 * q + e];
            // finite values are within 448 (1 + 2^-23); the clamp keeps the conversion in range
            if constexpr (UNB) {
                const float s = __fmul_rn(a, inv), b = __builtin_fminf(__builtin_fabsf(s), 448.0f);   // NaN: 448, replaced below
                const bool sub = b < 0x1p-6f;
                const float z = sub ? __fadd_rn(b, 0x1p-6f) : b;
                const uint32_t up = ((u[4 * q + e] >> SHIFT) & 0xffffu) << 4 | 8u;
                float r = __uint_as_float((__float_as_uint(z) + up) & ~0xfffffu);
                r = __builtin_fminf(sub ? r - 0x1p-6f : r, 448.0f);
                y[e] = LEAST ? (a > 0.0f ? __builtin_fmaxf(r, least) : 0.0f) : __builtin_copysignf(r, s);
            } else {
                y[e] = __builtin_amdgcn_fmed3f(__fmul_rn(a, inv), LEAST && a > 0.0f ? least : LEAST ? 0.0f : -448.0f, 448.0f);
            }
            if (nonfinite && !(__builtin_fabsf(a) < __builtin_inff())) bad |= 0x7fu << (8 * e);
        }
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], v, true);
        w[q] = (uint32_t)v | bad;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(uint2 c, float scale, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
        x[4 * q + 0] = __fmul_rn(lo[0], scale);
        x[4 * q + 1] = __fmul_rn(lo[1], scale);
        x[4 * q + 2] = __fmul_rn(hi[0], scale);
        x[4 * q + 3] = __fmul_rn(hi[1], scale);
    }
}

// How a thread reads and writes its 8 elements: one by one, in vectors where they are all inside, or
// in vectors (the whole block of threads is inside the tensor).
enum : int { kSingle = 0, kEdge = 1, kWhole = 2 };

// 8 elements from i (f32, or bf16 widened); elements at n and beyond read as zero
template <int VEC>
__device__ __forceinline__ void load8(const void* base, bool bf16, int64_t i, int64_t n, float (&x)[8]) {
    if (VEC == kWhole || (VEC == kEdge && i + 8 <= n)) {
        if (bf16) {
            const uint4 u = *(const uint4*)((const uint16_t*)base + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        } else {
            const float4 a = *(const float4*)((const float*)base + i), b = *(const float4*)((const float*)base + i + 4);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = i + e < n ? (bf16 ? bf16_bits_to_f32(((const uint16_t*)base)[i + e]) : ((const float*)base)[i + e]) : 0.0f;
}

template <int VEC>
__device__ __forceinline__ void store8(void* base, bool bf16, int64_t i, int64_t n, const float (&x)[8]) {
    if (VEC == kWhole || (VEC == kEdge && i + 8 <= n)) {
        if (bf16) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = f32_to_bf16_pair(x[2 * e], x[2 * e + 1]);
            *(uint4*)((uint16_t*)base + i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *(float4*)((float*)base + i) = make_float4(x[0], x[1], x[2], x[3]);
            *(float4*)((float*)base + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (i + e >= n) continue;
        if (bf16) ((uint16_t*)base)[i + e] = (uint16_t)f32_to_bf16_bits(x[e]);
        else ((float*)base)[i + e] = x[e];
    }
}

template <int VEC>
__device__ __forceinline__ uint2 load_codes(const void* base, int64_t i, int64_t n) {
    if (VEC == kWhole || (VEC == kEdge && i + 8 <= n)) return *(const uint2*)((const uint8_t*)base + i);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < n) w[e >> 2] |= (uint32_t)((const uint8_t*)base)[i + e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

template <int VEC>
__device__ __forceinline__ void store_codes(void* base, int64_t i, int64_t n, uint2 c) {
    if (VEC == kWhole || (VEC == kEdge && i + 8 <= n)) {
        *(uint2*)((uint8_t*)base + i) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < n) ((uint8_t*)base)[i + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
}

// What a thread reads for 8 elements, as it lies in memory.
template <bool S8>
struct Raw {
    float p[8], g[8], m[S8 ? 1 : 8], v[S8 ? 1 : 8];
    uint2 mc, vc;
    float sm, sv;
};
template <bool S8, int VEC>
__device__ __forceinline__ void adamw_load(const AdamWDesc& t, int64_t i, Raw<S8>& x) {
    const bool pb = (t.flags & kPBf16) != 0, gb = (t.flags & kGBf16) != 0;
    load8<VEC>(t.p, pb, i, t.n, x.p);
    load8<VEC>(t.g, gb, i, t.n, x.g);
    if constexpr (S8) {
        // lanes past the end hold zeros; their block may not exist
        const bool in = i < t.n;
        x.sm = in ? t.ms[i >> 8] : 0.0f;
        x.sv = in ? t.vs[i >> 8] : 0.0f;
        x.mc = load_codes<VEC>(t.m, i, t.n);
        x.vc = load_codes<VEC>(t.v, i, t.n);
    } else {
        load8<VEC>(t.m, false, i, t.n, x.m);
        load8<VEC>(t.v, false, i, t.n, x.v);
    }
}

template <bool S8, bool UNB, int VEC>
__device__ __forceinline__ void adamw_update(const AdamWArgs& a, const AdamWDesc& t, int64_t i, float gs, const Raw<S8>& x) {
    const bool pb = (t.flags & kPBf16) != 0;
    const int64_t n = t.n;
    float p[8], m[8], v[8], r[8];
    const int64_t blk = i >> 8;
    if constexpr (S8) {
        decode8(x.mc, x.sm, m);
        decode8(x.vc, x.sv, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = x.m[e], v[e] = x.v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float g = x.g[e] * gs;
        m[e] = __fadd_rn(__fmul_rn(a.b1, m[e]), __fmul_rn(a.c1, g));
        v[e] = __fadd_rn(__fmul_rn(a.b2, v[e]), __fmul_rn(__fmul_rn(a.c2, g), g));
        // correctly rounded: it decides codes, and the hardware's root takes v below 2^-126 for zero (an
        // update of m over eps then)
        r[e] = sqrtf(v[e]);
        const float d = __builtin_fmaf(r[e], a.rbc2, a.eps);
        p[e] = __builtin_fmaf(-t.alpha, m[e] * __builtin_amdgcn_rcpf(d), x.p[e] * t.decay);
    }
    store8<VEC>(t.p, pb, i, n, p);
    if (t.c) store8<VEC>(t.c, true, i, n, p);
    if constexpr (S8) {
        // one product per value tells whether any is NaN or infinite; only then are they left out of
        // the maxima and given the NaN code one by one
        float mm = 0.0f, mv = 0.0f, t0 = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mm = __builtin_fmaxf(mm, __builtin_fabsf(m[e]));
            mv = __builtin_fmaxf(mv, r[e]);
            t0 = __builtin_fmaf(m[e], 0.0f, t0);
            t0 = __builtin_fmaf(r[e], 0.0f, t0);
        }
        const bool nonfinite = t0 != t0;
        if (nonfinite) {
            mm = mv = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mm = __builtin_fmaxf(mm, fin_abs(m[e]));
                mv = __builtin_fmaxf(mv, fin_abs(r[e]));
            }
        }
        mm = half_max(mm);
        mv = half_max(mv);
        const bool zm = mm < 0x1p-118f, zv = mv < 0x1p-118f;
        uint32_t u[8] = {};
        if constexpr (UNB) {
            // two elements an output of the tensor's generator
            const uint64_t seed = splitmix64_at(a.seed, t.tensor);
            const uint64_t at = (uint64_t)(t.flags >> kFlagBits) * (kChunk / 2) + (uint64_t)i / 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t z = splitmix64_at(seed, at + e);
                u[2 * e] = (uint32_t)z;
                u[2 * e + 1] = (uint32_t)(z >> 32);
            }
        }
        store_codes<VEC>(t.m, i, n, encode8<false, UNB, 0>(m, zm ? 0.0f : __fmul_rn(448.0f, 1.0f / mm), nonfinite, u));
        store_codes<VEC>(t.v, i, n, encode8<true, UNB, 16>(r, zv ? 0.0f : __fmul_rn(448.0f, 1.0f / mv), nonfinite, u));
        if ((threadIdx.x & 31) == 0 && i < n) {
            t.ms[blk] = zm ? 0.0f : mm * (1.0f / 448.0f);
            t.vs[blk] = zv ? 0.0f : mv * (1.0f / 448.0f);
        }
    } else {
        store8<VEC>(t.m, false, i, n, m);
        store8<VEC>(t.v, false, i, n, v);
    }
}

template <bool S8, bool UNB>
__global__ __launch_bounds__(256) void adamw_kernel(AdamWArgs a) {
    const uint32_t b = blockIdx.x;
    int lo = 0, hi = a.count - 1;   // the last tensor whose first block is at or before b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    const AdamWDesc& t = a.t[lo];
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t i = (int64_t)(b - a.first[lo]) * kChunk + threadIdx.x * kPerThread;
    Raw<S8> x;
    if ((t.flags & kVec) && (int64_t)(b - a.first[lo] + 1) * kChunk <= t.n) {
        adamw_load<S8, kWhole>(t, i, x);
        adamw_update<S8, UNB, kWhole>(a, t, i, gs, x);
        return;
    }
    // a block of 256 elements is 32 consecutive lanes, so a half-wave is in or past the end as
    // a whole except where the tensor ends inside its block
    if ((i & ~(int64_t)255) >= t.n) return;
    if (t.flags & kVec) {
        adamw_load<S8, kEdge>(t, i, x);
        adamw_update<S8, UNB, kEdge>(a, t, i, gs, x);
    } else {
        adamw_load<S8, kSingle>(t, i, x);
        adamw_update<S8, UNB, kSingle>(a, t, i, gs, x);
    }
}

nm_status launch_adamw(const nm_adamw_tensor* ts, int count, nm_dtype sdt, double lr, double beta1, double beta2,
                       double eps, int64_t step, const uint64_t* seed, const float* grad_scale, hipStream_t s) {
    AdamWArgs a;
    a.seed = seed ? splitmix64_at(*seed, (uint64_t)step) : 0;
    const double bc1 = 1.0 - pow(beta1, (double)step), bc2 = 1.0 - pow(beta2, (double)step);
    a.grad_scale = grad_scale;
    a.b1 = (float)beta1;
    a.c1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.c2 = (float)(1.0 - beta2);
    a.rbc2 = (float)(1.0 / sqrt(bc2));
    a.eps = (float)eps;
    const bool s8 = sdt == NM_FP8;
    int k = 0;
    int64_t blocks = 0;
    nm_status st = NM_OK;
    adamw_pieces(
        count, kChunk, kMaxTensors, kAdamWMostBlocks, [&](int i) { return ts[i].n; },
        [&](int i, int64_t at, int64_t n, int64_t block) {
            const nm_adamw_tensor& t = ts[i];
            const int64_t ps = t.pdt == NM_BF16 ? 2 : 4, gs = t.gdt == NM_BF16 ? 2 : 4, ss = s8 ? 1 : 4;
            const double l = lr * (double)t.lr_scale;
            AdamWDesc& d = a.t[k];
            d.p = (uint8_t*)t.p + at * ps;
            d.g = (const uint8_t*)t.g + at * gs;
            d.m = (uint8_t*)t.m + at * ss;
            d.v = (uint8_t*)t.v + at * ss;
            d.ms = s8 ? t.m_scale + at / 256 : nullptr;
            d.vs = s8 ? t.v_scale + at / 256 : nullptr;
            d.c = t.copy ? (uint16_t*)t.copy + at : nullptr;
            d.n = n;
            d.alpha = (float)(l / bc1);
            d.decay = (float)(1.0 - l * (double)t.weight_decay);
            const uintptr_t al = (uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.copy |
                                 (s8 ? ((uintptr_t)t.m | (uintptr_t)t.v) << 1 : (uintptr_t)t.m | (uintptr_t)t.v);
            d.flags = (t.pdt == NM_BF16 ? kPBf16 : 0u) | (t.gdt == NM_BF16 ? kGBf16 : 0u) | ((al & 15u) == 0 ? kVec : 0u) |
                      (uint32_t)(at / kChunk) << kFlagBits;   // below 2^29: sizes are below 2^40
            d.tensor = (uint32_t)i;
            a.first[k++] = (uint32_t)block;
            blocks = block + ceil_div(n, kChunk);
        },
        [&]() {
            a.count = k;
            a.first[k] = (uint32_t)blocks;
            const dim3 grid((unsigned)blocks);
            if (s8 && seed) hipLaunchKernelGGL((adamw_kernel<true, true>), grid, dim3(256), 0, s, a);
            else if (s8) hipLaunchKernelGGL((adamw_kernel<true, false>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((adamw_kernel<false, false>), grid, dim3(256), 0, s, a);
            k = 0;
            st = check_launch("nm_adamw");
            return st == NM_OK;
        });
    return st;
}

}  // namespace nm
