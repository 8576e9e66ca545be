// Products of a few tokens with packed 2:4 weights streamed from memory: bf16 values, or 4-bit
// codes with group scales.  Shared by the 4-bit products and the mixture of sparse blocks.
//
// v_smfmac_f32_16x16x64_bf16: the packed weight is the sparse A operand (lane l: row l % 16, 8
// kept values of columns [16 (l / 16), +16) of a 64-column step, their 2-bit positions in the low
// 16 bits of the index operand), 16 tokens are the B operand (lane l: token l % 16, 8 columns from
// 8 (l / 16) and 8 from 32 + 8 (l / 16)); D: token l % 16, rows 4 (l / 16) .. + 3.
//
// The products are bound by the stream of the weight: 1.5 bits a weight in 4 bits, 9 in bf16.  A
// wave takes 16 weight rows and a unit of 256 columns (four steps) at a time.  In 4 bits a row's unit
// is 64 bytes of codes and 32 of positions: its four lanes load 16 and 8 bytes each (one
// instruction for a wave's codes, one for its positions), lane q of the four holding step q, and
// permlane swaps turn that into what each step's instruction wants (lane q holds quarter q of
// every step): four for the codes, five for the positions, where loads in the operands' own order
// would take four times the instructions for the same lines.
#pragma once

#include "nm_internal.h"

namespace nm {

enum { kFewBF16 = 0, kFewI4 = 1, kFewFP4 = 2 };

typedef __bf16 few_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 few_bf16x16 __attribute__((ext_vector_type(16)));
typedef float few_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t few_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t few_u32x8 __attribute__((ext_vector_type(8)));

// 8- and 16-byte loads of 4-byte aligned memory
struct __attribute__((packed, aligned(4))) few_pair {
    uint32_t a, b;
};

// 8 codes -> 8 bf16 values (the value of a code is exact)
template <int VT>
__device__ __forceinline__ few_u32x4 few_decode(uint32_t c) {
    few_u32x4 r;
    if constexpr (VT == kFewFP4) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
    } else {
        // magnitude m with its sign as the e4m3 code s0000mmm stands for m 2^-9: widened by the
        // conversion instruction with the factor 2^9
        const uint32_t lo = ((c & 0x07070707u) | ((c << 4) & ~0x07070707u)) & 0x87878787u;   // values 0, 2, 4, 6
        const uint32_t hi = (((c >> 4) & 0x07070707u) | (c & ~0x07070707u)) & 0x87878787u;   // 1, 3, 5, 7
        const uint32_t p0 = __builtin_amdgcn_perm(hi, lo, 0x05010400u);   // 0, 1, 2, 3
        const uint32_t p1 = __builtin_amdgcn_perm(hi, lo, 0x07030602u);   // 4, 5, 6, 7
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, false));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, true));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, false));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, true));
    }
    return r;
}

__device__ __forceinline__ void few_swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void few_swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

__device__ __forceinline__ float few_act(int act, float g) {
    switch (act) {
        case NM_ACT_SILU: return act_value<NM_ACT_SILU>(g);
        case NM_ACT_GELU: return act_value<NM_ACT_GELU>(g);
        case NM_ACT_GELU_TANH: return act_value<NM_ACT_GELU_TANH>(g);
        default: return act_value<NM_ACT_RELU2>(g);
    }
}

// 16 rows of one packed weight, as a wave sees them
struct FewRows {
    const uint8_t* vals;      // uniform: first row of the tile
    const uint32_t* idx;
    const uint16_t* scales;   // uniform: the tile's first row, group 0
    int64_t lds;
    uint32_t voff, ioff;      // the lane's row and place within it, in bytes
    int last;                 // rows of the tile - 1 (lanes past it re-read its last row)
};

__device__ __forceinline__ FewRows few_rows(const void* vals, const uint32_t* idx, const void* scales, int64_t ldv_bytes,
                                            int64_t ldi, int64_t lds, int64_t r0, int64_t R, int lane) {
    FewRows w;
    w.vals = (const uint8_t*)vals + r0 * ldv_bytes;
    w.idx = idx + r0 * ldi;
    w.scales = (const uint16_t*)scales + r0;
    w.lds = lds;
    w.last = (int)(R - r0 < 16 ? R - r0 - 1 : 15);
    const int row = (lane & 15) < w.last ? (lane & 15) : w.last;
    w.voff = (uint32_t)(row * ldv_bytes);
    w.ioff = (uint32_t)(row * ldi * 4);
    return w;
}

// A unit (256 columns) of a tile's rows in registers.  SPG: steps that share a scale (1, 2, 4).
template <int VT, int SPG>
struct FewUnit {
    static constexpr int NC = VT == kFewBF16 ? 16 : 4, NS = VT == kFewBF16 ? 1 : 4 / SPG;
    uint32_t c[NC];      // codes or values
    uint32_t i[4];       // positions
    uint32_t s[NS][2];   // scales of the lane's four rows
    // u: unit; width: the weight's (lifted) columns; gshift: log2 of the columns a scale serves
    __device__ __forceinline__ void load(const FewRows& w, int u, int width, int gshift, int lane) {
        const int q = lane >> 4;
        if constexpr (VT != kFewBF16) {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int g = (u * 256 + k * SPG * 64) >> gshift;
                if (u * 256 + k * SPG * 64 < width) {
                    const uint16_t* p = w.scales + g * w.lds;
                    if (w.last == 15) {
                        const uint2 v = *(const uint2*)(p + 4 * q);
                        s[k][0] = v.x;
                        s[k][1] = v.y;
                    } else {
                        uint32_t h[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[j] = p[4 * q + j < w.last ? 4 * q + j : w.last];
                        s[k][0] = h[0] | h[1] << 16;
                        s[k][1] = h[2] | h[3] << 16;
                    }
                } else {
                    s[k][0] = s[k][1] = 0;
                }
            }
        }
        if (u * 256 + 256 <= width) {
            const few_pair ip = *(const few_pair*)((const uint8_t*)w.idx + (w.ioff + u * 32 + q * 8));
            i[0] = ip.a;
            i[1] = ip.b;
            if constexpr (VT == kFewBF16) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint4 v = *(const uint4*)(w.vals + (w.voff + u * 256 + t * 64 + q * 16));
                    c[4 * t] = v.x;
                    c[4 * t + 1] = v.y;
                    c[4 * t + 2] = v.z;
                    c[4 * t + 3] = v.w;
                }
            } else {
                const uint4 v = *(const uint4*)(w.vals + (w.voff + u * 64 + q * 16));
                c[0] = v.x;
                c[1] = v.y;
                c[2] = v.z;
                c[3] = v.w;
            }
        } else {
            // the row ends inside this unit, at a multiple of 16 columns: a lane's piece of a step is
            // inside or past the end as a whole, and is loaded by itself
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int col = u * 256 + t * 64 + q * 16;
                const bool in = col < width;
                i[t] = in ? *(const uint16_t*)((const uint8_t*)w.idx + (w.ioff + col / 8)) : 0u;
                if constexpr (VT == kFewBF16) {
                    const uint4 v = in ? *(const uint4*)(w.vals + (w.voff + col)) : make_uint4(0, 0, 0, 0);
                    c[4 * t] = v.x;
                    c[4 * t + 1] = v.y;
                    c[4 * t + 2] = v.z;
                    c[4 * t + 3] = v.w;
                } else {
                    c[t] = in ? *(const uint32_t*)(w.vals + (w.voff + col / 4)) : 0u;
                }
            }
        }
    }
    // the loaded words in the operands' order (once, after load)
    __device__ __forceinline__ void order(int u, int width, int lane) {
        if (u * 256 + 256 > width) return;
        if constexpr (VT != kFewBF16) {
            few_swap32(c[0], c[2]);
            few_swap32(c[1], c[3]);
            few_swap16(c[0], c[1]);
            few_swap16(c[2], c[3]);
        }
        few_swap32(i[0], i[1]);       // i0: steps 0, 1 (both words), i1: steps 2, 3
        uint32_t a = i[0], b = i[0], d = i[1], e = i[1];
        few_swap16(a, b);
        few_swap16(d, e);
        const int half = (lane & 16);   // odd quarters take the upper half of their word
        i[0] = a >> half;
        i[1] = b >> half;
        i[2] = d >> half;
        i[3] = e >> half;
    }
    __device__ __forceinline__ few_bf16x8 values(int t) const {
        if constexpr (VT == kFewBF16)
            return __builtin_bit_cast(few_bf16x8, few_u32x4{c[4 * t], c[4 * t + 1], c[4 * t + 2], c[4 * t + 3]});
        else
            return __builtin_bit_cast(few_bf16x8, few_decode<VT>(c[t]));
    }
};

// 8 (lifted) columns of a token's row of X, from column col of the width: zeros past its end.
// A lifted column 4 w + l of window w is original column 2 Ns (w / (Ns - 1)) + 2 (w % (Ns - 1)) + l.
__device__ __forceinline__ few_u32x4 few_x8(const uint16_t* xrow, int col, int width, int Ns) {
    if (col >= width) return few_u32x4{0, 0, 0, 0};
    if (Ns == 0) {
        const uint4 v = *(const uint4*)(xrow + col);
        return few_u32x4{v.x, v.y, v.z, v.w};
    }
    const uint32_t win = (uint32_t)col >> 2, d = (uint32_t)(Ns - 1);
    const uint32_t g0 = win / d, r0 = win - g0 * d, g1 = (win + 1) / d, r1 = win + 1 - g1 * d;
    const few_pair a = *(const few_pair*)(xrow + 2 * (Ns * g0 + r0)), b = *(const few_pair*)(xrow + 2 * (Ns * g1 + r1));
    return few_u32x4{a.a, a.b, b.a, b.b};
}

// acc[i][j] += rows i (16 each) times tokens j (16 each), over units u0, u0 + du, ... < nu.
template <int VT, int SPG, int RT, int CT>
__device__ __forceinline__ void few_product(const FewRows (&w)[RT], const uint16_t* const (&xrow)[CT], int u0, int du, int nu,
                                            int width, int gshift, int Ns, int lane, few_f32x4 (&acc)[RT][CT]) {
    const int q = lane >> 4;
    FewUnit<VT, SPG> cur[RT];
    if (u0 < nu) {
#pragma unroll
        for (int i = 0; i < RT; ++i) cur[i].load(w[i], u0, width, gshift, lane);
    }
    for (int u = u0; u < nu; u += du) {
        few_u32x8 x[4][CT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int col = u * 256 + t * 64 + q * 8;
                const few_u32x4 lo = few_x8(xrow[j], col, width, Ns), hi = few_x8(xrow[j], col + 32, width, Ns);
                x[t][j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        FewUnit<VT, SPG> next[RT];
        if (u + du < nu) {
#pragma unroll
            for (int i = 0; i < RT; ++i) next[i].load(w[i], u + du, width, gshift, lane);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            cur[i].order(u, width, lane);
            few_f32x4 d[CT];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const few_bf16x8 a = cur[i].values(t);
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    if constexpr (VT == kFewBF16) {
                        acc[i][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, __builtin_bit_cast(few_bf16x16, x[t][j]),
                                                                              acc[i][j], (int)cur[i].i[t], 0, 0);
                    } else {
                        if (t % SPG == 0) d[j] = few_f32x4{0, 0, 0, 0};
                        d[j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, __builtin_bit_cast(few_bf16x16, x[t][j]), d[j],
                                                                         (int)cur[i].i[t], 0, 0);
                        if (t % SPG == SPG - 1) {
                            const uint32_t s0 = cur[i].s[t / SPG][0], s1 = cur[i].s[t / SPG][1];
                            const float s[4] = {__uint_as_float(s0 << 16), __uint_as_float(s0 & 0xffff0000u),
                                                __uint_as_float(s1 << 16), __uint_as_float(s1 & 0xffff0000u)};
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf(s[k], d[j][k], acc[i][j][k]);
                        }
                    }
                }
            }
        }
        if (u + du < nu) {
#pragma unroll
            for (int i = 0; i < RT; ++i) cur[i] = next[i];
        }
    }
}

}  // namespace nm
