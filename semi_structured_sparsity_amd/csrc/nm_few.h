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
// is 64 bytes of codes and 32 of positions: its four lanes load 16 bytes and two words each (one
// instruction for a wave's codes, two for its positions), lane q of the four holding step q, and
// permlane swaps turn that into what each step's instruction wants (lane q holds quarter q of
// every step): four for the codes, five for the positions, where loads in the operands' own order
// would take four times the instructions for the same lines.
// In 4 bits the products of a step or two are summed by the instruction in f32, scaled in f32 (one
// fused multiply-add for each of a lane's four rows) and added up: no value is rounded to fewer bits.
#pragma once

#include <type_traits>

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
    uint32_t voff, ioff;      // the lane's row, in bytes
    uint32_t soff;            // the lane's four output rows
};

// Lanes past the weight's last row re-read it; of the scales those of a run of four rows (the rows
// of scales are long enough for whole runs).
__device__ __forceinline__ FewRows few_rows(const void* vals, const uint32_t* idx, const void* scales, int64_t ldv_bytes,
                                            int64_t ldi, int64_t lds, int64_t r0, int64_t R, int lane) {
    FewRows w;
    w.vals = (const uint8_t*)vals + r0 * ldv_bytes;
    w.idx = idx + r0 * ldi;
    w.scales = (const uint16_t*)scales + r0;
    w.lds = lds;
    const int last = (int)(R - r0 < 16 ? R - r0 - 1 : 15), q = lane >> 4;
    const int row = (lane & 15) < last ? (lane & 15) : last;
    w.voff = (uint32_t)(row * ldv_bytes);
    w.ioff = (uint32_t)(row * ldi * 4);
    w.soff = 4u * (uint32_t)(q < last / 4 ? q : last / 4);
    return w;
}

// A unit (256 columns) of a tile's rows in registers.  SPG: steps that share a scale (1, 2; groups of
// 256 columns load theirs twice a unit).
// Columns past the weight's width meet zeros of X, so that what is loaded for them need only be
// readable and finite: the row's last bytes again.  (Codes always are finite, and a row with a NaN
// scale is NaN already; bf16 values are zeroed.)  No load is behind a branch, so that the compiler
// counts those in flight and waits for none too many.
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
            const int at = u * 64 + q * 16, most = (width / 4 - 1) & ~15;
            const uint4 v = *(const uint4*)(w.vals + (w.voff + (at < most ? at : most)));
            c[0] = v.x;
            c[1] = v.y;
            c[2] = v.z;
            c[3] = v.w;
            const int last = (width - 1) >> gshift;
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int g = (u * 256 + k * SPG * 64) >> gshift;
                const uint2 sv = *(const uint2*)(w.scales + (g < last ? g : last) * w.lds + w.soff);
                s[k][0] = sv.x;
                s[k][1] = sv.y;
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int col = u * 256 + t * 64 + q * 16;
                uint4 v = *(const uint4*)(w.vals + (w.voff + (col < width ? col : width - 16)));
                if (col >= width) v = make_uint4(0, 0, 0, 0);
                c[4 * t] = v.x;
                c[4 * t + 1] = v.y;
                c[4 * t + 2] = v.z;
                c[4 * t + 3] = v.w;
            }
        }
        const uint8_t* ip = (const uint8_t*)w.idx;
        const int word = u * 8 + q * 2, most = (width - 1) / 32;
        i[0] = *(const uint32_t*)(ip + (w.ioff + 4 * (word < most ? word : most)));
        i[1] = *(const uint32_t*)(ip + (w.ioff + 4 * (word + 1 < most ? word + 1 : most)));
    }
    // the loaded words in the operands' order (once, after load)
    __device__ __forceinline__ void order(int lane) {
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

// The division of a window's number by Ns - 1, as a product: exact below 2^29.
struct FewLift {
    int Ns;
    uint32_t magic;   // ceil(2^32 / (Ns - 1))
};
inline FewLift few_lift(int Ns) { return FewLift{Ns, Ns ? (uint32_t)(((1ull << 32) + (uint32_t)Ns - 2) / (uint32_t)(Ns - 1)) : 0u}; }

// 8 (lifted) columns of a token's row of X, from column col of the width: zeros past its end (the load
// itself goes to the row's last columns then, so that no branch is around it).
// A lifted column 4 w + l of window w is original column 2 Ns (w / (Ns - 1)) + 2 (w % (Ns - 1)) + l.
template <bool LIFT>
__device__ __forceinline__ few_u32x4 few_x8(const uint16_t* xrow, int col, int width, const FewLift& f) {
    const int at = col < width ? col : width - 8;
    few_u32x4 r;
    if constexpr (!LIFT) {
        const uint4 v = *(const uint4*)(xrow + at);
        r = few_u32x4{v.x, v.y, v.z, v.w};
    } else {
        // window w starts at 2 Ns g + 2 (w - (Ns - 1) g) = 2 (w + g), g = w / (Ns - 1)
        const uint32_t win = (uint32_t)at >> 2;
        const uint32_t g0 = __umulhi(win, f.magic), g1 = __umulhi(win + 1, f.magic);
        const few_pair a = *(const few_pair*)(xrow + 2 * (win + g0)), b = *(const few_pair*)(xrow + 2 * (win + 1 + g1));
        r = few_u32x4{a.a, a.b, b.a, b.b};
    }
    return col < width ? r : few_u32x4{0, 0, 0, 0};
}

// Where a wave's activation fragments come from; AHEAD: loads in flight that the multiplications wait for.
// FewXDirect: the tokens' rows in memory (16 CT tokens; each load is whole lines of 16 rows).
template <int CT, bool LIFT>
struct FewXDirect {
    static constexpr bool AHEAD = true;
    const uint16_t* row[CT];   // the lane's tokens
    __device__ __forceinline__ few_u32x8 frag(int j, int col, int width, const FewLift& f) const {
        const few_u32x4 lo = few_x8<LIFT>(row[j], col, width, f), hi = few_x8<LIFT>(row[j], col + 32, width, f);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};
// FewXLds: the (lifted) rows of up to 16 tokens in LDS, zeros up to a whole unit.  With one token the
// 64 lanes of a load want 64 bytes of memory, and the address unit still spends the time of 1 KB: from
// LDS they are a broadcast.
struct FewXLds {
    static constexpr bool AHEAD = false;
    const uint8_t* row;        // the lane's token
    __device__ __forceinline__ few_u32x8 frag(int, int col, int, const FewLift&) const {
        const few_u32x4 lo = *(const few_u32x4*)(row + 2 * col), hi = *(const few_u32x4*)(row + 2 * col + 64);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};
// bytes of a token's row in LDS: whole units, and 16 more so that 16 tokens' reads hit distinct banks
__host__ __device__ __forceinline__ int few_lds_row(int width) { return (width + 255) / 256 * 512 + 16; }

// Units u0, u0 + du, ... < nu: acc[i][j] += rows i (16 each) times tokens j (16 each).  cur holds
// unit u0 (loaded by the caller, who may have more to do while it is on its way).
// Loads return in order, so what is waited for first is issued first: a unit's activations (in two
// halves where 16 CT tokens' would take too many registers), then the next unit's weight, then the
// multiplications, which leave the weight in flight.
template <int VT, int SPG, int RT, int CT, typename XF>
__device__ __forceinline__ void few_product(FewUnit<VT, SPG> (&cur)[RT], const FewRows (&w)[RT], const XF& x, int u0, int du, int nu,
                                            int width, int gshift, const FewLift& lift, int lane, few_f32x4 (&acc)[RT][CT]) {
    constexpr int BATCH = CT <= 2 ? 4 : 2;   // steps
    const int q = lane >> 4;
    if (u0 >= nu) return;
    FewUnit<VT, SPG> next[RT];
    auto unit = [&](int u, auto more) __attribute__((always_inline)) {
        few_f32x4 d[RT][CT];
#pragma unroll
        for (int t0 = 0; t0 < 4; t0 += BATCH) {
            few_u32x8 b[BATCH][CT];
#pragma unroll
            for (int t = 0; t < BATCH; ++t)
#pragma unroll
                for (int j = 0; j < CT; ++j) b[t][j] = x.frag(j, u * 256 + (t0 + t) * 64 + q * 8, width, lift);
            if constexpr (decltype(more)::value) {
                if (t0 + BATCH == 4) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) next[i].load(w[i], u + du, width, gshift, lane);
                }
            }
            if constexpr (XF::AHEAD) __builtin_amdgcn_sched_barrier(0);
            if (t0 == 0) {
#pragma unroll
                for (int i = 0; i < RT; ++i) cur[i].order(lane);
            }
#pragma unroll
            for (int t = t0; t < t0 + BATCH; ++t)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const few_bf16x8 a = cur[i].values(t);
#pragma unroll
                    for (int j = 0; j < CT; ++j) {
                        const few_bf16x16 bj = __builtin_bit_cast(few_bf16x16, b[t - t0][j]);
                        if constexpr (VT == kFewBF16) {
                            acc[i][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, bj, acc[i][j], (int)cur[i].i[t], 0, 0);
                        } else {
                            if (t % SPG == 0) d[i][j] = few_f32x4{0, 0, 0, 0};
                            d[i][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, bj, d[i][j], (int)cur[i].i[t], 0, 0);
                            if (t % SPG == SPG - 1) {
                                const uint32_t s0 = cur[i].s[t / SPG][0], s1 = cur[i].s[t / SPG][1];
                                const float s[4] = {__uint_as_float(s0 << 16), __uint_as_float(s0 & 0xffff0000u),
                                                    __uint_as_float(s1 << 16), __uint_as_float(s1 & 0xffff0000u)};
#pragma unroll
                                for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf(s[k], d[i][j][k], acc[i][j][k]);
                            }
                        }
                    }
                }
        }
    };
    int u = u0;
    for (; u + du < nu; u += du) {
        unit(u, std::true_type{});
#pragma unroll
        for (int i = 0; i < RT; ++i) cur[i] = next[i];
    }
    unit(u, std::false_type{});
}

// The tokens' (lifted) rows into LDS, by all NT threads of a block: what few_lds_row lays out.  The
// first two chunks of 16 bytes a thread are loaded here and stored by store(), so that the caller
// can start the weight's loads between the two (loads return in order: behind them these would wait).
template <int NT>
struct FewStage {
    few_u32x4 v[2];
    __device__ __forceinline__ static few_u32x4 chunk(const uint16_t* X, int64_t ldx, int i, int per, int width, const FewLift& lift) {
        const int t = i / per;
        return lift.Ns ? few_x8<true>(X + t * ldx, 8 * (i - t * per), width, lift) : few_x8<false>(X + t * ldx, 8 * (i - t * per), width, lift);
    }
    __device__ __forceinline__ static void put(uint8_t* lds, int i, int per, int stride, const few_u32x4& v) {
        const int t = i / per;
        *(few_u32x4*)(lds + t * stride + 16 * (i - t * per)) = v;
    }
    __device__ __forceinline__ void load(const uint16_t* X, int64_t ldx, int T, int width, const FewLift& lift, uint8_t* lds, int tid) {
        const int per = (width + 255) / 256 * 32, all = T * per, stride = few_lds_row(width);
        for (int i = tid + 2 * NT; i < all; i += NT) put(lds, i, per, stride, chunk(X, ldx, i, per, width, lift));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = tid + k * NT;
            v[k] = chunk(X, ldx, i < all ? i : 0, per, width, lift);
        }
    }
    __device__ __forceinline__ void store(int T, int width, uint8_t* lds, int tid) const {
        const int per = (width + 255) / 256 * 32, all = T * per, stride = few_lds_row(width);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = tid + k * NT;
            if (i < all) put(lds, i, per, stride, v[k]);
        }
    }
};

}  // namespace nm
