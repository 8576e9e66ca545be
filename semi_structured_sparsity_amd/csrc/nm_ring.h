// Device pieces shared by the ring kernels of the products (k_spmm.hip) and of the gradients
// (k_grad.hip): operand types and matrix instructions, DMA loads into LDS, counted waits, tile
// order, tile stores.
#pragma once

#include "nm_internal.h"

namespace nm {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16_t __attribute__((ext_vector_type(16)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// OCP FP8 e4m3 code: one byte, multiplied by v_smfmac_f32_32x32x64_fp8_fp8 with the
// int8 instruction's operand layout and f32 accumulation.
struct fp8e4m3 {
    uint8_t v;
};

// Accumulator types and the sparse instruction of each operand type.  A is the
// lane's 16 bytes of compressed values, B its 32 bytes of the dense operand, idx
// its index bits (bf16: the lane's 16-bit half already selected).
template <typename T>
struct Mma {   // bf16
    using Acc = f32x16_t;
    using AccS = float;
    __device__ static Acc run(i32x4_t a, i32x8_t b, Acc c, int idx) {
        return __builtin_amdgcn_smfmac_f32_32x32x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                         __builtin_bit_cast(bf16x16_t, b), c, idx, 0, 0);
    }
};
template <>
struct Mma<int8_t> {
    using Acc = i32x16_t;
    using AccS = int32_t;
    __device__ static Acc run(i32x4_t a, i32x8_t b, Acc c, int idx) {
        return __builtin_amdgcn_smfmac_i32_32x32x64_i8(a, b, c, idx, 0, 0);
    }
};
template <>
struct Mma<fp8e4m3> {
    using Acc = f32x16_t;
    using AccS = float;
    __device__ static Acc run(i32x4_t a, i32x8_t b, Acc c, int idx) {
        return __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(a, b, c, idx, 0, 0);
    }
};

struct SpmmArgs {
    const uint8_t* X;      // [Mtok, ldx] elements of T
    const uint8_t* vals;   // [R, ldv] elements of T
    const uint32_t* idx;   // [R, ldi] words
    const float* x_scale;  // [Mtok] or null
    void* Y;               // [Mtok, ldy] of ydt
    void* part;            // split-K partials [KS][Mtok][R] (f32 or i32) or null
    int64_t ldx, ldv, ldi, ldy;
    int64_t Mtok, K, R;
    int64_t comp_bytes;    // packed value bytes per row (K'/2 * sizeof(T))
    int64_t idx_words;     // index words per row (ceil(K'/32): two 2-bit fields per 4 lifted columns)
    int64_t xrow_bytes;    // bytes of one row of the original (unlifted) X, for the in-kernel lift
    float w_scale;
    int scaled;
    int ydt;
    int nsteps, KS, steps_per_split;
    int tiles_r, tiles_t;
    int tile_rows;         // K-split ring: weight rows per row tile (0: the tile's height)
    // rank-r adapter term added to the accumulators (bf16 products only; rank 0: none):
    // u [Mtok, rank] (ldu) and the stacked up-projection B [R, rank] (ldb), both bf16
    const uint16_t* lr_u;
    const uint16_t* lr_b;
    int64_t ldu, ldb;
    int rank;
    // Hutchinson modes of the dense split ring: probes, their seed, stages per probe, rows
    // per probe
    uint64_t seed;
    int probes, pstages;
    int64_t prows;
    // score epilogue of the Hutchinson second product: W [rows of D, K] bf16 (ldw), eps, and
    // the per-block moments of the scores ([count | mean | m2][blocks])
    const uint16_t* sw;
    int64_t ldsw;
    float eps;
    double* mpart;
    // gated block (GLU): vals / idx / w_scale are the gate's and vals2 / idx2 / w_scale2 the up
    // projection's, R features each; Y is H, Y2 and Y3 the rounded G and U (ldy2) or null
    const uint8_t* vals2;
    const uint32_t* idx2;
    float w_scale2;
    int act;
    void *Y2, *Y3;
    int64_t ldy2;
};

// Block index -> (R tile, token tile).  Workgroups are dispatched round-robin
// over the 8 XCDs; the remap gives each XCD a contiguous range of tiles, and
// the range is walked in groups of 8 R tiles so that the blocks resident on one
// XCD at a time share their weight and activation tiles in that XCD's L2.
__device__ __forceinline__ void tile_of(int bid, int nb, int tiles_r, int tiles_t, int& tr, int& tt) {
    const int xcd = bid & 7, loc = bid >> 3;
    const int base = nb >> 3, rem = nb & 7;
    const int id = xcd * base + (xcd < rem ? xcd : rem) + loc;
    const int GR = 8;
    const int per_group = GR * tiles_t;
    const int grp = id / per_group;
    const int first = grp * GR;
    const int gsz = (tiles_r - first) < GR ? (tiles_r - first) : GR;
    const int in = id - grp * per_group;
    tr = first + in % gsz;
    tt = in / gsz;
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const lds_u8*)p;
}
__device__ __forceinline__ void dma16(uint32_t lds, const void* g) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
// A block-uniform pointer, moved to scalar registers.
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const void*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}
// saddr form: uniform 64-bit base in SGPRs + per-lane 32-bit byte offset
__device__ __forceinline__ void dma16s(uint32_t lds, const void* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4s(uint32_t lds, const void* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(uint32_t lds, const void* g) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
// Wait until at most N vector-memory loads of this wave are in flight and all its LDS
// reads are done, then meet the other waves.  The wait is a compiler builtin, so the
// compiler's own wait-count bookkeeping knows that every earlier LDS read has completed;
// the barrier is an opaque statement that no memory access moves across.
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit field");
    __builtin_amdgcn_sched_barrier(0);  // SMFMACs written after the barrier stay after it
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) expcnt(7) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_vm_all() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Index words are read from LDS one dword per lane.  Such a read is served a half-wave
// (32 lanes) at a time over 32 dword banks (measured with an LDS probe and the bank-conflict
// counter), and the 32 lanes of a half-wave read one word from each of 32 consecutive rows.
// A row of W index words (W a power of two, at most 32) therefore keeps logical word w at
// w ^ iswz<W>(r), r counted from a multiple of 32: the 32 reads then hit 32 distinct banks.
// Rows padded to a whole number of 16-byte pieces and swizzled by piece instead reach only
// 8 banks (a 4-way conflict, 4x the read time).
template <int W>
__device__ __forceinline__ int iswz(int r) {
    static_assert(W >= 1 && W <= 32 && (W & (W - 1)) == 0, "W a power of two up to 32");
    return (r / (32 / W)) & (W - 1);
}

// Words of the wave-private LDS buffer store_tile needs: SR sub-tiles x 64 lanes x 16
// accumulators, each lane's 16 padded to 20 words (16-byte pieces of 16 consecutive lanes
// then fall on distinct banks).
template <int SR>
constexpr int kStageWords = SR * 64 * 20;

// Stores a wave's SR x ST accumulator tiles (rows from rw, tokens from tw).  A lane
// holds token column l32 and rows 8*(e/4) + 4*h + e%4 of each 32x32 sub-tile.
// bf16 tiles fully inside Y (inside) with 8-byte aligned rows are stored straight from
// the accumulators, four consecutive rows per 8-byte store (measured as fast as staging
// for them).  Everything else goes through a wave-private LDS buffer of kStageWords<SR>
// words (stage, 16-byte aligned), since 4-byte outputs stored straight would scatter
// every instruction over 32 token rows of Y: each 32-token column of sub-tiles is written
// to LDS as whole accumulator vectors (stores of single extracted elements have been
// miscompiled), read back as 4-row runs of one token (a lane's elements 4q..4q+3 are 4
// consecutive rows), and stored as whole runs of Y's rows (32 lanes per token, 4
// outputs per lane), scaled and converted on the way.  The caller has finished every
// other use of the buffer.
template <typename T, int SR, int ST>
__device__ __forceinline__ void store_tile(const SpmmArgs& a, const typename Mma<T>::Acc (&acc)[SR][ST], int64_t rw,
                                           int64_t tw, bool inside, uint32_t* stage, int lane) {
    using AccV = typename Mma<T>::Acc;
    using AccS = typename Mma<T>::AccS;
    static_assert(SR == 4, "one token row of the wave's tile (4 sub-tiles) per half-wave");
    const int h = lane >> 5, l32 = lane & 31;
    if (inside && a.ydt == NM_BF16 && ((uintptr_t)a.Y % 8) == 0 && (a.ldy % 4) == 0) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
            const int64_t tok = tw + j * 32 + l32;
            const float sc = a.scaled ? __fmul_rn(a.w_scale, a.x_scale ? a.x_scale[tok] : 1.0f) : 1.0f;
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                uint16_t* yrow = (uint16_t*)a.Y + tok * a.ldy + rw + i * 32 + 4 * h;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[e] = (float)acc[i][j][4 * g + e];
                        if (a.scaled) f[e] = __fmul_rn(sc, f[e]);
                    }
                    *(uint2*)(yrow + 8 * g) = make_uint2(f32_to_bf16_bits(f[0]) | (f32_to_bf16_bits(f[1]) << 16),
                                                         f32_to_bf16_bits(f[2]) | (f32_to_bf16_bits(f[3]) << 16));
                }
            }
        }
        return;
    }
    const int es = a.ydt == NM_BF16 ? 2 : 4;
    // 16-byte (4-byte outputs) or 8-byte (bf16) vector stores need aligned rows of Y
    const bool vec = ((uintptr_t)a.Y % (4 * es)) == 0 && (a.ldy * es) % (4 * es) == 0;
    // reader: lane l32 of a half-wave takes rows 4*l32 .. 4*l32+3 of the wave's 128, which
    // are elements 4q .. 4q+3 of lane (token + 32 h') in sub-tile i
    const int ri = l32 >> 3, rq = (l32 & 7) >> 1, rh = l32 & 1;
#pragma unroll
    for (int j = 0; j < ST; ++j) {
#pragma unroll
        for (int i = 0; i < SR; ++i) *(AccV*)&stage[(i * 64 + lane) * 20] = acc[i][j];
        // lgkmcnt(0): this wave's LDS writes are done before any lane reads another's
        __builtin_amdgcn_s_waitcnt(0xc07f);
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
#pragma unroll 4
        for (int p = 0; p < 16; ++p) {
            const int tk = 2 * p + h;   // lanes 0-31 and 32-63 take two tokens per pass
            const int64_t tok = tw + j * 32 + tk;
            const uint4 raw = *(const uint4*)&stage[(ri * 64 + tk + 32 * rh) * 20 + 4 * rq];
            const int64_t r = rw + 4 * l32;
            if (tok >= a.Mtok || r >= a.R) continue;
            const AccS v[4] = {__builtin_bit_cast(AccS, raw.x), __builtin_bit_cast(AccS, raw.y),
                               __builtin_bit_cast(AccS, raw.z), __builtin_bit_cast(AccS, raw.w)};
            const int64_t o = tok * a.ldy + r;
            const bool full = vec && r + 3 < a.R;
            if (a.ydt == NM_I32) {
                if (full) {
                    *(uint4*)((int32_t*)a.Y + o) = raw;
                } else {
                    for (int e = 0; e < 4 && r + e < a.R; ++e) ((int32_t*)a.Y)[o + e] = (int32_t)v[e];
                }
                continue;
            }
            float f[4];
            if (a.scaled) {
                const float sc = __fmul_rn(a.w_scale, a.x_scale ? a.x_scale[tok] : 1.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = __fmul_rn(sc, (float)v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = (float)v[e];
            }
            if (a.ydt == NM_F32) {
                if (full) {
                    *(float4*)((float*)a.Y + o) = make_float4(f[0], f[1], f[2], f[3]);
                } else {
                    for (int e = 0; e < 4 && r + e < a.R; ++e) ((float*)a.Y)[o + e] = f[e];
                }
            } else {
                if (full) {
                    *(uint2*)((uint16_t*)a.Y + o) = make_uint2(f32_to_bf16_bits(f[0]) | (f32_to_bf16_bits(f[1]) << 16),
                                                               f32_to_bf16_bits(f[2]) | (f32_to_bf16_bits(f[3]) << 16));
                } else {
                    for (int e = 0; e < 4 && r + e < a.R; ++e) ((uint16_t*)a.Y)[o + e] = (uint16_t)f32_to_bf16_bits(f[e]);
                }
            }
        }
        // the next column of sub-tiles overwrites the buffer only after every lane has read it
        __builtin_amdgcn_s_waitcnt(0xc07f);
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
    }
}

// Compute units of the current device (cached per device).
inline int64_t device_cus() {
    static int64_t cache[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cache[dev] == 0) {
        int n = 0;
        cache[dev] = (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && n > 0) ? n : 256;
    }
    return cache[dev];
}

}  // namespace nm
