// Gradients of the sparse layer and of the gated feed-forward block (bf16, 2:4 and lifted (2N-2):2N).
//
// For y = x W^T with W [R, K] packed 2:4, and for a gated block with pre-activations
// G = x Wg^T, U = x Wu^T, H = act(G) . U:
//   dG = dH . U . act'(G),  dU = dH . act(G)
//   dX = dY W               (gated: dG Wg + dU Wu)
//   dV[r, j] = sum_m dY[m, r] X[m, col(r, j)]   for the kept positions col(r, j) only.
// A (2N-2):2N weight is a plain 2:4 one over the lifted width K' (lifted column 4 w + j of window
// w reads column orig of X): dV reads X's rows by that map, dX' is formed over K' and folded, each
// column's lifted ones (two at most) added in f32, except where dX has a dense copy of the weights
// to read, which is made over K.
// Neither product can use the sparse instructions: they skip zeros of the operand along the
// summed dimension, W is 2:4 along K, but dX sums over R and dV over the tokens.  Both run as
// dense products on 256 x 256 tiles (grad_ring_kernel), bound by the matrix
// cores and the operand stream; dV's epilogue keeps the packed positions of each tile, so the
// dense gradient never exists.
// The ring wants both operands with the summed dimension contiguous, so the operands
// are laid out once, in the workspace, by the bandwidth-bound kernels below:
//   D  [M, nmat * Rp]  dY, or dG | dU, the rows padded to Rp = a multiple of 64 with zeros,
//   DT [nmat * Rp, Mp] its transpose, the tokens padded to Mp = a multiple of 64 with zeros,
//   XT [K, Mp]         X transposed,
//   WT [K, nmat * Rp]  the packed weights, dense and transposed (many tokens; fewer decode them
//                      in the product, ring_decodes).
#include "nm_ring.h"

namespace nm {

// ------------------------------------------------------------------ layouts
// The operands' layouts, in one launch whose blocks take 64 x 64 tiles of dY (or of dH, G and
// U), 64 x 64 tiles of X and 64 x 128 tiles of the packed weights.  A thread holds two rows of its
// tile (2 p and 2 p + 1); transposed tiles go through LDS as row-pair words t[column][pair]
// with 33 words a column, the pairs of columns 64-127 swapped in eights, so that the 64
// lanes of a write fall on distinct banks.
struct PairTile {
    uint32_t t[128][33];
    __device__ static int at(int col, int pair) { return pair ^ (((col >> 6) & 1) * 8); }
    __device__ __forceinline__ void put(int col, int pair, uint32_t w) { t[col][at(col, pair)] = w; }
    // rows 8 q .. 8 q + 7 of a column, 16 bytes
    __device__ __forceinline__ uint4 get(int col, int q) const {
        const uint32_t* w = &t[col][at(col, 4 * q)];
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// 8 bf16 of a row from column c; zero past cols (or if !ok).  VEC: bytes of a load (16, or 4 where
// rows are only even, else 2)
template <int VEC>
__device__ __forceinline__ void load_row8(const uint16_t* __restrict__ row, int64_t c, int64_t cols, bool ok,
                                          uint32_t (&x)[8]) {
    if (VEC > 2 && ok && c + 8 <= cols) {
        uint32_t w[4];
        if constexpr (VEC == 16) {
            const uint4 u = *(const uint4*)(row + c);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ((const uint32_t*)(row + c))[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = w[e] & 0xffffu;
            x[2 * e + 1] = w[e] >> 16;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ok && c + e < cols ? row[c + e] : 0u;
}
__device__ __forceinline__ uint4 pack8(const uint32_t (&x)[8]) {
    return make_uint4(x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16));
}

// Decoding a group of 4 columns: its two values are one word, and its 4 bits of positions select
// from a table the byte selectors that spread them over the columns' two words (v_perm_b32:
// selectors 0-3 take a byte, 12 gives zero).  The table is 16 entries of 8 bytes in LDS, one bank
// pair each.
struct SpreadTable {
    uint2 sel[16];
    // by the first 16 threads of a block, before a barrier
    __device__ void fill(int tid) {
        if (tid >= 16) return;
        const uint32_t p0 = tid & 3u, p1 = tid >> 2;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            w[e >> 1] |= (p0 == e ? 0x0100u : p1 == e ? 0x0302u : 0x0c0cu) << (16 * (e & 1));
        sel[tid] = make_uint2(w[0], w[1]);
    }
};
// 16 columns of two packed rows (8 values and 16 bits of positions each) as the columns' row
// pairs: x[e] = row 0's column e | row 1's column e << 16
__device__ __forceinline__ void decode_pair16(const SpreadTable& t, uint4 v0, uint32_t b0, uint4 v1, uint32_t b1,
                                              uint32_t (&x)[16]) {
    const uint32_t a[4] = {v0.x, v0.y, v0.z, v0.w}, c[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint2 sa = t.sel[(b0 >> (4 * q)) & 15u], sc = t.sel[(b1 >> (4 * q)) & 15u];
        const uint32_t a0 = __builtin_amdgcn_perm(0, a[q], sa.x), a1 = __builtin_amdgcn_perm(0, a[q], sa.y);
        const uint32_t c0 = __builtin_amdgcn_perm(0, c[q], sc.x), c1 = __builtin_amdgcn_perm(0, c[q], sc.y);
        x[4 * q + 0] = __builtin_amdgcn_perm(c0, a0, 0x05040100u);
        x[4 * q + 1] = __builtin_amdgcn_perm(c0, a0, 0x07060302u);
        x[4 * q + 2] = __builtin_amdgcn_perm(c1, a1, 0x05040100u);
        x[4 * q + 3] = __builtin_amdgcn_perm(c1, a1, 0x07060302u);
    }
}

// Column of X under lifted column k of a (2 Ns - 2):2 Ns weight (Ns 0: itself).  From a window's
// first column on, the columns below never come before it.
__device__ __forceinline__ int64_t orig_col(int64_t k, int Ns) {
    if (Ns == 0) return k;
    const uint32_t w = (uint32_t)(k >> 2), n = (uint32_t)Ns - 1, g = w / n;   // below 2^20
    return (int64_t)(2 * (n + 1) * g + 2 * (w - g * n)) + (k & 3);
}

// Groups of a lifted weight in a tile of its dense copy: the most whose windows fit 128 lifted
// columns and end at a multiple of 16.
__host__ __device__ inline int lifted_tile_groups(int Ns) { return (32 / (Ns - 1)) & ~3; }
// Lifted columns over column p of a group: window w's is 4 w + p - 2 w, for first <= w <= last.
__device__ __forceinline__ int first_window(int p) { return p > 3 ? (p - 2) / 2 : 0; }
__device__ __forceinline__ int last_window(int p, int Ns) { return p / 2 < Ns - 2 ? p / 2 : Ns - 2; }

struct LayoutArgs {
    GradIn in;
    int64_t Rp, Mp, Rn;
    uint16_t *D, *DT, *XT, *WT;   // null: not needed
    int nd, nw, nx;               // blocks of the dY tiles, of the weights, of X
    int td, tw, tx;               // tiles along a row of each
};

// S [rows, cols] (lds), tile (ti, tj) -> T [cols, rowsp] and the copy C (ldc), both zero past the
// edges
template <int VEC>
__device__ __forceinline__ void transpose_tile(PairTile& tile, const uint16_t* __restrict__ S, int64_t lds, int64_t rows,
                                               int64_t cols, uint16_t* __restrict__ T, int64_t rowsp,
                                               uint16_t* __restrict__ C, int64_t ldc, int ti, int tj) {
    const int tid = threadIdx.x, c8 = tid & 7, pair = tid >> 3;
    const int64_t r0 = (int64_t)ti * 64, c0 = (int64_t)tj * 64;
    const int64_t r = r0 + 2 * pair, c = c0 + 8 * c8;
    uint32_t x[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load_row8<VEC>(S + (r + k) * lds, c, cols, r + k < rows, x[k]);
    if (C) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (r + k < rows) *(uint4*)(C + (r + k) * ldc + c) = pack8(x[k]);
    }
    if (!T) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) tile.put(c8 * 8 + e, pair, x[0][e] | (x[1][e] << 16));
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int col = (tid >> 3) + 32 * p, q = tid & 7;
        if (c0 + col < cols) *(uint4*)(T + (c0 + col) * rowsp + r0 + 8 * q) = tile.get(col, q);
    }
}

// dG | dU from dH, G, U: rows of D [M, 2 Rp] and of DT [2 Rp, Mp], padded with zeros.  They are
// rounded to bf16 here: operands of the bf16 matrix products, as the forward's activations are.
template <int ACT, int VEC>
__device__ __forceinline__ void glu_grad_tile(PairTile& tile, const LayoutArgs& a, int ti, int tj) {
    const GradIn& in = a.in;
    const int tid = threadIdx.x, c8 = tid & 7, pair = tid >> 3;
    const int64_t m0 = (int64_t)ti * 64, c0 = (int64_t)tj * 64;
    const int64_t m = m0 + 2 * pair, c = c0 + 8 * c8;
    uint32_t dg[2][8], du[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const bool ok = m + k < in.M;
        uint32_t h[8], g[8], u[8];
        load_row8<VEC>(in.dY + (m + k) * in.lddy, c, in.R, ok, h);
        load_row8<VEC>(in.G + (m + k) * in.ldg, c, in.R, ok, g);
        load_row8<VEC>(in.U + (m + k) * in.ldg, c, in.R, ok, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float hf = bf16_bits_to_f32(h[e]), gf = bf16_bits_to_f32(g[e]), uf = bf16_bits_to_f32(u[e]);
            float f, d;
            act_and_grad<ACT>(gf, f, d);
            const uint32_t both = f32_to_bf16_pair(hf * uf * d, hf * f);
            dg[k][e] = both & 0xffffu;
            du[k][e] = both >> 16;
        }
        if (a.D && ok) {
            *(uint4*)(a.D + (m + k) * a.Rn + c) = pack8(dg[k]);
            *(uint4*)(a.D + (m + k) * a.Rn + a.Rp + c) = pack8(du[k]);
        }
    }
    if (!a.DT) return;
    // columns 0-63 of the tile: dG, 64-127: dU
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        tile.put(c8 * 8 + e, pair, dg[0][e] | (dg[1][e] << 16));
        tile.put(64 + c8 * 8 + e, pair, du[0][e] | (du[1][e] << 16));
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int col = (tid >> 3) + 32 * p, q = tid & 7;
        *(uint4*)(a.DT + ((int64_t)(p >> 1) * a.Rp + c0 + (col & 63)) * a.Mp + m0 + 8 * q) = tile.get(col, q);
    }
}

// 64 rows x 128 columns of a packed 2:4 weight (a line of values per row) -> WT [K, Rn] at columns
// off + r (rows past R: zero).  Thread (c, pair): rows 2 pair, 2 pair + 1, columns 16 c ..: 8
// values and 16 bits of positions per row; K is a multiple of 16.
// A lifted weight's copy has the original columns (a quarter fewer at N = 3, three sevenths at N = 8): a tile holds whole
// groups, and a column under two windows is their sum, rounded to bf16 (exact where one of them is
// zero, as in any decomposed weight).
__device__ __forceinline__ void decode_tile(PairTile& tile, SpreadTable& table, const LayoutArgs& a, int mat, int ti, int tj) {
    const GradIn& in = a.in;
    const int tid = threadIdx.x, c = tid & 7, pair = tid >> 3;
    const int Ns = in.Ns, groups = Ns ? lifted_tile_groups(Ns) : 0, width = Ns ? groups * 4 * (Ns - 1) : 128;
    const int64_t r0 = (int64_t)ti * 64, k0 = (int64_t)tj * width, k = k0 + 16 * c;
    table.fill(tid);
    __syncthreads();
    uint4 v[2];
    uint32_t b[2], x[16];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t r = r0 + 2 * pair + j;
        const bool ok = r < in.R && k < in.Kl && 16 * c < width;
        v[j] = ok ? *(const uint4*)(in.vals[mat] + r * in.ldv + k / 2) : make_uint4(0, 0, 0, 0);
        b[j] = ok ? in.idx[mat][r * in.ldi + k / 32] >> (k & 16) : 0u;
    }
    decode_pair16(table, v[0], b[0], v[1], b[1], x);
#pragma unroll
    for (int e = 0; e < 16; ++e) tile.put(c * 16 + e, pair, x[e]);
    __syncthreads();
    if (Ns) {
        const int span = groups * 2 * Ns, q = tid & 7;
        const int64_t o0 = (int64_t)tj * span;
        for (int col = tid >> 3; col < span && o0 + col < in.K; col += 32) {
            const int g = col / (2 * Ns), p = col - g * 2 * Ns, w0 = first_window(p), w1 = last_window(p, Ns);
            const int l0 = 4 * (g * (Ns - 1) + w0) + p - 2 * w0;
            uint4 u = tile.get(l0, q);
            if (w1 > w0) {   // the next window's column is two on
                const uint4 v = tile.get(l0 + 2, q);
                auto add = [](uint32_t a, uint32_t b) {
                    return f32_to_bf16_pair(bf16_bits_to_f32(a & 0xffffu) + bf16_bits_to_f32(b & 0xffffu),
                                            bf16_bits_to_f32(a >> 16) + bf16_bits_to_f32(b >> 16));
                };
                u = make_uint4(add(u.x, v.x), add(u.y, v.y), add(u.z, v.z), add(u.w, v.w));
            }
            *(uint4*)(a.WT + (o0 + col) * a.Rn + mat * a.Rp + r0 + 8 * q) = u;
        }
        return;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int col = (tid >> 3) + 32 * p, q = tid & 7;
        if (k0 + col < in.Kl) *(uint4*)(a.WT + (k0 + col) * a.Rn + mat * a.Rp + r0 + 8 * q) = tile.get(col, q);
    }
}

// ACT: the gated block's activation, or -1: dY itself
template <int ACT, int VEC>
__global__ __launch_bounds__(256) void grad_layout_kernel(LayoutArgs a) {
    __shared__ PairTile tile;
    __shared__ SpreadTable table;
    int b = blockIdx.x;
    if (b < a.nw) {
        const int mat = b / (a.nw / (ACT >= 0 ? 2 : 1));
        b -= mat * (a.nw / 2);
        decode_tile(tile, table, a, mat, b / a.tw, b % a.tw);
    } else if (b < a.nw + a.nd) {
        b -= a.nw;
        if constexpr (ACT >= 0) glu_grad_tile<ACT, VEC>(tile, a, b / a.td, b % a.td);
        else transpose_tile<VEC>(tile, a.in.dY, a.in.lddy, a.in.M, a.in.R, a.DT, a.Mp, a.D, a.Rn, b / a.td, b % a.td);
    } else {
        b -= a.nw + a.nd;
        transpose_tile<16>(tile, a.in.X, a.in.ldx, a.in.M, a.in.K, a.XT, a.Mp, (uint16_t*)nullptr, 0, b / a.tx, b % a.tx);
    }
}

// ------------------------------------------------------------------ products
// One of the two products of a backward call: C^T tiles of 256 A rows x 256 B rows, summed over
// nsteps stages of 64 columns.
struct GradJob {
    const uint16_t *A, *B;
    int64_t lda, ldb, rowsA, rowsB;
    int nsteps, spp;          // stages, stages per split
    int tiles_a, tiles_b;     // tiles of a split
};
struct GradArgs {
    GradJob x, v;             // dX: A = WT (columns k), B = D (tokens); dV: A = XT (k), B = DT (rows r)
    int nx;                   // blocks of dX (tiles * splits), the first of the grid
    // dX
    void* dX;
    float* part;              // partials [split][M][K'] (splits, or a lifted weight), or null
    int64_t lddx;
    int dxf32;
    // dV
    const uint32_t* idx[2];
    void* dV[2];
    int64_t ldi, lddv, R, Rp;
    int dvf32, Ns;
    float* vpart;             // partials of the packed dV [split][weight][R][K'/2] where its tokens are split, or null
    // dX from the packed weights (DEC)
    const uint16_t* vals[2];
    int64_t ldv;
};

// Gradient of packed 2:4 values: of the tile's columns k (rows rw .. of the accumulators) of
// weight row r (the lane's token, from tw) only the kept positions are stored.  Elements
// 4g .. 4g+3 of a lane's sub-tile are columns 32 i + 8 g + 4 h .. + 3, one group of 4, whose
// two 2-bit positions are bits 4 (2 g + h) .. of the row's index word of those 32 columns.  A
// lane's 8 kept values alternate in pairs with the other half-wave's; two swaps across the
// halves leave each lane with the 8 consecutive values of 16 columns (K is a multiple of 16,
// so all of them exist or none).
// The positions are loaded before the products (grad_positions), so that no load is waited for here.
template <int SR, int ST>
__device__ __forceinline__ void grad_positions(const GradArgs& a, int64_t rw, int64_t tw, int lane, uint32_t (&word)[ST][SR]) {
#pragma unroll
    for (int j = 0; j < ST; ++j) {
        const int64_t q = tw + j * 32 + (lane & 31);   // stacked row
        const int mat = q >= a.Rp ? 1 : 0;
        const int64_t r = q - mat * a.Rp;
        const bool row_ok = q < a.v.rowsB && r < a.R;
        const uint32_t* irow = (mat ? a.idx[1] : a.idx[0]) + (row_ok ? r : 0) * a.ldi;
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            const int64_t k = rw + i * 32;
            word[j][i] = row_ok && k < a.v.rowsA ? irow[k >> 5] : 0u;
        }
    }
}
template <int SR, int ST>
__device__ __forceinline__ void store_grad_tile(const GradArgs& a, const f32x16_t (&acc)[SR][ST],
                                                const uint32_t (&words)[ST][SR], int64_t rw, int64_t tw, int lane) {
    const int64_t K = a.v.rowsA;
    const int h = lane >> 5, l32 = lane & 31;
#pragma unroll
    for (int j = 0; j < ST; ++j) {
        const int64_t q = tw + j * 32 + l32;   // stacked row
        const int mat = q >= a.Rp ? 1 : 0;
        const int64_t r = q - mat * a.Rp;
        const bool row_ok = q < a.v.rowsB && r < a.R;
        uint8_t* orow = (uint8_t*)(mat ? a.dV[1] : a.dV[0]);
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            const int64_t k = rw + i * 32;
            const uint32_t word = words[j][i];
            float v0[4], v1[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t b = (word >> (8 * g + 4 * h)) & 15u, p0 = b & 3u, p1 = b >> 2;
                const float x0 = acc[i][j][4 * g], x1 = acc[i][j][4 * g + 1], x2 = acc[i][j][4 * g + 2],
                            x3 = acc[i][j][4 * g + 3];
                const float lo0 = p0 & 1u ? x1 : x0, hi0 = p0 & 1u ? x3 : x2;
                const float lo1 = p1 & 1u ? x1 : x0, hi1 = p1 & 1u ? x3 : x2;
                v0[g] = p0 & 2u ? hi0 : lo0;
                v1[g] = p1 & 2u ? hi1 : lo1;
            }
            // lane half h: values of columns k + 16 h .. + 15
            const int64_t kc = k + 16 * h;
            const bool ok = row_ok && kc < K;
            const int64_t o = r * a.lddv + kc / 2;
            if (!a.dvf32) {
                uint32_t w[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) w[g] = f32_to_bf16_pair(v0[g], v1[g]);
                const auto s0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                if (ok) *(uint4*)((uint16_t*)orow + o) = make_uint4(s0[0], s0[1], s1[0], s1[1]);
            } else {
                uint32_t a0[4], a1[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) a0[g] = __float_as_uint(v0[g]), a1[g] = __float_as_uint(v1[g]);
                const auto s0 = __builtin_amdgcn_permlane32_swap(a0[0], a0[2], false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(a1[0], a1[2], false, false);
                const auto s2 = __builtin_amdgcn_permlane32_swap(a0[1], a0[3], false, false);
                const auto s3 = __builtin_amdgcn_permlane32_swap(a1[1], a1[3], false, false);
                if (ok) {
                    *(uint4*)((float*)orow + o) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
                    *(uint4*)((float*)orow + o + 4) = make_uint4(s2[0], s3[0], s2[1], s3[1]);
                }
            }
        }
    }
}

// Both products in one grid, dX's blocks first: a dX tile sums over all rows of the weights and a
// dV tile over all tokens, so the long blocks start first and the short ones fill the CUs
// beside and after them; a launch of its own for each would end in a part-filled round, and
// dX alone, with fewer tiles than CUs, would have to be split.
// A tile is 256 x 256, eight waves of 128 x 64 (two per SIMD); stages of 64 columns (a
// 128-byte line per row) in a two-slot LDS ring filled by DMA, dense v_mfma_f32_32x32x16_bf16.
// Each depth's fragments are read while the previous depth's MFMAs issue; one barrier a
// stage, before its last depth: the next stage has landed and every wave has read this one,
// whose slot is then refilled.
// Measured at 4096 tokens of an 8192 x 8192 layer: about 1.7 us a stage, 1.25 PFLOP/s.  What
// bounds it is power and the operand stream together: a loop of the same MFMAs alone on
// random operands runs a stage in 0.92 us, with the fragment reads 1.35, with the loads and
// the barrier 1.60.  No faster, to 1%: the loads spread over the stage's depths, all of a
// stage's fragments read ahead (4 sets), two depths ahead with 16 MFMAs between.
constexpr int kRingCol = 36, kRingA = (256 * kRingCol + 16 * 8) * 4;   // a decoded stage: words a column, bytes

// A tile.  DEC: dX with the A operand decoded from the packed weights into the ring's slot, as
// t[column][row pair] (36 words a column, 8 more every 16); each thread decodes two rows of 16
// columns a stage, loaded a stage ahead.
template <bool DEC>
__device__ __forceinline__ void grad_tile(const GradArgs& g, const GradJob& job, bool isx, int bid, int split, uint8_t* smem) {
    constexpr int SR = 4, ST = 2, WRN = 2, WTN = 4, NW = 8, T = 256, ROWB = 128, D = 4;
    constexpr int STAGE = T * ROWB, NL = STAGE / 1024 / NW;   // 4 loads of an operand per wave
    // slots: A, A, B, B (DEC: with A's padding) or A, B, A, B
    constexpr int BOFF = DEC ? 2 * kRingA : STAGE, ASLOT = DEC ? kRingA : 2 * STAGE, BSLOT = DEC ? STAGE : 2 * STAGE;
    static_assert(!DEC || BOFF + 2 * STAGE + sizeof(SpreadTable) <= NW * kStageWords<SR> * 4, "slots fit in the staging buffers");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % WRN, wt = wave / WRN;
    int ta, tb;
    tile_of(bid, job.tiles_a * job.tiles_b, job.tiles_a, job.tiles_b, ta, tb);
    const int64_t a0 = (int64_t)ta * T, b0 = (int64_t)tb * T;
    const int s_begin = split * job.spp;
    const int nsteps = job.nsteps - s_begin < job.spp ? job.nsteps - s_begin : job.spp;   // >= 1
    const uint32_t sbase = lds_addr(smem);
    auto sw = [](int r) { return (r >> 1) & 7; };   // row r: logical 16-byte chunk c at c ^ sw(r)
    // dV of a lifted weight reads X's rows by their columns (job.lda is then XT's row length)
    const int ns = isx ? 0 : g.Ns;
    const int64_t first = orig_col(a0, ns);
    const void* baseA = DEC ? nullptr : uniform_ptr(job.A + first * job.lda + (int64_t)s_begin * 64);
    const void* baseB = uniform_ptr(job.B + b0 * job.ldb + (int64_t)s_begin * 64);
    const int64_t amax = job.rowsA - 1 - a0, bmax = job.rowsB - 1 - b0;
    uint32_t oA[NL], oB[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int row = (wave * NL + i) * 8 + (lane >> 3);
        const uint32_t c = (uint32_t)(((lane & 7) ^ sw(row)) * 16);
        oA[i] = DEC ? 0 : (uint32_t)((orig_col(a0 + (row < amax ? row : amax), ns) - first) * job.lda * 2) + c;
        oB[i] = (uint32_t)((row < bmax ? row : bmax) * job.ldb * 2) + c;
    }
    auto issue = [&](int s) __attribute__((always_inline)) {
        if constexpr (!DEC) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                dma16s(sbase + (uint32_t)((s & 1) * ASLOT) + (wave * NL + i) * 1024, baseA, oA[i] + (uint32_t)(s * ROWB));
        }
#pragma unroll
        for (int i = 0; i < NL; ++i)
            dma16s(sbase + (uint32_t)(BOFF + (s & 1) * BSLOT) + (wave * NL + i) * 1024, baseB, oB[i] + (uint32_t)(s * ROWB));
    };
    // DEC: the thread's two rows (2 pair, 2 pair + 1 of the stage's 64) and 16 columns
    SpreadTable& table = *(SpreadTable*)(smem + BOFF + 2 * STAGE);
    const int dc = tid & 15, pair = tid >> 4;
    const bool kok = a0 + 16 * dc < job.rowsA;
    struct Packed {
        i32x4_t v[2];
        uint32_t ix[2];
    };
    auto load_packed = [&](int s, Packed& p) __attribute__((always_inline)) {
        const int64_t q0 = (int64_t)(s_begin + (s < nsteps ? s : nsteps - 1)) * 64;
        const int mat = q0 >= g.Rp ? 1 : 0;   // Rp is a multiple of 64: a stage is of one weight
        const uint16_t* vals = mat ? g.vals[1] : g.vals[0];
        const uint32_t* idx = mat ? g.idx[1] : g.idx[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t q = q0 - mat * g.Rp + 2 * pair + j, r = q < g.R ? q : 0, k = kok ? a0 + 16 * dc : 0;
            p.v[j] = *(const i32x4_t*)(vals + r * g.ldv + k / 2);
            p.ix[j] = idx[r * g.ldi + k / 32];
        }
    };
    auto decode = [&](int s, const Packed& p) __attribute__((always_inline)) {
        const int64_t q0 = (int64_t)(s_begin + s) * 64, q = q0 - (q0 >= g.Rp ? g.Rp : 0) + 2 * pair;
        const i32x4_t z0 = kok && q < g.R ? p.v[0] : i32x4_t{0, 0, 0, 0}, z1 = kok && q + 1 < g.R ? p.v[1] : i32x4_t{0, 0, 0, 0};
        uint32_t x[16];
        decode_pair16(table, __builtin_bit_cast(uint4, z0), p.ix[0] >> (16 * (dc & 1)), __builtin_bit_cast(uint4, z1),
                      p.ix[1] >> (16 * (dc & 1)), x);
        uint32_t* w = (uint32_t*)(smem + (s & 1) * ASLOT) + dc * (16 * kRingCol + 8) + pair;
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e * kRingCol] = x[e];
    };
    struct Frag {
        i32x4_t a[SR], b[ST];
    };
    const int h = lane >> 5, l32 = lane & 31;
    auto read_depth = [&](int s, int d, Frag& f) __attribute__((always_inline)) {
        const uint8_t* sA = smem + (s & 1) * ASLOT;
        const uint8_t* sB = smem + BOFF + (s & 1) * BSLOT;
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            const int row = (wr * SR + i) * 32 + l32;
            f.a[i] = DEC ? *(const i32x4_t*)(sA + row * (kRingCol * 4) + (row >> 4) * 32 + (2 * d + h) * 16)
                         : *(const i32x4_t*)(sA + row * ROWB + ((2 * d + h) ^ sw(row)) * 16);
        }
#pragma unroll
        for (int j = 0; j < ST; ++j) {
            const int row = (wt * ST + j) * 32 + l32;
            f.b[j] = *(const i32x4_t*)(sB + row * ROWB + ((2 * d + h) ^ sw(row)) * 16);
        }
    };
    f32x16_t acc[SR][ST];
#pragma unroll
    for (int i = 0; i < SR; ++i)
#pragma unroll
        for (int j = 0; j < ST; ++j) acc[i][j] = f32x16_t{};
    auto mfmas = [&](const Frag& f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < ST; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f.a[i]),
                                                                     __builtin_bit_cast(bf16x8_t, f.b[j]), acc[i][j], 0, 0, 0);
    };
    // a depth's fragment reads, one after each of its first MFMAs
    auto interleave = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SR + ST; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, SR * ST - SR - ST, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    uint32_t words[ST][SR] = {};
    if (!DEC && !isx) grad_positions<SR, ST>(g, a0 + wr * SR * 32, b0 + wt * ST * 32, lane, words);
    Frag fr[2];
    Packed pk[2];
    if constexpr (DEC) {
        load_packed(0, pk[0]);
        load_packed(1, pk[1]);
        table.fill(tid);
        __syncthreads();
        decode(0, pk[0]);
    }
    issue(0);
    if (nsteps > 1) issue(1);
    if (nsteps > 1) wait_vm_barrier<(DEC ? 1 : 2) * NL>();
    else wait_vm_barrier<0>();
    read_depth(0, 0, fr[0]);
    // one stage; DEC: cur holds the next stage's packed rows, the stage after's are loaded into nxt
    auto stage = [&](int s, Packed& cur, Packed& nxt) __attribute__((always_inline)) {
        if constexpr (DEC) {
            load_packed(s + 2, nxt);
            if (s + 1 < nsteps) decode(s + 1, cur);
        }
#pragma unroll
        for (int d = 0; d + 1 < D; ++d) {
            read_depth(s, d + 1, fr[(d + 1) & 1]);
            mfmas(fr[d & 1]);
            if constexpr (!DEC) interleave();
        }
        // the last depth's fragments complete before the branch (the barrier waits for them anyway)
        __builtin_amdgcn_s_waitcnt(0xc07f);
        if (s + 1 < nsteps) {
            wait_vm_barrier<0>();
            if (s + 2 < nsteps) issue(s + 2);
            read_depth(s + 1, 0, fr[0]);
        }
        mfmas(fr[(D - 1) & 1]);
    };
    if constexpr (DEC) {
        for (int s = 0; s < nsteps; s += 2) {
            stage(s, pk[1], pk[0]);
            if (s + 1 < nsteps) stage(s + 1, pk[0], pk[1]);
        }
    } else {
        for (int s = 0; s < nsteps; ++s) stage(s, pk[0], pk[1]);
    }
    wait_vm_all();
    if (!DEC && !isx) {
        if (g.vpart) {
            GradArgs p = g;
            const int64_t half = job.rowsA / 2, one = g.R * half;
            p.dV[0] = g.vpart + (int64_t)split * (job.rowsB > g.Rp ? 2 : 1) * one;
            p.dV[1] = (float*)p.dV[0] + one;
            p.lddv = half;
            p.dvf32 = 1;
            store_grad_tile<SR, ST>(p, acc, words, a0 + wr * SR * 32, b0 + wt * ST * 32, lane);
        } else {
            store_grad_tile<SR, ST>(g, acc, words, a0 + wr * SR * 32, b0 + wt * ST * 32, lane);
        }
        return;
    }
    __syncthreads();   // every wave has read the ring: its LDS stages the output
    SpmmArgs a{};
    a.Mtok = job.rowsB;
    a.R = job.rowsA;
    a.Y = g.part ? (void*)(g.part + (int64_t)split * a.Mtok * a.R) : g.dX;
    a.ydt = g.part || g.dxf32 ? NM_F32 : NM_BF16;
    a.ldy = g.part ? a.R : g.lddx;
    store_tile<uint16_t, SR, ST>(a, acc, a0 + wr * SR * 32, b0 + wt * ST * 32, a0 + T <= a.R && b0 + T <= a.Mtok,
                                 (uint32_t*)smem + wave * kStageWords<SR>, lane);
}

template <bool DEC>
__global__ __launch_bounds__(512, 1) void grad_ring_kernel(GradArgs g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[8 * kStageWords<4> * 4];
    if ((int)blockIdx.x < g.nx) {
        const int tiles = g.x.tiles_a * g.x.tiles_b, split = blockIdx.x / tiles;
        grad_tile<DEC>(g, g.x, true, blockIdx.x - split * tiles, split, smem);
    } else {
        const int tiles = g.v.tiles_a * g.v.tiles_b, b = blockIdx.x - g.nx, split = b / tiles;
        grad_tile<false>(g, g.v, false, b - split * tiles, split, smem);
    }
}

// ------------------------------------------------------------------ few tokens
// Up to 128 tokens the dense ring pays for 256-token tiles and for a dense copy of the weights;
// both products are then streams: dX reads the packed weights, dV writes its packed
// values.  One grid holds both.
// dX: a block sums dY W over a run of weight rows for 128 columns and all tokens (ST
// sub-tiles of 32).  64 rows a step: values (a line per row), positions and the tokens' 64
// columns of D are loaded PF steps ahead into registers (three blocks a CU then keep about
// 100 KB in flight, which a CU's share of the HBM rate needs), the weight is decoded into LDS
// as t[column][row pair] (36 words a column, and 8 more every 16 columns: writes and 16-byte
// fragment reads free of bank conflicts), and multiplied with v_mfma_f32_32x32x16_bf16;
// wave w takes columns 32 w .. + 31.  LDS is double buffered, one barrier a step.  Partials
// [split][M][K] in f32 are added by grad_reduce_kernel (a single split of a plain weight is dX
// itself).  Blocks of one split and all panels
// run on one XCD, whose L2 then serves the positions' lines (8 panels each) once.
// dV: 128 x 128 tiles, four waves of 64 x 64; the tile's tokens (one or two lines per row of XT
// and of DT) are loaded whole into LDS, the epilogue is the ring's.
struct FewArgs {
    GradArgs g;
    GradIn in;
    int64_t M, K, Rn;
    const uint16_t* D;
    int64_t ldd;
    int panels, splits, spp;   // 128-column panels of dX, splits of its Rn / 64 steps, steps per split
    int tk, tr;                // 128-wide tiles of dV along K and along the stacked rows
};
constexpr int kFewCol = 36, kFewWords = 128 * kFewCol + 8 * 8;   // a decoded step
constexpr int64_t kFewTokens = 128;                              // dV's tiles hold all tokens

template <int ST>
__global__ __launch_bounds__(256, ST == 4 ? 2 : 3) void grad_few_kernel(FewArgs a) {
    constexpr int PF = 4, DBYTES = 32 * ST * 128, LDS = 2 * (kFewWords * 4 + DBYTES);
    constexpr int HV = ST == 4 ? 2 : 1;   // 64-token halves of dV: Mp == 64 HV
    static_assert(LDS >= HV * 32 * 1024, "dV's tile fits");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
    __shared__ SpreadTable table;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto sw = [](int r) { return (r >> 1) & 7; };   // 128-byte row r: logical 16-byte chunk c at c ^ sw(r)
    if ((int)blockIdx.x >= a.g.nx) {   // dV
        // an XCD walks whole row panels (nx is a multiple of 8)
        const int b = blockIdx.x - a.g.nx, loc = b >> 3, tr = (loc / a.tk) * 8 + (b & 7);
        if (tr >= a.tr) return;
        const int64_t k0 = (int64_t)(loc % a.tk) * 128, q0 = (int64_t)tr * 128;
        const int64_t first = orig_col(k0, a.g.Ns);
        const void *baseA = uniform_ptr(a.g.v.A + first * 64 * HV), *baseB = uniform_ptr(a.g.v.B + q0 * 64 * HV);
        const int64_t kmax = a.K - 1 - k0, qmax = a.Rn - 1 - q0;
        const uint32_t sbase = lds_addr(smem);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (wave * 4 + i) * 8 + (lane >> 3);
            const uint32_t c = (uint32_t)(((lane & 7) ^ sw(row)) * 16);
            const uint32_t arow = (uint32_t)(orig_col(k0 + (row < kmax ? row : kmax), a.g.Ns) - first);
#pragma unroll
            for (int v = 0; v < HV; ++v) {
                const uint32_t at = sbase + v * 32768 + (wave * 4 + i) * 1024;
                dma16s(at, baseA, arow * (128u * HV) + 128u * v + c);
                dma16s(at + 16384, baseB, (uint32_t)(row < qmax ? row : qmax) * (128u * HV) + 128u * v + c);
            }
        }
        uint32_t words[2][2];
        grad_positions<2, 2>(a.g, k0 + (wave & 1) * 64, q0 + (wave >> 1) * 64, lane, words);
        f32x16_t acc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
        wait_vm_barrier<0>();
        const int ra = (wave & 1) * 64 + l32, rb = (wave >> 1) * 64 + l32;
#pragma unroll
        for (int dv = 0; dv < 4 * HV; ++dv) {
            const int d = dv & 3;
            const uint8_t* half = smem + (dv >> 2) * 32768;
            i32x4_t fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = *(const i32x4_t*)(half + (ra + 32 * i) * 128 + ((2 * d + h) ^ sw(ra + 32 * i)) * 16);
                fb[i] = *(const i32x4_t*)(half + 16384 + (rb + 32 * i) * 128 + ((2 * d + h) ^ sw(rb + 32 * i)) * 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa[i]),
                                                                         __builtin_bit_cast(bf16x8_t, fb[j]), acc[i][j], 0, 0, 0);
        }
        store_grad_tile<2, 2>(a.g, acc, words, k0 + (wave & 1) * 64, q0 + (wave >> 1) * 64, lane);
        return;
    }
    // dX: split 8 u + x of XCD x = b % 8, panels side by side
    const int loc = blockIdx.x >> 3, panel = loc % a.panels, split = (loc / a.panels) * 8 + (blockIdx.x & 7);
    if (split >= a.splits) return;
    const int64_t k0 = (int64_t)panel * 128;
    const int nstep = (int)(a.Rn / 64), s0 = split * a.spp, s1 = s0 + a.spp < nstep ? s0 + a.spp : nstep;
    const int c = tid & 7, pair = tid >> 3;
    const int64_t kc = k0 + 16 * c;
    const int64_t Rp = a.g.Rp;
    i32x4_t pv[PF][2], pd[PF][ST];   // values, positions and D of the steps ahead
    uint32_t pi[PF][2];
    // the tokens' rows of D: rows past M read the last one (their sums are not stored)
    const uint16_t* dp[ST];
#pragma unroll
    for (int j = 0; j < ST; ++j) {
        const int64_t m = 32 * j + (tid >> 3);
        dp[j] = a.D + (m < a.M ? m : a.M - 1) * a.ldd + 8 * c;
    }
    // steps past the last reload it (never used); rows past R and columns past K read row 0 or
    // column 0 and are zeroed at the decode
    const bool kok = kc < a.K;
    auto load = [&](int s, i32x4_t (&v)[2], uint32_t (&ix)[2], i32x4_t (&d)[ST]) __attribute__((always_inline)) {
        const int64_t q0 = (int64_t)(s < s1 ? s : s1 - 1) * 64;
        const int mat = q0 >= Rp ? 1 : 0;   // Rp is a multiple of 64: a step is of one weight
        const uint16_t* vals = mat ? a.in.vals[1] : a.in.vals[0];
        const uint32_t* idx = mat ? a.in.idx[1] : a.in.idx[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t q = q0 - mat * Rp + 2 * pair + j, r = q < a.in.R ? q : 0, k = kok ? kc : 0;
            v[j] = *(const i32x4_t*)(vals + r * a.in.ldv + k / 2);
            ix[j] = idx[r * a.in.ldi + k / 32];
        }
#pragma unroll
        for (int j = 0; j < ST; ++j) d[j] = *(const i32x4_t*)(dp[j] + q0);
    };
    f32x16_t acc[ST];
#pragma unroll
    for (int j = 0; j < ST; ++j) acc[j] = f32x16_t{};
#pragma unroll
    for (int u = 0; u < PF; ++u) load(s0 + u, pv[u], pi[u], pd[u]);
    table.fill(tid);
    __syncthreads();
    for (int sb = s0; sb < s1; sb += PF) {
#pragma unroll
        for (int u = 0; u < PF; ++u) {
            const int s = sb + u;
            if (s < s1) {   // the same for the whole block
                uint8_t* const buf = smem + (u & 1) * (kFewWords * 4 + DBYTES);
                uint8_t* const dbuf = buf + kFewWords * 4;
                const int64_t q = (int64_t)s * 64 - (s * 64 >= Rp ? Rp : 0) + 2 * pair;
                uint32_t x[16];
                const i32x4_t z0 = kok && q < a.in.R ? pv[u][0] : i32x4_t{0, 0, 0, 0};
                const i32x4_t z1 = kok && q + 1 < a.in.R ? pv[u][1] : i32x4_t{0, 0, 0, 0};
                decode_pair16(table, __builtin_bit_cast(uint4, z0), pi[u][0] >> (16 * (c & 1)),
                              __builtin_bit_cast(uint4, z1), pi[u][1] >> (16 * (c & 1)), x);
                uint32_t* w = (uint32_t*)buf + c * (16 * kFewCol + 8) + pair;
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e * kFewCol] = x[e];
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    const int m = 32 * j + (tid >> 3);
                    *(i32x4_t*)(dbuf + m * 128 + (c ^ sw(m)) * 16) = pd[u][j];
                }
                load(s + PF, pv[u], pi[u], pd[u]);
                __syncthreads();   // the buffer was last read two steps ago, before the last step's barrier
                const int col = 32 * wave + l32;
                const uint32_t* row = (const uint32_t*)buf + col * kFewCol + 8 * (col >> 4) + 4 * h;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const i32x4_t fa = *(const i32x4_t*)(row + 8 * d);
#pragma unroll
                    for (int j = 0; j < ST; ++j) {
                        const int m = 32 * j + l32;
                        const i32x4_t fb = *(const i32x4_t*)(dbuf + m * 128 + ((2 * d + h) ^ sw(m)) * 16);
                        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa),
                                                                          __builtin_bit_cast(bf16x8_t, fb), acc[j], 0, 0, 0);
                    }
                }
            }
        }
    }
    // a lane: token 32 j + l32, columns 8 g + 4 h .. + 3 of the wave's 32; no partials: dX itself
    float* part = a.g.part + (int64_t)split * a.M * a.K;
    if (!a.g.part) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
            const int64_t m = 32 * j + l32;
            if (m >= a.M) continue;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t k = k0 + 32 * wave + 8 * (e >> 2) + 4 * h + (e & 3), o = m * a.g.lddx + k;
                if (k >= a.K) continue;
                if (a.g.dxf32) ((float*)a.g.dX)[o] = acc[j][e];
                else ((uint16_t*)a.g.dX)[o] = (uint16_t)f32_to_bf16_bits(acc[j][e]);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < ST; ++j) {
        const int64_t m = 32 * j + l32;
        if (m >= a.M) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t k = k0 + 32 * wave + 8 * g + 4 * h;
            if (k < a.K)
                *(float4*)(part + m * a.K + k) = make_float4(acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]);
        }
    }
}

// dX [M, K] from its partials [splits][M][Kl], in split order; Ns: column k from the lifted columns
// above it, windows in order
__global__ __launch_bounds__(256) void grad_reduce_kernel(const float* __restrict__ part, int splits, int64_t M, int64_t K,
                                                          int64_t Kl, int Ns, void* __restrict__ dX, int64_t lddx, int f32) {
    const int64_t total = M * K;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t m = t / K, k = t - m * K;
        float v;
        if (Ns == 0) {
            v = split_sum(part + t, splits, total);
        } else {
            const int g = (int)((uint32_t)k / (uint32_t)(2 * Ns)), p = (int)k - g * 2 * Ns;
            v = 0.0f;
            for (int w = first_window(p); w <= last_window(p, Ns); ++w)
                v += split_sum(part + m * Kl + 4 * (g * (Ns - 1) + w) + p - 2 * w, splits, M * Kl);
        }
        if (f32) ((float*)dX)[m * lddx + k] = v;
        else ((uint16_t*)dX)[m * lddx + k] = (uint16_t)f32_to_bf16_bits(v);
    }
}

// Packed dV of one weight (blockIdx.y) from its partials, in split order
__global__ __launch_bounds__(256) void grad_reduce_v_kernel(const float* __restrict__ part, int splits, int64_t R, int64_t half,
                                                            GradOut out) {
    const int64_t total = R * half, all = total * gridDim.y;
    void* dV = out.dV[blockIdx.y];
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t / half, o = r * out.lddv + t - r * half;
        const float v = split_sum(part + blockIdx.y * total + t, splits, all);
        if (out.dvdt == NM_F32) ((float*)dV)[o] = v;
        else ((uint16_t*)dV)[o] = (uint16_t)f32_to_bf16_bits(v);
    }
}

// ------------------------------------------------------------------ host side
// Splits of dX's sum (Rn / 64 stages).  Beside dV no block should run longer than the whole
// call's share of a CU (at least 16 stages); alone, the count whose rounds take least.  A
// stage of a tile measured at about 1.8 us in full rounds, partials at about 4 TB/s with a
// launch of their own.
static int grad_x_splits(int64_t M, int64_t K, int64_t Rn, bool with_v) {
    const int64_t cus = device_cus(), tiles = ceil_div(K, 256) * ceil_div(M, 256), ns = Rn / 64;
    const int64_t vwork = with_v ? ceil_div(K, 256) * ceil_div(Rn, 256) * ceil_div(M, 64) : 0;
    int best = 1;
    double best_us = 1e30;
    for (int64_t ks = 1; ks <= 16 && ks * 4 <= ns + 3; ++ks) {
        const int64_t one = ceil_div(ns, ks) + 2;
        const int64_t share = ceil_div(tiles * ks * one + vwork, cus), rounds = ceil_div(tiles * ks, cus) * one;
        const int64_t stages = with_v ? (share > rounds ? share : rounds) : rounds;
        const double us = 1.8 * (double)stages + (ks > 1 ? 4.0 + 8e-6 / 4.0 * (double)(ks * M * K) : 0.0);
        if (us < best_us) {
            best_us = us;
            best = (int)ks;
        }
    }
    return best;
}

// Splits of dV's sum (the tokens, Mp / 64 stages) where its tiles, beside dX's blocks, leave CUs idle:
// a stage is about 1.7 us, the partials' launch 6 and each megabyte of them 1.  Measured, plain and
// gated: 2048 tokens of 1024 x 1024 62.8 -> 43.9 and 68.0 -> 55.7 us, 2000 of 512 x 512 51.8 -> 30.8 and
// 60.0 -> 34.0; without the partials' price 1163 of 459 x 3600, gated, went from 46.7 to 59.2.
// As many as nx = 0 gives is the most any call takes.
static int grad_v_splits(int64_t M, int64_t K, int64_t R, int64_t Rn, int nmat, int64_t nx) {
    const int64_t tiles = ceil_div(K, 256) * ceil_div(Rn, 256), ns = ceil_div(M, 64);
    const double one_mb = (double)(nmat * R * (K / 2)) * 4e-6;
    int best = 1;
    double best_us = 1.7 * (double)ns;
    for (int64_t n = 2; n * tiles <= device_cus() - nx && n <= ns / 4; ++n) {
        const double us = 1.7 * (double)ceil_div(ns, n) + 6.0 + one_mb * (double)n;
        if (us < best_us) {
            best_us = us;
            best = (int)n;
        }
    }
    return best;
}
static size_t grad_v_part_bytes(int64_t M, int64_t K, int64_t R, int64_t Rn, int nmat) {
    const int n = grad_v_splits(M, K, R, Rn, nmat, 0);
    return n > 1 ? (size_t)n * (size_t)(nmat * R * (K / 2)) * 4 : 0;
}

// partials of dX over K columns: with splits, or a lifted dX' to fold
static size_t grad_x_part_bytes(int64_t M, int64_t K, int64_t Rn, bool lifted) {
    size_t n = lifted ? (size_t)(M * K) * 4 : 0;
    for (int v = 0; v < 2; ++v) {
        const int ks = grad_x_splits(M, K, Rn, v != 0);
        if (ks > 1 && (size_t)ks * (size_t)(M * K) * 4 > n) n = (size_t)ks * (size_t)(M * K) * 4;
    }
    return n;
}

static int64_t up64(int64_t n) { return (n + 63) & ~(int64_t)63; }
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Splits of the few-token dX: about three blocks a CU, in eights (one per XCD).
static bool few_tokens(int64_t M) { return M <= kFewTokens; }
static int few_splits(int64_t K, int64_t Rn, int* spp) {
    const int64_t steps = Rn / 64, panels = ceil_div(K, 128);
    int64_t n = ceil_div(3 * device_cus(), panels * 8) * 8;
    // at least the steps loaded ahead per split: more splits of a small weight are all partials
    if (n > steps / 4) n = steps / 4 > 1 ? steps / 4 : 1;
    *spp = (int)ceil_div(steps, n);
    return (int)ceil_div(steps, *spp);
}

// Whether dX's tiles decode the packed weights themselves.  Every token tile decodes them again
// (about half a microsecond a stage), the dense copy costs 3 bytes per weight once.
// Measured on the gated block's backward at 11008 x 4096: 129 tokens 193 -> 137 us, 256
// 211 -> 158, 512 297 -> 257, 768 391 -> 357, 1024 464 -> 462, 2048 767 -> 865; on small weights the longer
// stages cost more than the copy (4096 x 1024 at 256 tokens 37.1 -> 40.2, 5504 x 2048 73 -> 59).
// A lifted weight's copy is over K, the decoded tiles over K': 6:8 at 256 tokens 267 -> 204 us, 512
// 363 -> 343, 768 463 -> 476; 8:10 (K = 4160) 267 -> 223, 370 -> 359, 473 -> 502.
static bool ring_decodes(int64_t M, int64_t K, int64_t Rn, int Ns) {
    return M <= (Ns ? 2 : 3) * 256 && K * Rn >= ((int64_t)1 << 24);
}

// Workspace of one backward call, in the order it is carved.
struct GradWs {
    size_t d = 0, dt = 0, xt = 0, wt = 0, part = 0, vpart = 0;
    size_t total() const { return d + dt + xt + wt + part + vpart; }
};
static int64_t lifted_width(int64_t K, int Ns) { return Ns ? K / (2 * Ns) * 4 * (Ns - 1) : K; }
static GradWs grad_ws_layout(int64_t M, int64_t Korig, int64_t R, int Ns, int nmat) {
    GradWs w;
    if (M <= 0 || Korig <= 0 || R <= 0) return w;
    const int64_t K = lifted_width(Korig, Ns);
    const int64_t Rn = nmat * up64(R), Mp = up64(M);
    w.d = up256((size_t)(M * Rn * 2));
    w.dt = up256((size_t)(Rn * Mp * 2));
    w.xt = up256((size_t)(Korig * Mp * 2));
    if (few_tokens(M)) {
        int spp;
        w.part = up256((size_t)few_splits(K, Rn, &spp) * (size_t)(M * K) * 4);
        return w;
    }
    const bool dec = ring_decodes(M, K, Rn, Ns);
    if (!dec) w.wt = up256((size_t)(Korig * Rn * 2));
    w.part = up256(grad_x_part_bytes(M, dec ? K : Korig, Rn, dec && Ns != 0));
    w.vpart = up256(grad_v_part_bytes(M, K, R, Rn, nmat));
    return w;
}
size_t grad_ws(int64_t M, int64_t K, int64_t R, int Ns, int nmat) { return grad_ws_layout(M, K, R, Ns, nmat).total(); }

// bytes that every row start is a multiple of: 16, 4 or 2
static int row_align(const void* p, int64_t ld) {
    const uintptr_t a = (uintptr_t)p | (uintptr_t)(ld * 2);
    return (a & 15u) == 0 ? 16 : (a & 3u) == 0 ? 4 : 2;
}

// a row-major matrix of width 2-byte units set to zero (ld in bytes)
__global__ __launch_bounds__(256) void zero_rows_kernel(uint8_t* __restrict__ p, int64_t rows, int64_t width, int64_t ld) {
    const int64_t n = rows * width;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        *(uint16_t*)(p + (i / width) * ld + (i % width) * 2) = 0;
}

nm_status launch_grad(const GradIn& given, const GradOut& out, int nmat, void* ws, hipStream_t s) {
    GradIn in = given;
    in.Kl = lifted_width(in.K, in.Ns);
    if (in.M == 0 || in.R == 0) {
        // an empty sum: dV is zero without tokens, dX without rows
        auto zero = [&](void* p, int64_t rows, int64_t width, int64_t ld) {   // in 2-byte units
            if (p && rows > 0)
                hipLaunchKernelGGL(zero_rows_kernel, dim3(grid_cap(ceil_div(rows * width, 256), 8192)), dim3(256), 0, s,
                                   (uint8_t*)p, rows, width, ld * 2);
        };
        const int64_t vs = out.dvdt == NM_BF16 ? 1 : 2, xs = out.dxdt == NM_BF16 ? 1 : 2;
        for (int i = 0; i < nmat; ++i) zero(out.dV[i], in.R, in.Kl / 2 * vs, out.lddv * vs);
        zero(out.dX, in.M, in.K * xs, out.lddx * xs);
        return check_launch("backward");
    }
    const int64_t Rp = up64(in.R), Rn = nmat * Rp, Mp = up64(in.M);
    const GradWs w = grad_ws_layout(in.M, in.K, in.R, in.Ns, nmat);
    uint8_t* p = (uint8_t*)ws;
    uint16_t* D = (uint16_t*)p;
    uint16_t* DT = (uint16_t*)(p + w.d);
    uint16_t* XT = (uint16_t*)(p + w.d + w.dt);
    uint16_t* WT = (uint16_t*)(p + w.d + w.dt + w.xt);
    float* PART = (float*)(p + w.d + w.dt + w.xt + w.wt);
    const bool dx = out.dX != nullptr, dv = out.dV[0] != nullptr;
    int vec = row_align(in.dY, in.lddy);
    if (nmat == 2) {
        const int g = row_align(in.G, in.ldg), u = row_align(in.U, in.ldg);
        vec = g < vec ? g : vec;
        vec = u < vec ? u : vec;
    }
    // dX reads dY itself where its rows are whole 64-column stages on 16-byte boundaries
    const bool direct = nmat == 1 && vec == 16 && in.R == Rp && in.lddy < (1 << 23);
    const uint16_t* B = direct ? in.dY : D;
    const int64_t ldb = direct ? in.lddy : Rn;
    LayoutArgs l{};
    l.in = in;
    l.Rp = Rp;
    l.Mp = Mp;
    l.Rn = Rn;
    l.D = dx && !direct ? D : nullptr;
    l.DT = dv ? DT : nullptr;
    l.XT = XT;
    l.WT = WT;
    l.td = (int)(Rp / 64);
    l.tw = (int)ceil_div(in.Kl, in.Ns ? lifted_tile_groups(in.Ns) * 4 * (in.Ns - 1) : 128);
    l.tx = (int)ceil_div(in.K, 64);
    l.nd = l.D || l.DT ? l.td * (int)(Mp / 64) : 0;
    const bool dec = !few_tokens(in.M) && ring_decodes(in.M, in.Kl, Rn, in.Ns);
    const int64_t Kx = few_tokens(in.M) || dec ? in.Kl : in.K;   // columns of dX's product
    l.nw = dx && !few_tokens(in.M) && !dec ? l.tw * (int)(Rp / 64) * nmat : 0;
    l.nx = dv ? l.tx * (int)(Mp / 64) : 0;
    const dim3 gl((unsigned)(l.nd + l.nw + l.nx));
    if (gl.x) {
#define NM_LAYOUT(A)                                                                                  \
    do {                                                                                              \
        if (vec == 16) hipLaunchKernelGGL((grad_layout_kernel<A, 16>), gl, dim3(256), 0, s, l);       \
        else if (vec == 4) hipLaunchKernelGGL((grad_layout_kernel<A, 4>), gl, dim3(256), 0, s, l);    \
        else hipLaunchKernelGGL((grad_layout_kernel<A, 2>), gl, dim3(256), 0, s, l);                  \
    } while (0)
    if (nmat == 1) NM_LAYOUT(-1);
    else if (in.act == NM_ACT_SILU) NM_LAYOUT(NM_ACT_SILU);
    else if (in.act == NM_ACT_GELU) NM_LAYOUT(NM_ACT_GELU);
    else if (in.act == NM_ACT_GELU_TANH) NM_LAYOUT(NM_ACT_GELU_TANH);
    else NM_LAYOUT(NM_ACT_RELU2);
    }
#undef NM_LAYOUT
    GradArgs g{};
    int nv = 0, splits = 1, vsplits = 1;
    for (int i = 0; i < 2; ++i) {
        g.vals[i] = in.vals[i];
        g.idx[i] = in.idx[i];
        g.dV[i] = out.dV[i];
    }
    g.Ns = in.Ns;
    g.ldv = in.ldv;
    g.ldi = in.ldi;
    g.R = in.R;
    g.Rp = Rp;
    if (dx) {
        splits = grad_x_splits(in.M, Kx, Rn, dv);
        GradJob& j = g.x;
        j.A = WT;
        j.lda = Rn;
        j.rowsA = Kx;
        j.B = B;
        j.ldb = ldb;
        j.rowsB = in.M;
        j.nsteps = (int)(Rn / 64);
        j.spp = (int)ceil_div(j.nsteps, splits);
        splits = (int)ceil_div(j.nsteps, j.spp);
        j.tiles_a = (int)ceil_div(Kx, 256);
        j.tiles_b = (int)ceil_div(in.M, 256);
        g.nx = j.tiles_a * j.tiles_b * splits;
        g.dX = out.dX;
        g.part = splits > 1 || Kx != in.K ? PART : nullptr;
        g.lddx = out.lddx;
        g.dxf32 = out.dxdt == NM_F32;
    }
    if (dv) {
        GradJob& j = g.v;
        j.A = XT;
        j.lda = Mp;
        j.rowsA = in.Kl;
        j.B = DT;
        j.ldb = Mp;
        j.rowsB = Rn;
        j.nsteps = j.spp = (int)(Mp / 64);
        j.tiles_a = (int)ceil_div(in.Kl, 256);
        j.tiles_b = (int)ceil_div(Rn, 256);
        nv = j.tiles_a * j.tiles_b;
        if (!few_tokens(in.M)) {
            vsplits = grad_v_splits(in.M, in.Kl, in.R, Rn, nmat, g.nx);
            j.spp = (int)ceil_div(j.nsteps, vsplits);
            vsplits = (int)ceil_div(j.nsteps, j.spp);
            nv *= vsplits;
            g.vpart = vsplits > 1 ? (float*)((uint8_t*)PART + w.part) : nullptr;
        }
        g.lddv = out.lddv;
        g.dvf32 = out.dvdt == NM_F32;
    }
    if (few_tokens(in.M)) {
        FewArgs f{};
        f.in = in;
        f.M = in.M;
        f.K = in.Kl;
        f.Rn = Rn;
        f.D = B;
        f.ldd = ldb;
        f.tk = (int)ceil_div(in.Kl, 128);
        f.tr = (int)ceil_div(Rn, 128);
        if (dx) {
            f.panels = (int)ceil_div(in.Kl, 128);
            f.splits = splits = few_splits(in.Kl, Rn, &f.spp);
            g.nx = (int)ceil_div(splits, 8) * 8 * f.panels;
            g.part = splits > 1 || Kx != in.K ? PART : nullptr;
        }
        f.g = g;
        const dim3 gf((unsigned)(g.nx + (dv ? f.tk * (int)ceil_div(f.tr, 8) * 8 : 0)));
        if (in.M <= 32) hipLaunchKernelGGL(grad_few_kernel<1>, gf, dim3(256), 0, s, f);
        else if (in.M <= 64) hipLaunchKernelGGL(grad_few_kernel<2>, gf, dim3(256), 0, s, f);
        else hipLaunchKernelGGL(grad_few_kernel<4>, gf, dim3(256), 0, s, f);
    } else {
        const dim3 gr((unsigned)(g.nx + nv));
        if (dec) hipLaunchKernelGGL(grad_ring_kernel<true>, gr, dim3(512), 0, s, g);
        else hipLaunchKernelGGL(grad_ring_kernel<false>, gr, dim3(512), 0, s, g);
    }
    if (g.part)
        hipLaunchKernelGGL(grad_reduce_kernel, dim3(grid_cap(ceil_div(in.M * in.K, 256), 8192)), dim3(256), 0, s, PART,
                           splits, in.M, in.K, Kx, Kx != in.K ? in.Ns : 0, out.dX, out.lddx, g.dxf32);
    if (g.vpart)
        hipLaunchKernelGGL(grad_reduce_v_kernel, dim3(grid_cap(ceil_div(in.R * in.Kl / 2, 256), 4096), (unsigned)nmat), dim3(256),
                           0, s, g.vpart, vsplits, in.R, in.Kl / 2, out);
    return check_launch(nmat == 2 ? "nm_spmm_glu_backward" : "nm_spmm_backward");
}

}  // namespace nm
