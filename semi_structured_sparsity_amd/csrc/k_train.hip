// Gradients of the sparse layer and of the gated feed-forward block (bf16, plain 2:4).
//
// For y = x W^T with W [R, K] packed 2:4, and for a gated block with pre-activations
// G = x Wg^T, U = x Wu^T, H = act(G) . U:
//   dG = dH . U . act'(G),  dU = dH . act(G)
//   dX = dY W               (gated: dG Wg + dU Wu)
//   dV[r, j] = sum_m dY[m, r] X[m, col(r, j)]   for the kept positions col(r, j) only.
// Neither product can use the sparse instructions: they skip zeros of the operand along the
// summed dimension, W is 2:4 along K, but dX sums over R and dV over the tokens.  Both run as
// dense products on 256 x 256 tiles (dense_ring_kernel, k_spmm.hip), bound by the matrix
// cores and the operand stream; dV's epilogue keeps the packed positions of each tile, so the
// dense gradient never exists.
// The dense ring wants both operands with the summed dimension contiguous, so the operands
// are laid out once, in the workspace, by the bandwidth-bound kernels below:
//   D  [M, nmat * Rp]  dY, or dG | dU, the rows padded to Rp = a multiple of 64 with zeros,
//   DT [nmat * Rp, Mp] its transpose, the tokens padded to Mp = a multiple of 64 with zeros,
//   XT [K, Mp]         X transposed,
//   WT [K, nmat * Rp]  the packed weights, dense and transposed.
#include "nm_internal.h"

namespace nm {

// ------------------------------------------------------------------ layout kernels
// 64 x 64 tiles of a [rows, cols] bf16 matrix; 256 threads, each a pair of rows (2 p, 2 p + 1)
// and 8 columns.  The transposed tile goes through LDS as row-pair words T[column][pair]
// (stride 33 words: the 64 lanes of a write fall on 64 distinct banks).
struct PairTile {
    uint32_t t[64][33];
    // lo / hi: the thread's 8 elements of the even / odd row
    __device__ __forceinline__ void put(int c8, int pair, const uint32_t (&lo)[8], const uint32_t (&hi)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[c8 * 8 + i][pair] = lo[i] | (hi[i] << 16);
    }
    // 8 rows (of the source) of one column, 16 bytes
    __device__ __forceinline__ uint4 get(int col, int q) const {
        return make_uint4(t[col][4 * q], t[col][4 * q + 1], t[col][4 * q + 2], t[col][4 * q + 3]);
    }
};

// 8 bf16 of a row from column c; zero past cols (or if !ok)
template <bool VEC>
__device__ __forceinline__ void load_row8(const uint16_t* __restrict__ row, int64_t c, int64_t cols, bool ok,
                                          uint32_t (&x)[8]) {
    if (VEC && ok && c + 8 <= cols) {
        const uint4 u = *(const uint4*)(row + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
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

// S [rows, cols] (lds) -> T [cols, rowsp] (rows >= rows: zero) and, if C, the copy C [rows, ldc]
// with columns cols .. colsp zero.  Grid: (column tiles of colsp, row tiles of rowsp).
template <bool VEC>
__global__ __launch_bounds__(256) void transpose_pad_kernel(const uint16_t* __restrict__ S, int64_t lds, int64_t rows,
                                                            int64_t cols, uint16_t* __restrict__ T, int64_t rowsp,
                                                            uint16_t* __restrict__ C, int64_t ldc) {
    __shared__ PairTile tile;
    const int tid = threadIdx.x, c8 = tid & 7, pair = tid >> 3;
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int64_t r = r0 + 2 * pair, c = c0 + 8 * c8;
    uint32_t lo[8], hi[8];
    load_row8<VEC>(S + r * lds, c, cols, r < rows, lo);
    load_row8<VEC>(S + (r + 1) * lds, c, cols, r + 1 < rows, hi);
    if (C) {
        if (r < rows) *(uint4*)(C + r * ldc + c) = pack8(lo);
        if (r + 1 < rows) *(uint4*)(C + (r + 1) * ldc + c) = pack8(hi);
    }
    tile.put(c8, pair, lo, hi);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int col = (tid >> 3) + 32 * p, q = tid & 7;
        if (T && c0 + col < cols) *(uint4*)(T + (c0 + col) * rowsp + r0 + 8 * q) = tile.get(col, q);
    }
}

// dG | dU from dH, G, U (bf16 [M, R]); D [M, 2 Rp] and DT [2 Rp, Mp], both padded with zeros.
// dG and dU are rounded to bf16 here: they are operands of the bf16 matrix products, as the
// activations of the forward pass are.
template <int ACT, bool VEC>
__global__ __launch_bounds__(256) void glu_grad_kernel(const uint16_t* __restrict__ dH, int64_t lddh,
                                                       const uint16_t* __restrict__ G, const uint16_t* __restrict__ U,
                                                       int64_t ldg, int64_t M, int64_t R, int64_t Rp, int64_t Mp,
                                                       uint16_t* __restrict__ D, uint16_t* __restrict__ DT) {
    __shared__ PairTile tile[2];
    const int tid = threadIdx.x, c8 = tid & 7, pair = tid >> 3;
    const int64_t m0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int64_t m = m0 + 2 * pair, c = c0 + 8 * c8;
    uint32_t dg[2][8], du[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const bool ok = m + k < M;
        uint32_t h[8], g[8], u[8];
        load_row8<VEC>(dH + (m + k) * lddh, c, R, ok, h);
        load_row8<VEC>(G + (m + k) * ldg, c, R, ok, g);
        load_row8<VEC>(U + (m + k) * ldg, c, R, ok, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float hf = bf16_bits_to_f32(h[e]), gf = bf16_bits_to_f32(g[e]), uf = bf16_bits_to_f32(u[e]);
            float f, d;
            act_and_grad<ACT>(gf, f, d);
            dg[k][e] = f32_to_bf16_bits(hf * uf * d);
            du[k][e] = f32_to_bf16_bits(hf * f);
        }
        if (D && ok) {
            *(uint4*)(D + (m + k) * 2 * Rp + c) = pack8(dg[k]);
            *(uint4*)(D + (m + k) * 2 * Rp + Rp + c) = pack8(du[k]);
        }
    }
    if (!DT) return;
    tile[0].put(c8, pair, dg[0], dg[1]);
    tile[1].put(c8, pair, du[0], du[1]);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int col = (tid >> 3) + 32 * (p & 1), q = tid & 7, mat = p >> 1;
        *(uint4*)(DT + (mat * Rp + c0 + col) * Mp + m0 + 8 * q) = tile[mat].get(col, q);
    }
}

// Packed 2:4 rows -> WT [K, ldt] at columns off .. off + Rp (rows r >= R: zero).  A block
// takes 64 weight rows x 64 columns; thread (c8, pair): rows 2 pair, 2 pair + 1, the two
// groups of 4 columns from 8 c8 (4 values, one byte of positions per row).
__global__ __launch_bounds__(256) void decode_t_kernel(const uint16_t* __restrict__ vals, int64_t ldv,
                                                       const uint32_t* __restrict__ idx, int64_t ldi, int64_t R,
                                                       int64_t K, uint16_t* __restrict__ WT, int64_t ldt) {
    __shared__ PairTile tile;
    const int tid = threadIdx.x, c8 = tid & 7, pair = tid >> 3;
    const int64_t r0 = (int64_t)blockIdx.y * 64, k0 = (int64_t)blockIdx.x * 64;
    const int64_t k = k0 + 8 * c8;
    uint32_t x[2][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t r = r0 + 2 * pair + j;
        const bool ok = r < R && k < K;   // K is a multiple of 16: the thread's 8 columns are all inside or all past it
        const uint2 v = ok ? *(const uint2*)(vals + r * ldv + k / 2) : make_uint2(0, 0);
        const uint32_t b = ok ? (idx[r * ldi + k / 32] >> (8 * (c8 & 3))) & 0xffu : 0x44u;
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t v0 = w[q] & 0xffffu, v1 = w[q] >> 16;
            const uint32_t p0 = (b >> (4 * q)) & 3u, p1 = (b >> (4 * q + 2)) & 3u;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) x[j][4 * q + e] = (p0 == e ? v0 : 0u) | (p1 == e ? v1 : 0u);
        }
    }
    tile.put(c8, pair, x[0], x[1]);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int col = (tid >> 3) + 32 * p, q = tid & 7;
        if (k0 + col < K) *(uint4*)(WT + (k0 + col) * ldt + r0 + 8 * q) = tile.get(col, q);
    }
}

// ------------------------------------------------------------------ host side
static int64_t up64(int64_t n) { return (n + 63) & ~(int64_t)63; }
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace of one backward call, in the order it is carved.
struct GradWs {
    size_t d = 0, dt = 0, xt = 0, wt = 0, part = 0;
    size_t total() const { return d + dt + xt + wt + part; }
};
static GradWs grad_ws_layout(int64_t M, int64_t K, int64_t R, int nmat) {
    GradWs w;
    if (M <= 0 || K <= 0 || R <= 0) return w;
    const int64_t Rn = nmat * up64(R), Mp = up64(M);
    w.d = up256((size_t)(M * Rn * 2));
    w.dt = up256((size_t)(Rn * Mp * 2));
    w.xt = up256((size_t)(K * Mp * 2));
    w.wt = up256((size_t)(K * Rn * 2));
    w.part = up256(grad_x_part_bytes(M, K, Rn));
    return w;
}
size_t grad_ws(int64_t M, int64_t K, int64_t R, int nmat) { return grad_ws_layout(M, K, R, nmat).total(); }

template <bool VEC>
static void glu_grad_act(nm_act act, dim3 g, hipStream_t s, const GradIn& in, int64_t Rp, int64_t Mp, uint16_t* D,
                         uint16_t* DT) {
#define NM_GLU_GRAD(A)                                                                                                 \
    hipLaunchKernelGGL((glu_grad_kernel<A, VEC>), g, dim3(256), 0, s, in.dY, in.lddy, in.G, in.U, in.ldg, in.M, in.R,  \
                       Rp, Mp, D, DT)
    if (act == NM_ACT_SILU) NM_GLU_GRAD(NM_ACT_SILU);
    else if (act == NM_ACT_GELU) NM_GLU_GRAD(NM_ACT_GELU);
    else if (act == NM_ACT_GELU_TANH) NM_GLU_GRAD(NM_ACT_GELU_TANH);
    else NM_GLU_GRAD(NM_ACT_RELU2);
#undef NM_GLU_GRAD
}

static bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

// a row-major matrix of width 2-byte units set to zero (ld in bytes)
__global__ __launch_bounds__(256) void zero_rows_kernel(uint8_t* __restrict__ p, int64_t rows, int64_t width, int64_t ld) {
    const int64_t n = rows * width;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        *(uint16_t*)(p + (i / width) * ld + (i % width) * 2) = 0;
}

nm_status launch_grad(const GradIn& in, const GradOut& out, int nmat, void* ws, hipStream_t s) {
    if (in.M == 0 || in.R == 0) {
        // an empty sum: dV is zero without tokens, dX without rows
        auto zero = [&](void* p, int64_t rows, int64_t width, int64_t ld) {   // in 2-byte units
            if (p && rows > 0)
                hipLaunchKernelGGL(zero_rows_kernel, dim3(grid_cap(ceil_div(rows * width, 256), 8192)), dim3(256), 0, s,
                                   (uint8_t*)p, rows, width, ld * 2);
        };
        const int64_t vs = out.dvdt == NM_BF16 ? 1 : 2, xs = out.dxdt == NM_BF16 ? 1 : 2;
        for (int i = 0; i < nmat; ++i) zero(out.dV[i], in.R, in.K / 2 * vs, out.lddv * vs);
        zero(out.dX, in.M, in.K * xs, out.lddx * xs);
        return check_launch("backward");
    }
    const int64_t Rp = up64(in.R), Rn = nmat * Rp, Mp = up64(in.M);
    const GradWs w = grad_ws_layout(in.M, in.K, in.R, nmat);
    uint8_t* p = (uint8_t*)ws;
    uint16_t* D = (uint16_t*)p;
    uint16_t* DT = (uint16_t*)(p + w.d);
    uint16_t* XT = (uint16_t*)(p + w.d + w.dt);
    uint16_t* WT = (uint16_t*)(p + w.d + w.dt + w.xt);
    float* PART = (float*)(p + w.d + w.dt + w.xt + w.wt);
    const dim3 gd((unsigned)(Rp / 64), (unsigned)(Mp / 64));
    const uint16_t* B = D;   // the operand of dX
    int64_t ldb = Rn;
    if (nmat == 2) {
        uint16_t *d = out.dX ? D : nullptr, *dt = out.dV[0] ? DT : nullptr;
        if (rows16(in.dY, in.lddy) && rows16(in.G, in.ldg) && rows16(in.U, in.ldg))
            glu_grad_act<true>(in.act, gd, s, in, Rp, Mp, d, dt);
        else glu_grad_act<false>(in.act, gd, s, in, Rp, Mp, d, dt);
    } else {
        // dY itself where its rows are whole 64-column stages on 16-byte boundaries
        const bool vec = rows16(in.dY, in.lddy), direct = vec && in.R == Rp && in.lddy < (1 << 23);
        uint16_t *c = out.dX && !direct ? D : nullptr, *dt = out.dV[0] ? DT : nullptr;
        if (c || dt) {
            if (vec)
                hipLaunchKernelGGL(transpose_pad_kernel<true>, gd, dim3(256), 0, s, in.dY, in.lddy, in.M, in.R, dt, Mp, c, Rn);
            else
                hipLaunchKernelGGL(transpose_pad_kernel<false>, gd, dim3(256), 0, s, in.dY, in.lddy, in.M, in.R, dt, Mp, c, Rn);
        }
        if (direct) {
            B = in.dY;
            ldb = in.lddy;
        }
    }
    if (out.dX) {
        const dim3 gw((unsigned)ceil_div(in.K, 64), (unsigned)(Rp / 64));
        for (int i = 0; i < nmat; ++i)
            hipLaunchKernelGGL(decode_t_kernel, gw, dim3(256), 0, s, in.vals[i], in.ldv, in.idx[i], in.ldi, in.R, in.K,
                               WT + i * Rp, Rn);
        const nm_status st = launch_grad_x(WT, Rn, B, ldb, in.M, in.K, out.dX, out.dxdt, out.lddx, PART, s);
        if (st != NM_OK) return st;
    }
    if (out.dV[0]) {
        const dim3 gx((unsigned)ceil_div(in.K, 64), (unsigned)(Mp / 64));
        hipLaunchKernelGGL(transpose_pad_kernel<true>, gx, dim3(256), 0, s, in.X, in.ldx, in.M, in.K, XT, Mp,
                           (uint16_t*)nullptr, (int64_t)0);
        const nm_status st = launch_grad_v(XT, DT, Mp, in, out, nmat, Rp, s);
        if (st != NM_OK) return st;
    }
    return check_launch(nmat == 2 ? "nm_spmm_glu_backward" : "nm_spmm_backward");
}

}  // namespace nm
