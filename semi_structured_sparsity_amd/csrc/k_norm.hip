// The norms before and after a block with its gate and residual scale, and their gradients:
//   Z = a X + gate . norm_post(Y),  N = norm_pre(Z)
// One pass over the tokens each way, bound by memory.  A block of threads holds a token's row in
// registers (V consecutive columns a thread and vector, NV vectors), so that the statistics, Z, the second
// norm and its codes are made without reading anything again.
#include "nm_codes.h"

namespace nm {

struct NormSide {
    int kind;            // nm_norm
    const void *w, *b;
};

struct NormArgs {
    const void* X;
    int64_t ldx;
    int M, C;
    float res;
    const uint16_t* Y;
    int64_t ldyb;
    const void* gate;
    int64_t ldg;
    int gate_rows;
    NormSide post, pre;
    int w32;
    float eps;
    void* Z;
    int64_t ldz;
    void* N;
    int64_t ldn;
    int ndt, Ns;
    float* n_scale;
};

// V columns from column c of a row, as f32
template <int V>
__device__ __forceinline__ void norm_load(float (&v)[V], const void* row, bool f32, int c) {
    if constexpr (V == 8) {
        if (f32) {
            const float4* p = (const float4*)((const float*)row + c);
            const float4 a = p[0], b = p[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *(const uint4*)((const uint16_t*)row + c);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f32 ? ((const float*)row)[c + i] : bf16_bits_to_f32(((const uint16_t*)row)[c + i]);
    }
}

template <int V>
__device__ __forceinline__ void norm_store(const float (&v)[V], void* row, bool f32, int c) {
    if constexpr (V == 8) {
        if (f32) {
            float4* p = (float4*)((float*)row + c);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *(uint4*)((uint16_t*)row + c) = make_uint4(f32_to_bf16_pair(v[0], v[1]), f32_to_bf16_pair(v[2], v[3]),
                                                       f32_to_bf16_pair(v[4], v[5]), f32_to_bf16_pair(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (f32) ((float*)row)[c + i] = v[i];
            else ((uint16_t*)row)[c + i] = (uint16_t)f32_to_bf16_bits(v[i]);
        }
    }
}

// Sums over the block, the same in every thread: lanes by a butterfly, waves in order.  `turn` picks
// one of two buffers, so that one barrier a call is enough.
struct NormSum {
    float (*buf)[16][2];   // [2][waves][2]
    int turn, waves, lane, wave;
    __device__ __forceinline__ void two(float& a, float& b) {
        for (int off = 32; off; off >>= 1) {
            a += __shfl_xor(a, off);
            b += __shfl_xor(b, off);
        }
        if (waves == 1) return;
        turn ^= 1;
        if (lane == 0) {
            buf[turn][wave][0] = a;
            buf[turn][wave][1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
        for (int w = 0; w < waves; ++w) {
            a += buf[turn][w][0];
            b += buf[turn][w][1];
        }
    }
    __device__ __forceinline__ float one(float a) {
        float b = 0.0f;
        two(a, b);
        return a;
    }
    __device__ __forceinline__ float most(float a) {
        for (int off = 32; off; off >>= 1) a = __builtin_fmaxf(a, __shfl_xor(a, off));
        if (waves == 1) return a;
        turn ^= 1;
        if (lane == 0) buf[turn][wave][0] = a;
        __syncthreads();
        for (int w = 0; w < waves; ++w) a = __builtin_fmaxf(a, buf[turn][w][0]);
        return a;
    }
};

// norm of the row v in place: (v - mean) r w + b
template <int V, int NV>
__device__ __forceinline__ void norm_row(float (&v)[NV][V], const NormSide& n, bool w32, float eps, int C, int t, int nt,
                                         NormSum& sum) {
    if (n.kind == NM_NORM_NONE) return;
    const float inv = 1.0f / (float)C;
    if (n.kind == NM_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) s += v[k][i];      // columns past the end hold zeros
        const float mean = sum.one(s) * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if ((k * nt + t) * V < C) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] -= mean;
            }
    }
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) q = __builtin_fmaf(v[k][i], v[k][i], q);
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum.one(q), inv, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * nt + t) * V;
        if (c < C) {
            float w[V], b[V];
            if (n.w) norm_load<V>(w, n.w, w32, c);
            if (n.b) norm_load<V>(b, n.b, w32, c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] *= r;
                if (n.w) v[k][i] *= w[i];
                if (n.b) v[k][i] += b[i];
            }
        }
    }
}

template <int V, int NV, bool X32>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
    __shared__ float buf[2][16][2];
    extern __shared__ __attribute__((aligned(16))) uint8_t codes[];   // a row's codes, where they are lifted
    const int t = threadIdx.x, nt = blockDim.x, C = a.C;
    NormSum sum{buf, 0, nt / 64, t & 63, t >> 6};
    const int64_t m = blockIdx.x;
    float z[NV][V];
    if (a.Y) {
        float x[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) {
                norm_load<V>(z[k], a.Y + m * a.ldyb, false, c);
                norm_load<V>(x[k], (const uint8_t*)a.X + m * a.ldx * (X32 ? 4 : 2), X32, c);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] = 0.0f;
            }
        }
        norm_row<V, NV>(z, a.post, a.w32, a.eps, C, t, nt, sum);
        const uint8_t* gate = a.gate ? (const uint8_t*)a.gate + m / a.gate_rows * a.ldg * (a.w32 ? 4 : 2) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) {
                float g[V];
                if (gate) norm_load<V>(g, gate, a.w32, c);
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] = __builtin_fmaf(a.res, x[k][i], gate ? g[i] * z[k][i] : z[k][i]);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) {
                norm_load<V>(z[k], (const uint8_t*)a.X + m * a.ldx * (X32 ? 4 : 2), X32, c);
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] *= a.res;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] = 0.0f;
            }
        }
    }
    if (a.Z) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) norm_store<V>(z[k], (uint8_t*)a.Z + m * a.ldz * (X32 ? 4 : 2), X32, c);
        }
    }
    if (!a.N) return;
    norm_row<V, NV>(z, a.pre, a.w32, a.eps, C, t, nt, sum);
    if (a.ndt == NM_BF16 || a.ndt == NM_F32) {
        const bool n32 = a.ndt == NM_F32;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) norm_store<V>(z[k], (uint8_t*)a.N + m * a.ldn * (n32 ? 4 : 2), n32, c);
        }
        return;
    }
    if constexpr (V == 8) {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if ((k * nt + t) * V < C) {
#pragma unroll
                for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(z[k][i]));
            }
        top = sum.most(top);
        const bool fp8 = a.ndt == NM_FP8;
        const float s = __fdiv_rn(top, fp8 ? 448.0f : 127.0f);
        if (t == 0) a.n_scale[m] = s;
        uint8_t* out = (uint8_t*)a.N + m * a.ldn;
        const bool fast = s > 0.0f && s <= 3.0e38f;
        const RowDiv rd = row_div(fast ? s : 1.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c >= C) continue;
            uint32_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = fast ? row_quot(z[k][i], rd) : s > 0.0f ? __fdiv_rn(z[k][i], s) : 0.0f;
                if (fp8) q[i] = e4m3_code(__builtin_fminf(__builtin_fmaxf(v, -448.0f), 448.0f));
                else q[i] = (uint32_t)(int32_t)__builtin_fminf(__builtin_fmaxf(rintf(v), -127.0f), 127.0f) & 0xffu;
                if (!(s > 0.0f)) q[i] = 0;
            }
            const uint32_t lo = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, hi = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
            if (a.Ns == 0) {
                uint32_t* o = (uint32_t*)(out + c);
                o[0] = lo;
                o[1] = hi;
            } else if (a.Ns == 4) {      // a vector is a group: windows of bytes 0-3, 2-5, 4-7
                uint32_t* o = (uint32_t*)(out + c / 8 * 12);
                o[0] = lo;
                o[1] = lo >> 16 | hi << 16;
                o[2] = hi;
            } else {
                *(uint2*)(codes + c) = make_uint2(lo, hi);
            }
        }
        if (a.Ns == 0 || a.Ns == 4) return;
        __syncthreads();
        const int d = a.Ns - 1, windows = C / (2 * a.Ns) * d;
        for (int w = t; w < windows; w += nt) {
            const uint16_t* p = (const uint16_t*)(codes + 2 * (a.Ns * (w / d) + w % d));
            ((uint32_t*)out)[w] = p[0] | (uint32_t)p[1] << 16;
        }
    }
}

// ------------------------------------------------------------------ backward
struct NormBwdArgs {
    const void* Z;
    int64_t ldz;
    const void* dZ;
    int64_t lddz;
    const void* dN;
    int64_t lddn;
    int dn32;
    int M, C;
    float res;
    const uint16_t* Y;
    int64_t ldyb;
    const void* gate;
    int64_t ldg;
    int gate_rows;
    NormSide post, pre;
    int w32;
    float eps;
    void* dX;
    int64_t lddx;
    uint16_t* dY;
    int64_t lddy;
    float* sums[5];     // dw_pre, db_pre, dw_post, db_post, dgate; null: not wanted
    float* part;        // [5][blocks][C]
    int rows, blocks;   // rows of a block, blocks
    int per_gate;       // blocks of a gate row; 0: a block holds whole gate rows and writes dgate itself
};

// A block walks its rows; a thread keeps its columns, so that the parameter sums stay in its registers
// and leave once, as one partial per block.
template <int V, int NV, bool X32>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs a) {
    __shared__ float buf[2][16][2];
    const int t = threadIdx.x, nt = blockDim.x, C = a.C;
    NormSum sum{buf, 0, nt / 64, t & 63, t >> 6};
    int64_t m0, m1;
    if (a.per_gate) {
        const int64_t g = blockIdx.x / a.per_gate, k = blockIdx.x % a.per_gate;
        m0 = g * a.gate_rows + k * a.rows;
        m1 = m0 + a.rows < (g + 1) * a.gate_rows ? m0 + a.rows : (g + 1) * a.gate_rows;
    } else {
        m0 = (int64_t)blockIdx.x * a.rows;
        m1 = m0 + a.rows;
    }
    m1 = m1 < a.M ? m1 : a.M;
    const float inv = 1.0f / (float)C;
    const bool pre = a.pre.kind != NM_NORM_NONE && a.dN, post = a.post.kind != NM_NORM_NONE;
    const bool layer = (pre && a.pre.kind == NM_NORM_LAYER) || (post && a.post.kind == NM_NORM_LAYER);
    float acc[5][NV][V];
#pragma unroll
    for (int s = 0; s < 5; ++s)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[s][k][i] = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        float z[NV][V], d[NV][V], g[NV][V], y[NV][V];   // z, dn, dz, y; columns past the end hold zeros
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) z[k][i] = d[k][i] = g[k][i] = y[k][i] = 0.0f;
            if (c < C) {
                if (pre) {
                    norm_load<V>(z[k], (const uint8_t*)a.Z + m * a.ldz * (X32 ? 4 : 2), X32, c);
                    norm_load<V>(d[k], (const uint8_t*)a.dN + m * a.lddn * (a.dn32 ? 4 : 2), a.dn32, c);
                }
                if (a.dZ) norm_load<V>(g[k], (const uint8_t*)a.dZ + m * a.lddz * (X32 ? 4 : 2), X32, c);
                if (a.Y) norm_load<V>(y[k], a.Y + m * a.ldyb, false, c);
            }
        }
        // statistics of z and y together
        float s0 = 0.0f, s1 = 0.0f;
        if (layer) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s0 += z[k][i];
                    s1 += y[k][i];
                }
            sum.two(s0, s1);
            const float mz = pre && a.pre.kind == NM_NORM_LAYER ? s0 * inv : 0.0f;
            const float my = post && a.post.kind == NM_NORM_LAYER ? s1 * inv : 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * nt + t) * V < C) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        z[k][i] -= mz;
                        y[k][i] -= my;
                    }
                }
            s0 = s1 = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s0 = __builtin_fmaf(z[k][i], z[k][i], s0);
                s1 = __builtin_fmaf(y[k][i], y[k][i], s1);
            }
        sum.two(s0, s1);
        const float rz = 1.0f / __builtin_sqrtf(__builtin_fmaf(s0, inv, a.eps));
        const float ry = post ? 1.0f / __builtin_sqrtf(__builtin_fmaf(s1, inv, a.eps)) : 1.0f;
        // through norm_pre: z becomes its normalised value, d the gradient of that
        if (pre) {
            s0 = s1 = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * nt + t) * V;
                if (c < C) {
                    float w[V];
                    if (a.pre.w) norm_load<V>(w, a.pre.w, a.w32, c);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        z[k][i] *= rz;
                        acc[0][k][i] = __builtin_fmaf(d[k][i], z[k][i], acc[0][k][i]);
                        acc[1][k][i] += d[k][i];
                        if (a.pre.w) d[k][i] *= w[i];
                        s0 = __builtin_fmaf(d[k][i], z[k][i], s0);
                        s1 += d[k][i];
                    }
                }
            }
            sum.two(s0, s1);
            s0 *= inv;
            s1 = a.pre.kind == NM_NORM_LAYER ? s1 * inv : 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    g[k][i] = __builtin_fmaf(rz, d[k][i] - s1 - z[k][i] * s0, g[k][i]);
        }
        if (a.dX) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * nt + t) * V;
                if (c < C) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = a.res * g[k][i];
                    norm_store<V>(o, (uint8_t*)a.dX + m * a.lddx * (X32 ? 4 : 2), X32, c);
                }
            }
        }
        if (!a.Y) continue;
        // through the gate and norm_post: y becomes its normalised value, g the gradient of that
        const int64_t gr = m / a.gate_rows;
        s0 = s1 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) {
                float w[V], b[V], ga[V];
                if (a.post.w) norm_load<V>(w, a.post.w, a.w32, c);
                if (a.post.b && a.sums[4]) norm_load<V>(b, a.post.b, a.w32, c);
                if (a.gate) norm_load<V>(ga, (const uint8_t*)a.gate + gr * a.ldg * (a.w32 ? 4 : 2), a.w32, c);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    y[k][i] *= ry;
                    if (a.sums[4]) {
                        float u = a.post.w ? y[k][i] * w[i] : y[k][i];
                        if (a.post.b) u += b[i];
                        acc[4][k][i] = __builtin_fmaf(g[k][i], u, acc[4][k][i]);
                    }
                    if (a.gate) g[k][i] *= ga[i];
                    acc[2][k][i] = __builtin_fmaf(g[k][i], y[k][i], acc[2][k][i]);
                    acc[3][k][i] += g[k][i];
                    if (a.post.w) g[k][i] *= w[i];
                    s0 = __builtin_fmaf(g[k][i], y[k][i], s0);
                    s1 += g[k][i];
                }
            }
        }
        if (a.dY) {
            if (post) {
                sum.two(s0, s1);
                s0 *= inv;
                s1 = a.post.kind == NM_NORM_LAYER ? s1 * inv : 0.0f;
            } else {
                s0 = s1 = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * nt + t) * V;
                if (c < C) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = ry * (g[k][i] - s1 - y[k][i] * s0);
                    norm_store<V>(o, a.dY + m * a.lddy, false, c);
                }
            }
        }
        if (a.sums[4] && !a.per_gate && (m + 1 == m1 || (m + 1) / a.gate_rows != gr)) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * nt + t) * V;
                if (c < C) norm_store<V>(acc[4][k], a.sums[4] + gr * C, true, c);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[4][k][i] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 5; ++s) {
        if (!a.sums[s] || (s == 4 && !a.per_gate)) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * nt + t) * V;
            if (c < C) norm_store<V>(acc[s][k], a.part + ((int64_t)s * a.blocks + blockIdx.x) * C, true, c);
        }
    }
}

// Partial sums of the blocks added in order: 64 columns a block, 16 runs of partials side by side.
// grid: x columns, y sums (4: dgate, one z per gate row).
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormBwdArgs a, int gates) {
    __shared__ float red[16][64];
    const int s = blockIdx.y < 4 ? (int)blockIdx.y : 4, gr = blockIdx.y < 4 ? 0 : (int)blockIdx.y - 4;
    if (!a.sums[s]) return;
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), run = threadIdx.x >> 6;
    const int first = s == 4 ? gr * a.per_gate : 0, count = s == 4 ? a.per_gate : a.blocks;
    const int per = (count + 15) / 16, b0 = run * per, b1 = b0 + per < count ? b0 + per : count;
    float v = 0.0f;
    if (c < a.C) {
        const float* p = a.part + ((int64_t)s * a.blocks + first) * a.C + c;
#pragma unroll 8
        for (int b = b0; b < b1; ++b) v += p[(int64_t)b * a.C];
    }
    red[run][threadIdx.x & 63] = v;
    __syncthreads();
    if (run || c >= a.C) return;
    for (int i = 1; i < 16; ++i) v += red[i][threadIdx.x];
    a.sums[s][(int64_t)gr * a.C + c] = v;
}

// ------------------------------------------------------------------ host
static bool aligned_rows(const void* p, int64_t ld, int64_t es) {
    return !p || (((uintptr_t)p & 15u) == 0 && ld * es % 16 == 0);
}

// threads of a block for V columns a vector and NV vectors a thread
static int norm_threads(int C, int V, int NV) {
    const int t = (int)ceil_div(C, V * NV);
    return (t + 63) / 64 * 64;
}

template <int V, int NV>
static void norm_go(const NormArgs& a, bool x32, hipStream_t s) {
    const dim3 grid((unsigned)a.M), block((unsigned)norm_threads(a.C, V, NV));
    const size_t lds = a.Ns && a.Ns != 4 ? (size_t)a.C : 0;
    if (x32) hipLaunchKernelGGL((norm_kernel<V, NV, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((norm_kernel<V, NV, false>), grid, block, lds, s, a);
}

nm_status launch_block_norm(const NormIn& in, hipStream_t s) {
    NormArgs a{};
    const int64_t xs = in.xdt == NM_F32 ? 4 : 2, wsz = in.wdt == NM_F32 ? 4 : 2;
    a.X = in.X;
    a.ldx = in.ldx;
    a.M = (int)in.Mtok;
    a.C = (int)in.C;
    a.res = in.res_scale;
    a.Y = (const uint16_t*)in.Y;
    a.ldyb = in.ldyb;
    a.gate = in.gate;
    a.ldg = in.ldg;
    a.gate_rows = (int)(in.gate_rows > 0 && in.gate_rows < in.Mtok ? in.gate_rows : in.Mtok);
    a.post = {in.post, in.w_post, in.b_post};
    a.pre = {in.pre, in.w_pre, in.b_pre};
    a.w32 = in.wdt == NM_F32;
    a.eps = in.eps;
    a.Z = in.Z;
    a.ldz = in.ldz;
    a.N = in.N;
    a.ldn = in.ldn;
    a.ndt = in.ndt;
    a.Ns = in.Ns;
    a.n_scale = in.n_scale;
    const bool code = in.ndt == NM_I8 || in.ndt == NM_FP8;
    const bool vec = in.C % 8 == 0 && aligned_rows(in.X, in.ldx, xs) && aligned_rows(in.Y, in.ldyb, 2) &&
                     aligned_rows(in.gate, in.ldg, wsz) && aligned_rows(in.Z, in.ldz, xs) && aligned_rows(in.w_post, 8, 2) &&
                     aligned_rows(in.b_post, 8, 2) && aligned_rows(in.w_pre, 8, 2) && aligned_rows(in.b_pre, 8, 2) &&
                     (code || aligned_rows(in.N, in.ldn, in.ndt == NM_F32 ? 4 : 2));
    const bool x32 = in.xdt == NM_F32;
    if (vec) {
        if (in.C <= 8192) norm_go<8, 1>(a, x32, s);
        else if (in.C <= 16384) norm_go<8, 2>(a, x32, s);
        else norm_go<8, 4>(a, x32, s);
    } else if (code) {
        return set_error(NM_ERR_ALIGN, "nm_block_norm: codes need 16-byte aligned rows of the inputs and Z");
    } else {
        if (in.C <= 4096) norm_go<1, 4>(a, x32, s);
        else norm_go<1, 32>(a, x32, s);
    }
    return check_launch("nm_block_norm");
}

// rows of a block and how gate rows fall on blocks
struct NormPlan {
    int rows, blocks, per_gate, gates;
};
static NormPlan norm_plan(int64_t M, int64_t gate_rows) {
    NormPlan p{};
    const int64_t gr = gate_rows > 0 && gate_rows < M ? gate_rows : (M > 0 ? M : 1);
    const int64_t want = M / 512 > 4 ? M / 512 : 4;   // rows a block
    p.gates = (int)(M > 0 ? ceil_div(M, gr) : 1);
    if (gr <= want) {
        p.rows = (int)(want / gr * gr);
        p.blocks = (int)ceil_div(M, p.rows);
    } else {
        p.per_gate = (int)ceil_div(gr, want);
        p.rows = (int)ceil_div(gr, p.per_gate);
        p.blocks = p.gates * p.per_gate;
    }
    return p;
}

size_t block_norm_bwd_ws(int64_t M, int64_t C, int64_t gate_rows) {
    return (size_t)norm_plan(M, gate_rows).blocks * (size_t)C * 5 * 4;
}

template <int V, int NV>
static void norm_bwd_go(const NormBwdArgs& a, bool x32, hipStream_t s) {
    const dim3 grid((unsigned)a.blocks), block((unsigned)norm_threads(a.C, V, NV));
    if (x32) hipLaunchKernelGGL((norm_bwd_kernel<V, NV, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((norm_bwd_kernel<V, NV, false>), grid, block, 0, s, a);
}

nm_status launch_block_norm_bwd(const NormBwdIn& in, void* ws, hipStream_t s) {
    NormBwdArgs a{};
    const int64_t xs = in.xdt == NM_F32 ? 4 : 2, wsz = in.wdt == NM_F32 ? 4 : 2;
    const NormPlan p = norm_plan(in.Mtok, in.gate_rows);
    a.Z = in.Z;
    a.ldz = in.ldz;
    a.dZ = in.dZ;
    a.lddz = in.lddz;
    a.dN = in.dN;
    a.lddn = in.lddn;
    a.dn32 = in.dndt == NM_F32;
    a.M = (int)in.Mtok;
    a.C = (int)in.C;
    a.res = in.res_scale;
    a.Y = (const uint16_t*)in.Y;
    a.ldyb = in.ldyb;
    a.gate = in.gate;
    a.ldg = in.ldg;
    a.gate_rows = (int)(in.gate_rows > 0 && in.gate_rows < in.Mtok ? in.gate_rows : (in.Mtok > 0 ? in.Mtok : 1));
    a.post = {in.post, in.w_post, in.b_post};
    a.pre = {in.pre, in.w_pre, nullptr};
    a.w32 = in.wdt == NM_F32;
    a.eps = in.eps;
    a.dX = in.dX;
    a.lddx = in.lddx;
    a.dY = (uint16_t*)in.dY;
    a.lddy = in.lddy;
    bool sums = false;
    for (int i = 0; i < 5; ++i) {
        a.sums[i] = in.sums[i];
        sums |= in.sums[i] != nullptr;
    }
    a.part = (float*)ws;
    a.rows = p.rows;
    a.blocks = p.blocks;
    a.per_gate = p.per_gate;
    const bool x32 = in.xdt == NM_F32;
    if (in.Mtok > 0) {
        const bool vec = in.C % 8 == 0 && aligned_rows(in.Z, in.ldz, xs) && aligned_rows(in.dZ, in.lddz, xs) &&
                         aligned_rows(in.dN, in.lddn, in.dndt == NM_F32 ? 4 : 2) && aligned_rows(in.Y, in.ldyb, 2) &&
                         aligned_rows(in.gate, in.ldg, wsz) && aligned_rows(in.dX, in.lddx, xs) && aligned_rows(in.dY, in.lddy, 2) &&
                         aligned_rows(in.w_post, 8, 2) && aligned_rows(in.b_post, 8, 2) && aligned_rows(in.w_pre, 8, 2) &&
                         aligned_rows(in.sums[4], in.C, 4);
        if (vec) {
            if (in.C <= 8192) norm_bwd_go<8, 1>(a, x32, s);
            else if (in.C <= 16384) norm_bwd_go<8, 2>(a, x32, s);
            else norm_bwd_go<8, 4>(a, x32, s);
        } else {
            if (in.C <= 4096) norm_bwd_go<1, 4>(a, x32, s);
            else norm_bwd_go<1, 32>(a, x32, s);
        }
    }
    // without tokens every sum is of no partials; whole gate rows of a block are written by it
    if (sums) {
        const bool reduce_gate = in.sums[4] && (p.per_gate > 0 || in.Mtok == 0);
        hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)ceil_div(in.C, 64), (unsigned)(reduce_gate ? 4 + p.gates : 4)), dim3(1024),
                           0, s, a, p.gates);
    }
    return check_launch("nm_block_norm_backward");
}

}  // namespace nm
