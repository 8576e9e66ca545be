// A mixture-of-experts layer of sparse gated blocks for a few tokens, in three launches:
//   moe_logits_kernel  router logits (dense MFMA), K split over blocks, partials in f32
//   moe_up_kernel      every block picks the experts of all tokens for itself from the logits (no
//                      launch between), then H = act(x Wg^T) . (x Wu^T) of one expert's 16 features
//   moe_down_kernel    Y: a block owns output columns and adds up, for them, every picked expert's
//                      product in a fixed order
// An expert's tokens are gathered by lane in the activation's loads (16 at a time are the B
// operand); its weight is streamed as in the 4-bit products (nm_few.h).
#include "nm_few.h"

namespace nm {

constexpr int kMoeTokens = 64, kMoeTopk = 16, kMoeExperts = 512;

struct MoeArgs {
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* router;
    int64_t ldr;
    const float* bias;
    int T, K, F, E, topk, sigmoid, renorm, Ns, wK, wF, gshift, act, ksplit;
    float route_scale;
    nm_experts w[3];       // gate, up, down; ld_vals and es_vals in bytes
    float* logits;         // [ksplit][T][E]
    uint16_t* H;           // [T * topk, ldh]
    int64_t ldh;
    int32_t* sel;          // [T, topk]
    float* wts;
    int32_t* sel_out;
    float* wts_out;
    void* Y;
    int64_t ldy;
    int y32;
};

// ------------------------------------------------------------------ router
typedef short moe_s16x8 __attribute__((ext_vector_type(8)));

// Logits of 16 experts (rows of A) and 16 tokens (columns of B) over one K split: four waves take
// 32-column steps in turn, summed through LDS in wave order.
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float red[4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    const int e = e0 + (lane & 15), t = t0 + (lane & 15), q = lane >> 4;
    const uint16_t* wr = a.router + (int64_t)(e < a.E ? e : a.E - 1) * a.ldr;
    const uint16_t* xr = a.X + (int64_t)(t < a.T ? t : a.T - 1) * a.ldx;
    const int steps = (a.K + 31) / 32, per = (steps + a.ksplit - 1) / a.ksplit;
    const int s0 = blockIdx.z * per, s1 = s0 + per < steps ? s0 + per : steps;
    few_f32x4 acc = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = s0 + wave; s < s1; s += 4) {
        const int col = 32 * s + 8 * q;
        uint4 w = make_uint4(0, 0, 0, 0), x = w;
        if (col < a.K) {
            w = *(const uint4*)(wr + col);
            x = *(const uint4*)(xr + col);
        }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(few_bf16x8, w), __builtin_bit_cast(few_bf16x8, x), acc, 0,
                                                      0, 0);
    }
    *(few_f32x4*)&red[wave][lane * 4] = acc;
    __syncthreads();
    const int k = threadIdx.x;   // lane k / 4's accumulator k % 4
    const int tt = t0 + ((k >> 2) & 15), ee = e0 + 4 * (k >> 6) + (k & 3);
    if (tt < a.T && ee < a.E)
        a.logits[((int64_t)blockIdx.z * a.T + tt) * a.E + ee] = (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
}

// The topk experts of token t and their weights, by one wave: sel[0 .. topk), wts[0 .. topk).
// Lane l holds experts l, l + 64, ...
template <int NE>
__device__ __forceinline__ void moe_pick(const MoeArgs& a, int t, int lane, int32_t* sel, float* wts) {
    float l[NE];
    double key[NE];
    const double none = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        l[i] = 0.0f;
        key[i] = none;
        if (e < a.E) {
            l[i] = split_sum(a.logits + (int64_t)t * a.E + e, a.ksplit, (int64_t)a.T * a.E);
        }
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (lane + 64 * i < a.E) top = __builtin_fmaxf(top, l[i]);
    for (int off = 32; off; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
    float p[NE], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const bool in = lane + 64 * i < a.E;
        p[i] = !in ? 0.0f : a.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - top);
        sum += p[i];
    }
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        if (!a.sigmoid) p[i] = p[i] / sum;
        if (e < a.E) {
            // with a bias two probabilities may lie closer than f32 tells apart
            if (a.bias)
                key[i] = (a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top) / (double)sum) +
                         (double)a.bias[e];
            else
                key[i] = (double)l[i];
            if (!(key[i] == key[i])) key[i] = none;
        }
    }
    uint32_t taken = 0;   // of this lane's experts
    float total = 0.0f, mine = 0.0f;
    int my_sel = 0;
    for (int j = 0; j < a.topk; ++j) {
        double best = none;
        int at = 1 << 30;
        float bp = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E && !(taken >> i & 1) && (at == 1 << 30 || key[i] > best)) {
                best = key[i];
                at = e;
                bp = p[i];
            }
        }
        for (int off = 32; off; off >>= 1) {
            const double ob = __shfl_xor(best, off);
            const int oa = __shfl_xor(at, off);
            const float op = __shfl_xor(bp, off);
            const bool other = at == 1 << 30 ? oa != 1 << 30 : oa != 1 << 30 && (ob > best || (ob == best && oa < at));
            if (other) {
                best = ob;
                at = oa;
                bp = op;
            }
        }
        if ((at & 63) == lane) taken |= 1u << (at >> 6);
        total += bp;
        if (lane == j) {
            my_sel = at;
            mine = bp;
        }
    }
    if (lane < a.topk) {
        sel[lane] = my_sel;
        wts[lane] = a.route_scale * (a.renorm ? mine / total : mine);
    }
}

// ------------------------------------------------------------------ gate and up
// grid: x feature tiles of 16, y picked experts.  A block finds the experts of all tokens, takes the
// y-th picked one (in order of the expert's number) and its (token, slot) pairs in order.
template <int NE>
__device__ __forceinline__ void moe_route(const MoeArgs& a, int32_t* sel, float* wts, int tid, int nw) {
    const int lane = tid & 63, wave = tid >> 6;
    for (int t = wave; t < a.T; t += nw) moe_pick<NE>(a, t, lane, sel + t * a.topk, wts + t * a.topk);
    __syncthreads();
}

// the n-th (from 0) expert of those in sel[0 .. pairs), by number, or -1; one wave's lanes all get it
__device__ __forceinline__ int moe_nth(const uint64_t (&used)[kMoeExperts / 64], int n) {
    for (int i = 0; i < kMoeExperts / 64; ++i) {
        uint64_t m = used[i];
        const int c = __popcll(m);
        if (n >= c) {
            n -= c;
            continue;
        }
        for (; n; --n) m &= m - 1;
        return 64 * i + __ffsll((unsigned long long)m) - 1;
    }
    return -1;
}

template <int VT, int SPG, int NW>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float red[NW][2][256];
    __shared__ int32_t sel[kMoeTokens * kMoeTopk];
    __shared__ float wts[kMoeTokens * kMoeTopk];
    __shared__ uint64_t used[kMoeExperts / 64];
    __shared__ int16_t list[kMoeTokens * kMoeTopk];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid < kMoeExperts / 64) used[tid] = 0;
    if (a.E <= 64) moe_route<1>(a, sel, wts, tid, NW);
    else if (a.E <= 128) moe_route<2>(a, sel, wts, tid, NW);
    else if (a.E <= 256) moe_route<4>(a, sel, wts, tid, NW);
    else moe_route<8>(a, sel, wts, tid, NW);
    const int pairs = a.T * a.topk;
    for (int p = tid; p < pairs; p += NW * 64) {
        atomicOr((unsigned long long*)&used[sel[p] >> 6], 1ull << (sel[p] & 63));
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            a.sel[p] = sel[p];
            a.wts[p] = wts[p];
            if (a.sel_out) a.sel_out[p] = sel[p];
            if (a.wts_out) a.wts_out[p] = wts[p];
        }
    }
    __syncthreads();
    const int e = moe_nth(used, blockIdx.y);
    if (e < 0) return;
    if (wave == 0) {
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const bool hit = p0 + lane < pairs && sel[p0 + lane] == e;
            const uint64_t m = __ballot(hit);
            if (hit) list[n + __popcll(m & ((1ull << lane) - 1))] = (int16_t)(p0 + lane);
            n += __popcll(m);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    FewRows w[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
        w[m] = few_rows((const uint8_t*)a.w[m].vals + e * a.w[m].es_vals, a.w[m].idx + e * a.w[m].es_idx,
                        (const uint16_t*)a.w[m].scales + e * a.w[m].es_scales, a.w[m].ld_vals, a.w[m].ld_idx, a.w[m].ld_scales,
                        f0, a.F, lane);
    for (int c = 0; c < n; c += 16) {
        const int i = c + (lane & 15) < n ? c + (lane & 15) : n - 1;
        const uint16_t* xrow[1] = {a.X + (int64_t)(list[i] / a.topk) * a.ldx};
        few_f32x4 acc[2][1] = {{few_f32x4{0, 0, 0, 0}}, {few_f32x4{0, 0, 0, 0}}};
        few_product<VT, SPG, 2, 1>(w, xrow, wave, NW, (a.wK + 255) / 256, a.wK, a.gshift, a.Ns, lane, acc);
        if (c) __syncthreads();
        *(few_f32x4*)&red[wave][0][lane * 4] = acc[0][0];
        *(few_f32x4*)&red[wave][1][lane * 4] = acc[1][0];
        __syncthreads();
        if (tid < 256) {
            const int k = c + ((tid >> 2) & 15);
            const int64_t f = f0 + 4 * (tid >> 6) + (tid & 3);
            if (k < n && f < a.F) {
                float g = 0.0f, u = 0.0f;
#pragma unroll
                for (int v = 0; v < NW; ++v) {
                    g += red[v][0][tid];
                    u += red[v][1][tid];
                }
                a.H[(int64_t)list[k] * a.ldh + f] = (uint16_t)f32_to_bf16_bits(few_act(a.act, g) * u);
            }
        }
    }
}

// ------------------------------------------------------------------ down
// grid: x tiles of 16 output columns.  Wave work items are (picked expert, slice of its width); a
// pair's partial sums stay in LDS per slice, weighted, and are added up token by token.
template <int VT, int SPG, int NW>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeArgs a, int slices) {
    extern __shared__ __attribute__((aligned(16))) float part[];   // [slices][pairs][16]
    __shared__ int32_t sel[kMoeTokens * kMoeTopk];
    __shared__ uint64_t used[kMoeExperts / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.topk;
    if (tid < kMoeExperts / 64) used[tid] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += NW * 64) {
        const int s = a.sel[p];
        sel[p] = s;
        atomicOr((unsigned long long*)&used[s >> 6], 1ull << (s & 63));
    }
    __syncthreads();
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    const int units = (a.wF + 255) / 256;
    for (int item = wave;; item += NW) {
        const int e = moe_nth(used, item / slices), sl = item % slices;
        if (e < 0) break;
        const FewRows w[1] = {few_rows((const uint8_t*)a.w[2].vals + e * a.w[2].es_vals, a.w[2].idx + e * a.w[2].es_idx,
                                       (const uint16_t*)a.w[2].scales + e * a.w[2].es_scales, a.w[2].ld_vals, a.w[2].ld_idx,
                                       a.w[2].ld_scales, r0, a.K, lane)};
        // the expert's pairs, 16 at a time: lane k of 16 has the k-th from the position reached
        int p0 = 0;
        while (p0 < pairs) {
            int mine = -1, n = 0, at = p0;
            for (; at < pairs && n < 16; at += 64) {
                uint64_t m = __ballot(at + lane < pairs && sel[at + lane < pairs ? at + lane : 0] == e);
                while (m && n < 16) {
                    const int b = __ffsll((unsigned long long)m) - 1;
                    m &= m - 1;
                    if ((lane & 15) == n) mine = at + b;
                    p0 = at + b + 1;
                    ++n;
                }
                if (m) break;
            }
            if (n < 16) p0 = pairs;
            if (n == 0) break;
            const bool real = mine >= 0;
            const int first = __shfl(mine, 0);
            const uint16_t* xrow[1] = {a.H + (int64_t)(real ? mine : first) * a.ldh};
            few_f32x4 acc[1][1] = {{few_f32x4{0, 0, 0, 0}}};
            few_product<VT, SPG, 1, 1>(w, xrow, sl, slices, units, a.wF, a.gshift, a.Ns, lane, acc);
            if (real) {
                const float wt = a.wts[mine];
                few_f32x4 v = acc[0][0];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] *= wt;
                *(few_f32x4*)&part[((int64_t)sl * pairs + mine) * 16 + 4 * (lane >> 4)] = v;
            }
        }
    }
    __syncthreads();
    for (int o = tid; o < a.T * 16; o += NW * 64) {
        const int t = o >> 4, r = o & 15;
        if (r0 + r >= a.K) continue;
        float v = 0.0f;
        for (int j = 0; j < a.topk; ++j)
            for (int s = 0; s < slices; ++s) v += part[((int64_t)s * pairs + t * a.topk + j) * 16 + r];
        if (a.y32) ((float*)a.Y)[t * a.ldy + r0 + r] = v;
        else ((uint16_t*)a.Y)[t * a.ldy + r0 + r] = (uint16_t)f32_to_bf16_bits(v);
    }
}

// ------------------------------------------------------------------ host
constexpr int kMoeWaves = 16, kMoeSplit = 8;

static int moe_ksplit(int64_t T, int64_t K, int E) {
    // blocks of the router's product: enough of them that each reads a few KB
    const int64_t tiles = ceil_div(E, 16) * ceil_div(T, 16);
    int64_t s = ceil_div(K, 512);
    if (s > kMoeSplit) s = kMoeSplit;
    while (s > 1 && tiles * s > 512) s /= 2;
    return (int)(s < 1 ? 1 : s);
}

size_t moe_ws(int64_t T, int64_t K, int64_t F, int E, int topk) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    return up((size_t)kMoeSplit * T * E * 4) + up((size_t)T * topk * ((F + 7) / 8 * 8) * 2) + 2 * up((size_t)T * topk * 4);
}

template <int VT, int SPG>
static nm_status moe_go(const MoeArgs& a, hipStream_t s) {
    const int pairs = a.T * a.topk, picked = pairs < a.E ? pairs : a.E;
    hipLaunchKernelGGL(moe_logits_kernel, dim3((a.E + 15) / 16, (a.T + 15) / 16, a.ksplit), dim3(256), 0, s, a);
    hipLaunchKernelGGL((moe_up_kernel<VT, SPG, kMoeWaves>), dim3((a.F + 15) / 16, picked), dim3(kMoeWaves * 64), 0, s, a);
    // slices of an expert's width: so many that every wave of a block has one where few experts are
    // picked, as long as the partial sums fit
    int slices = (kMoeWaves + picked - 1) / picked;
    const int units = (a.wF + 255) / 256;
    if (slices > units) slices = units;
    while (slices > 1 && slices * pairs > 1024) --slices;
    hipLaunchKernelGGL((moe_down_kernel<VT, SPG, kMoeWaves>), dim3((a.K + 15) / 16), dim3(kMoeWaves * 64),
                       (size_t)slices * pairs * 64, s, a, slices);
    return check_launch("nm_moe");
}

nm_status launch_moe(const MoeIn& in, void* ws, hipStream_t s) {
    MoeArgs a{};
    a.X = (const uint16_t*)in.X;
    a.ldx = in.ldx;
    a.router = (const uint16_t*)in.router;
    a.ldr = in.ldr;
    a.bias = in.bias;
    a.T = (int)in.Mtok;
    a.K = (int)in.K;
    a.F = (int)in.F;
    a.E = in.E;
    a.topk = in.topk;
    a.sigmoid = in.route == NM_ROUTE_SIGMOID;
    a.renorm = in.renorm;
    a.route_scale = in.route_scale;
    a.Ns = in.Ns;
    a.wK = (int)(in.Ns ? in.K / (2 * in.Ns) * 4 * (in.Ns - 1) : in.K);
    a.wF = (int)(in.Ns ? in.F / (2 * in.Ns) * 4 * (in.Ns - 1) : in.F);
    a.gshift = in.group == 64 ? 6 : in.group == 128 ? 7 : 8;
    a.act = in.act;
    a.ksplit = moe_ksplit(in.Mtok, in.K, in.E);
    for (int m = 0; m < 3; ++m) {
        a.w[m] = in.w[m];
        if (in.vdt == NM_BF16) {
            a.w[m].ld_vals *= 2;
            a.w[m].es_vals *= 2;
            a.w[m].scales = nullptr;
        }
    }
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    uint8_t* p = (uint8_t*)ws;
    a.logits = (float*)p;
    p += up((size_t)kMoeSplit * in.Mtok * in.E * 4);
    a.ldh = (in.F + 7) / 8 * 8;
    a.H = (uint16_t*)p;
    p += up((size_t)in.Mtok * in.topk * a.ldh * 2);
    a.sel = (int32_t*)p;
    p += up((size_t)in.Mtok * in.topk * 4);
    a.wts = (float*)p;
    a.sel_out = in.sel;
    a.wts_out = in.wts;
    a.Y = in.Y;
    a.ldy = in.ldy;
    a.y32 = in.ydt == NM_F32;
    if (in.vdt == NM_BF16) return moe_go<kFewBF16, 1>(a, s);
    if (in.vdt == NM_I4) return a.gshift == 6 ? moe_go<kFewI4, 1>(a, s) : a.gshift == 7 ? moe_go<kFewI4, 2>(a, s) : moe_go<kFewI4, 4>(a, s);
    return a.gshift == 6 ? moe_go<kFewFP4, 1>(a, s) : a.gshift == 7 ? moe_go<kFewFP4, 2>(a, s) : moe_go<kFewFP4, 4>(a, s);
}

}  // namespace nm
