// few.cu -- the whole layer for a few tokens (at most FEW_MAX_T).
//
// A batch this small is one pass over the weights of the experts it hits.  The
// hidden units of those experts, laid end to end (experts ascending, then the
// shared one), are cut into equal parts; a CTA computes H = g silu(x w1) (x w3)
// for its part, keeps it in shared memory and multiplies it straight away by
// the columns of w2 that belong to it.  Gate/up and down so run without a
// grid-wide step between them, and each CTA streams the same bytes whatever
// the routing.  What a part adds to a token's output goes to a row of its own
// in the workspace; the combine adds a token's rows in a fixed order, so the
// result does not depend on which CTA finished first.
#include <math.h>

#include "common.cuh"
#include "few.h"
#include "kernels.h"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int FT = FEW_MAX_T;
constexpr int THREADS = 256;

// The routing of the batch, worked out by every CTA for itself (128
// assignments at most) in shared memory.
struct Routing {
    int32_t sel[FT * MAX_K];        // [t * k + j] expert
    float g[FT * MAX_K];            // its gate
    int32_t lead[FT * MAX_K];       // 1: the batch's first assignment to its expert
    int32_t item_of[FT * MAX_K];    // item of the assignment
    int32_t pos_of[FT * MAX_K];     // its place in the item's token list, -1 if dropped
    int32_t items;                  // hit experts + the shared one
    int32_t expert[FEW_MAX_ITEMS];  // expert of an item, -1: shared
    int32_t n[FEW_MAX_ITEMS];       // tokens it serves
    int32_t row0[FEW_MAX_ITEMS];    // first row of its partial outputs
    uint8_t tok[FEW_MAX_ITEMS][FT];
    float gate[FEW_MAX_ITEMS][FT];
    int64_t tot;                    // granules of all items
    int V;                          // parts
};

// Part that holds granule x (the parts' bounds are v tot / V rounded down).
__device__ __forceinline__ int part_of(int64_t x, int64_t tot, int V) {
    return (int)(((x + 1) * V - 1) / tot);
}

__device__ __forceinline__ int64_t item_start(int i, int A, int gE) { return (int64_t)min(i, A) * gE; }

// Top-k and gates of one token by one warp: each lane keeps the k best of its
// experts, k rounds of an arg-max over the lanes' best merge them.
__device__ void route_token(const FewArgs& a, int t, Routing& r) {
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k;
    const float* z = a.logits + (int64_t)t * E;
    float lv[MAX_K];
    int li[MAX_K];
#pragma unroll
    for (int j = 0; j < MAX_K; ++j) {
        lv[j] = -INFINITY;
        li[j] = -1;
    }
    for (int e = lane; e < E; e += 32)
        topk_insert(lv, li, k, finite_or_minus_inf(a.bias ? z[e] + a.bias[e] : z[e]), e);
    float vs[MAX_K];
    int is[MAX_K];
#pragma unroll
    for (int j = 0; j < MAX_K; ++j) {
        vs[j] = -INFINITY;
        is[j] = 0;
        if (j >= k) continue;
        float bv = lv[0];
        int bi = li[0] < 0 ? 0x7fffffff : li[0];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        vs[j] = bv;
        is[j] = bi;
        if (li[0] == bi) {
#pragma unroll
            for (int q = 0; q < MAX_K - 1; ++q) {
                lv[q] = lv[q + 1];
                li[q] = li[q + 1];
            }
            lv[MAX_K - 1] = -INFINITY;
            li[MAX_K - 1] = -1;
        }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < MAX_K; ++j)
        if (j < k) s += expf(vs[j] - vs[0]);
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < MAX_K; ++j)
            if (j < k) {
                r.sel[t * k + j] = is[j];
                r.g[t * k + j] = expf(vs[j] - vs[0]) / s;
            }
    }
}

// Fills r: capacity in token order, the hit experts ascending with their
// tokens and gates, the shared expert last, and the rows of the partial
// outputs.  Called by every thread of the CTA.
__device__ void route_batch(const FewArgs& a, Routing& r) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    const int N = a.T * a.k, k = a.k;
    for (int t = tid >> 5; t < a.T; t += nthr >> 5) route_token(a, t, r);
    __syncthreads();
    for (int i = tid; i < N; i += nthr) {
        int before = 0;
        for (int b = 0; b < i; ++b) before += r.sel[b] == r.sel[i];
        r.lead[i] = before == 0;
        r.pos_of[i] = before < a.C ? before : -1;
    }
    __syncthreads();
    for (int i = tid; i < N; i += nthr) {
        int at = 0, count = 0;
        for (int b = 0; b < N; ++b) {
            at += r.lead[b] && r.sel[b] < r.sel[i];
            count += r.sel[b] == r.sel[i];
        }
        r.item_of[i] = at;
        if (r.lead[i]) {
            r.expert[at] = r.sel[i];
            r.n[at] = (int)min((int64_t)count, a.C);
        }
        const int p = r.pos_of[i];
        if (p >= 0) {
            r.tok[at][p] = (uint8_t)(i / k);
            r.gate[at][p] = r.g[i];
        }
    }
    int A = 0;
    for (int b = 0; b < N; ++b) A += r.lead[b];
    if (tid < a.T && a.hsum > 0) {
        r.tok[A][tid] = (uint8_t)tid;
        r.gate[A][tid] = 1.0f;
    }
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int64_t tot = (int64_t)A * gE + gS;
    const int V = few_parts(tot, gridDim.x);
    if (tid == 0) {
        if (gS) {
            r.expert[A] = -1;
            r.n[A] = a.T;
        }
        r.items = A + (gS > 0);
        r.tot = tot;
        r.V = V;
    }
    __syncthreads();
    // exclusive prefix over the items of tokens x parts
    if (tid < 32) {
        const int per = (FEW_MAX_ITEMS + 31) / 32;
        int mine = 0;
        for (int q = 0; q < per; ++q) {
            const int i = tid * per + q;
            if (i < r.items) {
                const int64_t s = item_start(i, A, gE), e = s + (i < A ? gE : gS);
                mine += r.n[i] * (part_of(e - 1, tot, V) - part_of(s, tot, V) + 1);
            }
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (tid >= o) incl += v;
        }
        int at = incl - mine;
        for (int q = 0; q < per; ++q) {
            const int i = tid * per + q;
            if (i < r.items) {
                const int64_t s = item_start(i, A, gE), e = s + (i < A ? gE : gS);
                r.row0[i] = at;
                at += r.n[i] * (part_of(e - 1, tot, V) - part_of(s, tot, V) + 1);
            }
        }
    }
    __syncthreads();
}

// The routing outputs and the combine's table (written by one CTA).
__device__ void publish_routing(const FewArgs& a, const Routing& r) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    const int N = a.T * a.k, k = a.k;
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int A = r.items - (gS > 0);
    for (int e = tid; e < a.E; e += nthr) {
        int routed = 0;
        for (int b = 0; b < N; ++b) routed += r.sel[b] == e;
        a.routed[e] = routed;
        a.kept[e] = (int)min((int64_t)routed, a.C);
    }
    for (int i = tid; i < N + a.T; i += nthr) {
        const bool shared = i >= N;
        const int t = shared ? i - N : i / k;
        const int item = shared ? A : r.item_of[i], pos = shared ? t : r.pos_of[i];
        int4 row = make_int4(0, 0, 0, 0);
        if (pos >= 0 && !(shared && gS == 0)) {
            const int64_t s = item_start(item, A, gE), e = s + (shared ? gS : gE);
            row.x = r.row0[item] + pos;
            row.y = part_of(e - 1, r.tot, r.V) - part_of(s, r.tot, r.V) + 1;
            row.z = r.n[item];
        }
        a.table[t * (k + 1) + (shared ? k : i % k)] = row;
        if (!shared) {
            a.topk_idx[i] = r.sel[i];
            a.topk_gate[i] = r.g[i];
        }
    }
}

// ---------------------------------------------------------------- weights, element by element

__device__ __forceinline__ float q4_code(uint32_t word, int nibble) {
    return (float)((int)((word >> (4 * nibble)) & 15u) - 8);
}

// Packed gate (up = 0) or up (up = 1) weight of hidden unit j at column c.
__device__ float w13_at(const FewArgs& a, int expert, int j, int up, int c) {
    const bool shared = expert < 0;
    const int hid = shared ? a.hsum : a.h, e = shared ? 0 : expert, d = a.d;
    const void* W = shared ? a.w13s : a.w13;
    if (a.G == 0) {
        const int64_t row = (int64_t)e * 2 * hid + 256 * (j / 128) + 128 * up + j % 128;
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(W)[row * d + c]);
    }
    const int n = shared ? 1 : a.E;
    const int64_t blk = ((int64_t)e * (hid / 8) + j / 8) * (d / 128) + c / 128;
    const int kk = c % 128, s = kk / 16, q = kk % 16, gq = j % 8;
    const int reg = 2 * (q / 8) + up, t = (q % 8) / 2, lane = gq * 4 + t;
    const uint32_t word = reinterpret_cast<const uint32_t*>(
        W)[blk * 256 + (s / 4) * 128 + lane * 4 + s % 4];
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(
        reinterpret_cast<const uint8_t*>(W) + q13_code_bytes(n, hid, d));
    return q4_code(word, reg + 4 * (q & 1)) *
           __bfloat162float(sc[(blk * (128 / a.G) + kk / a.G) * 16 + up * 8 + gq]);
}

// Down weight of output column c and hidden unit j.
__device__ float w2_at(const FewArgs& a, int expert, int c, int j) {
    const bool shared = expert < 0;
    const int hid = shared ? a.hsum : a.h, e = shared ? 0 : expert, d = a.d;
    const void* W = shared ? a.w2s : a.w2;
    if (a.G == 0)
        return __bfloat162float(
            reinterpret_cast<const __nv_bfloat16*>(W)[((int64_t)e * d + c) * hid + j]);
    const int n = shared ? 1 : a.E;
    const int64_t rb = (int64_t)e * (d / 128) + c / 128;
    const int rr = c % 128, tile = rr / 16, s = (j % 32) / 16, q = j % 16;
    const int reg = 2 * (q / 8) + (rr % 16) / 8, lane = (rr % 8) * 4 + (q % 8) / 2;
    const uint32_t word = reinterpret_cast<const uint32_t*>(
        W)[((rb * (hid / 32) + j / 32) * 8 + tile) * 64 + lane * 2 + s];
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(
        reinterpret_cast<const uint8_t*>(W) + q2_code_bytes(n, hid, d));
    return q4_code(word, reg + 4 * (q & 1)) *
           __bfloat162float(sc[(rb * (hid / a.G) + j / a.G) * 128 + rr]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(THREADS) few_ffn_kernel(FewArgs a) {
    __shared__ Routing r;
    __shared__ float H[FT][FEW_HCAP];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    route_batch(a, r);
    if (blockIdx.x == 0) publish_routing(a, r);
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int A = r.items - (gS > 0);
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        const int64_t g0 = (int64_t)v * r.tot / r.V, g1 = (int64_t)(v + 1) * r.tot / r.V;
        __syncthreads();
        for (int64_t gg = g0; gg < g1; ++gg) {
            const int i = (int)min(gg / gE, (int64_t)A);
            const int j = (int)(gg - item_start(i, A, gE)) * FEW_GRAN + warp;
            for (int p = 0; p < r.n[i]; ++p) {
                const __nv_bfloat16* xr = x + (int64_t)r.tok[i][p] * a.d;
                float ga = 0.f, up = 0.f;
                for (int c = lane; c < a.d; c += 32) {
                    const float xv = __bfloat162float(xr[c]);
                    ga += xv * w13_at(a, r.expert[i], j, 0, c);
                    up += xv * w13_at(a, r.expert[i], j, 1, c);
                }
                ga = warp_sum(ga);
                up = warp_sum(up);
                if (lane == 0)
                    H[p][(int)(gg - g0) * FEW_GRAN + warp] = silu_f(ga) * up * r.gate[i][p];
            }
        }
        __syncthreads();
        for (int64_t s0 = g0; s0 < g1;) {
            const int i = (int)min(s0 / gE, (int64_t)A);
            const int64_t is = item_start(i, A, gE), ie = is + (i < A ? gE : gS);
            const int64_t s1 = min(ie, g1);
            const int row = r.row0[i] + (v - part_of(is, r.tot, r.V)) * r.n[i];
            const int j0 = (int)(s0 - is) * FEW_GRAN, len = (int)(s1 - s0) * FEW_GRAN;
            for (int c = tid; c < a.d; c += THREADS)
                for (int p = 0; p < r.n[i]; ++p) {
                    float y = 0.f;
                    for (int q = 0; q < len; ++q)
                        y += w2_at(a, r.expert[i], c, j0 + q) * H[p][(int)(s0 - g0) * FEW_GRAN + q];
                    a.part[(int64_t)(row + p) * a.d + c] = y;
                }
            s0 = s1;
        }
    }
}

// out[t][c] = sum over the uses of token t (choices in order, then the shared
// expert) and their parts in order of the partial rows.
__global__ void __launch_bounds__(THREADS) few_combine_kernel(FewArgs a) {
    const int t = blockIdx.y, c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= a.d) return;
    float s = 0.f;
    for (int j = 0; j <= a.k; ++j) {
        const int4 u = a.table[t * (a.k + 1) + j];
        for (int q = 0; q < u.y; ++q) s += a.part[(int64_t)(u.x + q * u.z) * a.d + c];
    }
    reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t)t * a.d + c] = __float2bfloat16_rn(s);
}

}  // namespace

int64_t few_part_rows(int T, int h, int E, int k, int hsum) {
    // A hit experts serve T k assignments at most; an item of g granules meets
    // at most g V / tot + 2 parts
    int64_t most = 0;
    const int64_t gE = h / FEW_GRAN, gS = hsum / FEW_GRAN;
    const int hi = E < T * k ? E : T * k;
    for (int A = k; A <= hi; ++A) {
        const int64_t tot = A * gE + gS, V = few_parts(tot, FEW_CTAS);
        const int64_t rows = (int64_t)T * k * (gE * V / tot + 2) + (gS ? T * (gS * V / tot + 2) : 0);
        most = rows > most ? rows : most;
    }
    return most;
}

int launch_few_ffn(const FewArgs& a, cudaStream_t st) {
    few_ffn_kernel<<<FEW_CTAS, THREADS, 0, st>>>(a);
    note_launch();
    return launch_result();
}

int launch_few_combine(const FewArgs& a, cudaStream_t st) {
    few_combine_kernel<<<dim3((a.d + THREADS - 1) / THREADS, a.T), THREADS, 0, st>>>(a);
    note_launch();
    return launch_result();
}

}  // namespace moe
