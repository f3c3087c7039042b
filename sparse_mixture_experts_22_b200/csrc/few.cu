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

// ---------------------------------------------------------------- instructions

// Bulk copy of `bytes` (a multiple of 16) from global memory, completing on bar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_addr(bar)),
        "l"(policy)
        : "memory");
}

// 3-D tiled bulk tensor load (tma_load_2d_hint's, with a third coordinate).
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int c0, int c1, int c2, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2),
        "l"(policy)
        : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One arrive of this thread on bar once its cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The eight codes of a word as an A fragment: or-ing a nibble u = q + 8 into the
// mantissa of 128 gives the bf16 128 + u, and 128 + u - 136 = q is exact.
__device__ __forceinline__ void codes_to_frag(uint32_t w, uint32_t (&a)[4]) {
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), off);
        a[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float((uint32_t)v << 16);
}

// ---------------------------------------------------------------- the expert kernel
//
// Sixteen warps multiply what two others bring in through a ring of stages:
// one issues the weights' copies (tensor maps for bf16, one bulk copy per stage
// for 4 bits), the other copies the expert's token rows 16 bytes a lane; both
// signal the stage's mbarrier.  Weights are the A operand (16 rows), the tokens
// of one expert the B operand (8 columns a tile), so one instruction takes 256
// weights from registers whatever the number of tokens.
//
// First half, per granule (32 hidden units): four tiles of 16 rows, the gate and
// the up rows of 8 units each, so that a lane's accumulators hold both for the
// same unit and token.  KW warps share the columns of a stage; their sums meet
// in shared memory at the end of d, where H = g silu(a) u is formed in fp32 and
// stored as two bf16 parts.  Second half: 256 rows of w2 (16 a warp) by the
// part's columns against both parts of H; the products of one expert go to the
// part's own rows of the partial outputs.
//
// Copied bf16 tiles are swizzled and token rows pitched by 16 bytes, so that
// ldmatrix meets no bank twice; 4-bit codes arrive in fragment order and are
// read as they lie.
template <int G, int NT>
struct Shape {
    static constexpr bool Q4 = G > 0;
    static constexpr int GG = Q4 ? G : 128;
    static constexpr int KP = Q4 ? 128 : 64;               // columns of a warp in a stage
    static constexpr int KW = Q4 && NT == 1 ? 8 : 4;       // warps along the columns
    static constexpr int KA = KW * KP;                     // columns of a stage
    static constexpr int GW = 16 / KW;                     // warps along the 16-row tiles
    static constexpr int MW = 4 / GW;                      // tiles of a warp
    static constexpr int QB = q13_block_bytes(GG);
    static constexpr int XPITCH = KA * 2 + 16;             // bytes of a token's row in a stage
    static constexpr int XOFF = Q4 ? KA / 128 * QB : KA * 128;  // where its tokens begin
    // down: 2 blocks of 128 rows x 8 panels of 32 units (4 bits) or 2 (bf16)
    static constexpr int PANELS = Q4 ? 8 : 2;
    static constexpr int SCALES = 32768;                   // 4 bits: where its scales begin
    static constexpr int GROUPS = GG == 32 ? 8 : 256 / GG + 1;  // groups that 8 panels can meet
    static constexpr int HPITCH = (FEW_HCAP + 8) * 2;      // bytes of a token's row of H
    static constexpr int HPART = NT * 8 * HPITCH;
    static constexpr int RED = 16 * MW * NT * 8 * 20 * 4;  // bytes of the warps' sums
    static __host__ __device__ int slot(int T) {
        const int up = XOFF + T * XPITCH, down = Q4 ? SCALES + 2 * GROUPS * 256 : 32768;
        return ((up > down ? up : down) + 1023) / 1024 * 1024;
    }
    static __host__ __device__ size_t fixed() {
        return 1024 + 2 * HPART + RED + sizeof(Routing) + 512;
    }
};

constexpr int MAX_STAGES = 12;
constexpr int CONSUMERS = 512;
constexpr int FFN_THREADS = CONSUMERS + 64;
constexpr int MAX_SEGS = FEW_HCAP / 128 + 2;  // experts (at least 128 units each) a part can meet

// One expert's share of a part.
struct Seg {
    int item, expert, n;   // expert -1: shared; tokens
    int j0, len;           // hidden units j0 .. j0 + len
    int row;               // its first row of the partial outputs
    int hb;                // where its H begins
};

// Share i of part v (granules g0 .. g1); false past the last one.
__device__ __forceinline__ bool segment(const FewArgs& a, const Routing& r, int v, int64_t g0,
                                        int64_t g1, int i, Seg& s) {
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int A = r.items - (gS > 0);
    s.item = (int)min(g0 / gE, (int64_t)A) + i;
    if (s.item >= r.items) return false;
    const int64_t is = item_start(s.item, A, gE);
    const int64_t s0 = max(is, g0), s1 = min(is + (s.item < A ? gE : gS), g1);
    if (s0 >= s1) return false;
    s.expert = r.expert[s.item];
    s.n = r.n[s.item];
    s.j0 = (int)(s0 - is) * FEW_GRAN;
    s.len = (int)(s1 - s0) * FEW_GRAN;
    s.row = r.row0[s.item] + (v - part_of(is, r.tot, r.V)) * s.n;
    s.hb = (int)(s0 - g0) * FEW_GRAN;
    return true;
}

// A warp writes part v's shares to segs; returns how many there are.
__device__ __forceinline__ int segments(const FewArgs& a, const Routing& r, int v, Seg* segs) {
    const int lane = threadIdx.x & 31;
    const int64_t g0 = (int64_t)v * r.tot / r.V, g1 = (int64_t)(v + 1) * r.tot / r.V;
    Seg s;
    const bool have = lane < MAX_SEGS && segment(a, r, v, g0, g1, lane, s);
    __syncwarp();
    if (have) segs[lane] = s;
    __syncwarp();
    return __popc(__ballot_sync(0xffffffffu, have));
}

// A ring position: stage and the parity of its current phase.
struct Ring {
    int stage = 0, stages;
    uint32_t phase = 0;
    __device__ void next() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// Calls up(seg, unit, k0) for every stage of the first half and
// down(seg, r0, p0, np) for every stage of the second (r0 the first of up to 256
// rows of d, np panels of 32 units from panel p0 of the share) of all parts of
// this block, in ring order; a call that returns false ends it.
template <int G, int NT, typename Up, typename Down>
__device__ __forceinline__ void for_stages(const FewArgs& a, const Routing& r, Seg* segs, Up up,
                                           Down down) {
    using S = Shape<G, NT>;
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        const int n = segments(a, r, v, segs);
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < segs[i].len; j += FEW_GRAN)
                for (int k0 = 0; k0 < a.d; k0 += S::KA)
                    if (!up(segs[i], segs[i].j0 + j, k0)) return;
        for (int r0 = 0; r0 < a.d; r0 += 256)
            for (int i = 0; i < n; ++i)
                for (int p = 0; p < segs[i].len / 32; p += S::PANELS)
                    if (!down(segs[i], r0, p, min(S::PANELS, segs[i].len / 32 - p))) return;
    }
}

// The weights' copies.
template <int G, int NT>
__device__ void bring_weights(const FewArgs& a, const Routing& r, const FewMaps& maps, Seg* segs,
                              uint8_t* ring, int slot, int stages, uint64_t* full,
                              uint64_t* empty, int32_t* issued) {
    using S = Shape<G, NT>;
    const int lane = threadIdx.x & 31;
    const int d = a.d;
    const uint64_t once = l2_policy_evict_first();
    Ring p;
    p.stages = stages;
    int count = 0;
    // waits for the stage to be free and announces its bytes
    auto open = [&](uint32_t bytes) -> bool {
        const bool ok = mbar_wait(&empty[p.stage], p.phase ^ 1, a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) report_timeout(a.status);
            return false;
        }
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[p.stage], bytes);
            *issued = ++count;
        }
        __syncwarp();
        return true;
    };
    auto up = [&](const Seg& s, int j, int k0) -> bool {
        const bool shared = s.expert < 0;
        const int hid = shared ? a.hsum : a.h, e = shared ? 0 : s.expert;
        const int kn = min(S::KA, d - k0);
        uint8_t* dst = ring + (size_t)p.stage * slot;
        if (!open(S::Q4 ? kn / 128 * S::QB : kn * 128)) return false;
        if (S::Q4) {
            const uint8_t* W = reinterpret_cast<const uint8_t*>(shared ? a.w13s : a.w13);
            const int64_t blk = ((int64_t)e * (hid / 32) + j / 32) * (d / 128) + k0 / 128;
            if (lane == 0)
                bulk_load(smem_addr(dst), W + blk * S::QB, kn / 128 * S::QB, &full[p.stage], once);
        } else if (lane < kn / 64) {
            tma_load_3d_hint(dst + lane * 8192, shared ? &maps.w13s : &maps.w13, &full[p.stage],
                             k0 + lane * 64, j % 128, 2 * (int)(((int64_t)e * hid + j) / 128), once);
        }
        p.next();
        return true;
    };
    auto down = [&](const Seg& s, int r0, int p0, int np) -> bool {
        const bool shared = s.expert < 0;
        const int hid = shared ? a.hsum : a.h, e = shared ? 0 : s.expert;
        const int nb = min(2, (d - r0) / 128);
        uint8_t* dst = ring + (size_t)p.stage * slot;
        if (S::Q4) {
            const uint8_t* W = reinterpret_cast<const uint8_t*>(shared ? a.w2s : a.w2);
            const uint8_t* sc = W + q2_code_bytes(shared ? 1 : a.E, hid, d);
            const int pp = s.j0 / 32 + p0;
            const int q0 = pp * 32 / S::GG, nq = ((pp + np) * 32 - 1) / S::GG - q0 + 1;
            if (!open(nb * (np * 2048 + nq * 256))) return false;
            const int b = lane & 1;
            const int64_t rb = (int64_t)e * (d / 128) + r0 / 128 + b;
            if (b < nb && lane < 2)
                bulk_load(smem_addr(dst) + b * 16384, W + (rb * (hid / 32) + pp) * 2048, np * 2048,
                          &full[p.stage], once);
            if (b < nb && (lane >> 1) == 1)
                bulk_load(smem_addr(dst) + S::SCALES + b * S::GROUPS * 256,
                          sc + (rb * (hid / S::GG) + q0) * 256, nq * 256, &full[p.stage], once);
        } else {
            if (!open(nb * np * 8192)) return false;
            const int b = lane & 1, c = lane >> 1;
            if (b < nb && c < np)
                tma_load_2d_hint(dst + lane * 8192, shared ? &maps.w2s : &maps.w2, &full[p.stage],
                                 s.j0 + (p0 + c) * 32, e * d + r0 + 128 * b, once);
        }
        p.next();
        return true;
    };
    for_stages<G, NT>(a, r, segs, up, down);
}

// The token rows of the first half, 16 bytes a lane; every lane arrives on
// every stage, when its copies have landed.
template <int G, int NT>
__device__ void bring_tokens(const FewArgs& a, const Routing& r, Seg* segs, uint8_t* ring,
                             int slot, int stages, uint64_t* full, uint64_t* empty) {
    using S = Shape<G, NT>;
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    Ring p;
    p.stages = stages;
    auto open = [&]() -> bool {
        const bool ok = mbar_wait(&empty[p.stage], p.phase ^ 1, a.wait_limit_ns);
        return __all_sync(0xffffffffu, ok);
    };
    auto up = [&](const Seg& s, int, int k0) -> bool {
        if (!open()) return false;
        const int vecs = min(S::KA, a.d - k0) / 8;
        const uint32_t dst = smem_addr(ring + (size_t)p.stage * slot) + S::XOFF;
        for (int n = 0; n < s.n; ++n) {
            const __nv_bfloat16* src = x + (int64_t)r.tok[s.item][n] * a.d + k0;
#pragma unroll
            for (int q = 0; q < S::KA / 256; ++q)
                if (q * 32 + lane < vecs)
                    cp_async16(dst + n * S::XPITCH + (q * 32 + lane) * 16, src + (q * 32 + lane) * 8);
        }
        cp_async_arrive(&full[p.stage]);
        p.next();
        return true;
    };
    auto down = [&](const Seg&, int, int, int) -> bool {
        if (!open()) return false;
        mbar_arrive(&full[p.stage]);
        p.next();
        return true;
    };
    for_stages<G, NT>(a, r, segs, up, down);
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int G, int NT>
__device__ void consume(const FewArgs& a, const Routing& r, Seg* segs, uint8_t* ring, int slot,
                        int stages, uint64_t* full, uint64_t* empty, uint8_t* Hs, float* red,
                        int32_t* flags) {
    using S = Shape<G, NT>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kw = warp % S::KW, gw = warp / S::KW;
    const int fg = lane >> 2, ft = lane & 3;         // row and column pair of a fragment
    const int lm = lane & 7, lq = lane >> 3;         // row and matrix of an ldmatrix address
    const int d = a.d;
    const uint32_t hs = smem_addr(Hs);
    Ring p;
    p.stages = stages;
    bool lost = false;  // a wait ran out: go on without waiting, so that the barriers are met
    auto wait = [&]() -> uint32_t {
        if (!lost && !mbar_wait(&full[p.stage], p.phase, a.wait_limit_ns)) {
            lost = true;
            flags[0] = 1;
            report_timeout(a.status);
        }
        lost = __any_sync(0xffffffffu, lost);
        return smem_addr(ring + (size_t)p.stage * slot);
    };
    auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[p.stage]);
        p.next();
    };
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        named_sync(1, CONSUMERS);  // the last part's shares and H have been read
        if (warp == 0) {
            const int n = segments(a, r, v, segs);
            if (lane == 0) flags[2] = n;
        }
        named_sync(1, CONSUMERS);
        const int nseg = flags[2];
        // ---------------------------------------------------- H
        for (int i = 0; i < nseg; ++i) {
            const Seg s = segs[i];
            // rows of tokens past the expert's repeat its last one: their columns
            // of the product are never read
            uint32_t xrow[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                xrow[nt] = S::XOFF + min(nt * 8 + lm, s.n - 1) * S::XPITCH +
                           (kw * S::KP + lq * 8) * 2;
            for (int j = 0; j < s.len; j += FEW_GRAN) {
                float acc[S::MW][NT][4];
#pragma unroll
                for (int m = 0; m < S::MW; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[m][nt][q] = 0.f;
                for (int k0 = 0; k0 < d; k0 += S::KA) {
                    const uint32_t st = wait();
                    if (!lost && k0 + kw * S::KP < d) {
                        uint32_t b[NT][S::KP / 32][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if (nt * 8 < s.n) {
#pragma unroll
                                for (int q = 0; q < S::KP / 32; ++q)
                                    ldmatrix4(st + xrow[nt] + q * 64, b[nt][q]);
                            }
#pragma unroll
                        for (int m = 0; m < S::MW; ++m) {
                            const int g = m * S::GW + gw;
                            if (S::Q4) {
                                const uint4* cw = reinterpret_cast<const uint4*>(
                                    ring + (size_t)p.stage * slot + kw * S::QB + g * 1024);
                                uint32_t w[8];
                                *reinterpret_cast<uint4*>(w) = cw[lane];
                                *reinterpret_cast<uint4*>(w + 4) = cw[32 + lane];
                                const uint32_t sa = st + kw * S::QB + 4096 + (g * 16 + fg) * 2;
#pragma unroll
                                for (int q = 0; q < 128 / S::GG; ++q) {
                                    float c[NT][4];
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
                                    for (int u = q * (S::GG / 16); u < (q + 1) * (S::GG / 16); ++u) {
                                        uint32_t f[4];
                                        codes_to_frag(w[u], f);
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt)
                                            if (nt * 8 < s.n)
                                                mma(c[nt], f, b[nt][u / 2][2 * (u & 1)],
                                                    b[nt][u / 2][2 * (u & 1) + 1]);
                                    }
                                    const float sl = lds_bf16(sa + q * 128);
                                    const float sh = lds_bf16(sa + q * 128 + 16);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        acc[m][nt][0] = fmaf(c[nt][0], sl, acc[m][nt][0]);
                                        acc[m][nt][1] = fmaf(c[nt][1], sl, acc[m][nt][1]);
                                        acc[m][nt][2] = fmaf(c[nt][2], sh, acc[m][nt][2]);
                                        acc[m][nt][3] = fmaf(c[nt][3], sh, acc[m][nt][3]);
                                    }
                                }
                            } else {
                                // box of this warp's 64 columns: 32 gate rows, 32 up rows
                                const uint32_t wa = st + kw * 8192 + ((lq & 1) * 32 + g * 8 + lm) * 128;
#pragma unroll
                                for (int u = 0; u < S::KP / 16; ++u) {
                                    uint32_t f[4];
                                    ldmatrix4(wa + (((u * 2 + (lq >> 1)) ^ lm) << 4), f);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        if (nt * 8 < s.n)
                                            mma(acc[m][nt], f, b[nt][u / 2][2 * (u & 1)],
                                                b[nt][u / 2][2 * (u & 1) + 1]);
                                }
                            }
                        }
                    }
                    done();
                }
                named_sync(1, CONSUMERS);  // the last granule's sums have been read
#pragma unroll
                for (int m = 0; m < S::MW; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* q = red + ((warp * S::MW + m) * NT + nt) * 160 + 2 * ft * 20 + fg;
                        q[0] = acc[m][nt][0];
                        q[20] = acc[m][nt][1];
                        q[8] = acc[m][nt][2];
                        q[28] = acc[m][nt][3];
                    }
                named_sync(1, CONSUMERS);
                __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(Hs);
                if (tid < FEW_GRAN * s.n) {
                    const int jj = tid & 7, g = (tid >> 3) & 3, n = tid >> 5;
                    float ga = 0.f, up = 0.f;
#pragma unroll
                    for (int w = 0; w < S::KW; ++w) {
                        const float* q = red + ((((g % S::GW) * S::KW + w) * S::MW + g / S::GW) * NT +
                                                n / 8) * 160 + (n & 7) * 20 + jj;
                        ga += q[0];
                        up += q[8];
                    }
                    const float hv = silu_f(ga) * up * r.gate[s.item][n];
                    const float hi = bf16_round(hv);
                    const int at = n * (S::HPITCH / 2) + s.hb + j + g * 8 + jj;
                    H[at] = __float2bfloat16_rn(hi);
                    H[S::HPART / 2 + at] = __float2bfloat16_rn(hv - hi);
                }
            }
        }
        named_sync(1, CONSUMERS);
        // ---------------------------------------------------- this part of the output
        const int rb = warp >> 3, tile = warp & 7;  // this warp's 16 rows of 256
        for (int r0 = 0; r0 < d; r0 += 256) {
            const bool mine = r0 + rb * 128 < d;
            for (int i = 0; i < nseg; ++i) {
                const Seg s = segs[i];
                // one chain of products for each part of H
                float acc[NT][4], low[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[nt][q] = low[nt][q] = 0.f;
                // H fragments: matrices (high, k), (high, k + 8), (low, k), (low, k + 8)
                uint32_t hrow[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    hrow[nt] = hs + (lq >> 1) * S::HPART + min(nt * 8 + lm, s.n - 1) * S::HPITCH +
                               (s.hb + (lq & 1) * 8) * 2;
                for (int p0 = 0; p0 < s.len / 32; p0 += S::PANELS) {
                    const int np = min(S::PANELS, s.len / 32 - p0);
                    const uint32_t st = wait();
                    if (!lost && mine) {
                        const int pp = s.j0 / 32 + p0, q0 = pp * 32 / S::GG;
#pragma unroll 2
                        for (int c = 0; c < np; ++c) {
                            uint32_t b[NT][2][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (nt * 8 < s.n) {
                                    ldmatrix4(hrow[nt] + (p0 + c) * 64, b[nt][0]);
                                    ldmatrix4(hrow[nt] + (p0 + c) * 64 + 32, b[nt][1]);
                                }
                            if (S::Q4) {
                                const uint2 w = reinterpret_cast<const uint2*>(
                                    ring + (size_t)p.stage * slot + rb * 16384 +
                                    (c * 8 + tile) * 256)[lane];
                                const uint32_t sa = st + S::SCALES +
                                                    (rb * S::GROUPS + (pp + c) * 32 / S::GG - q0) * 256 +
                                                    (tile * 16 + fg) * 2;
                                const float sl = lds_bf16(sa), sh = lds_bf16(sa + 16);
                                uint32_t f0[4], f1[4];
                                codes_to_frag(w.x, f0);
                                codes_to_frag(w.y, f1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    if (nt * 8 < s.n) {
                                        float ch[4] = {0.f, 0.f, 0.f, 0.f};
                                        float cl[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma(ch, f0, b[nt][0][0], b[nt][0][1]);
                                        mma(cl, f0, b[nt][0][2], b[nt][0][3]);
                                        mma(ch, f1, b[nt][1][0], b[nt][1][1]);
                                        mma(cl, f1, b[nt][1][2], b[nt][1][3]);
                                        acc[nt][0] = fmaf(ch[0] + cl[0], sl, acc[nt][0]);
                                        acc[nt][1] = fmaf(ch[1] + cl[1], sl, acc[nt][1]);
                                        acc[nt][2] = fmaf(ch[2] + cl[2], sh, acc[nt][2]);
                                        acc[nt][3] = fmaf(ch[3] + cl[3], sh, acc[nt][3]);
                                    }
                            } else {
                                // box (c, rb): 128 rows of 64 bytes
                                const int row = tile * 16 + (lq & 1) * 8 + lm;
                                const uint32_t wa = st + (c * 2 + rb) * 8192 + row * 64;
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    uint32_t f[4];
                                    ldmatrix4(wa + (((u * 2 + (lq >> 1)) ^ ((lm >> 1) & 3)) << 4), f);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        if (nt * 8 < s.n) {
                                            mma(acc[nt], f, b[nt][u][0], b[nt][u][1]);
                                            mma(low[nt], f, b[nt][u][2], b[nt][u][3]);
                                        }
                                }
                            }
                        }
                    }
                    done();
                }
                if (mine) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int n = nt * 8 + 2 * ft;
                        float* q = a.part + (int64_t)(s.row + n) * d + r0 + rb * 128 + tile * 16 + fg;
                        if (n < s.n) {
                            q[0] = acc[nt][0] + low[nt][0];
                            q[8] = acc[nt][2] + low[nt][2];
                        }
                        if (n + 1 < s.n) {
                            q[d] = acc[nt][1] + low[nt][1];
                            q[d + 8] = acc[nt][3] + low[nt][3];
                        }
                    }
                }
            }
        }
    }
}

template <int G, int NT>
__global__ void __launch_bounds__(FFN_THREADS, 1)
    few_ffn_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a,
                   int slot, int stages) {
    using S = Shape<G, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + (-smem_addr(smem_raw) & 1023);
    uint8_t* Hs = ring + (size_t)slot * stages;
    float* red = reinterpret_cast<float*>(Hs + 2 * S::HPART);
    Routing& r = *reinterpret_cast<Routing*>(Hs + 2 * S::HPART + S::RED);
    uint64_t* full = reinterpret_cast<uint64_t*>(
        reinterpret_cast<uint8_t*>(&r) + (sizeof(Routing) + 15) / 16 * 16);
    uint64_t* empty = full + MAX_STAGES;
    int32_t* flags = reinterpret_cast<int32_t*>(empty + MAX_STAGES);  // a wait ran out; stages issued; shares of the part
    __shared__ Seg segs[3][MAX_SEGS];
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1 + 32);  // the weights' announcement, the token warp's lanes
            mbar_init(&empty[i], CONSUMERS / 32);
        }
        flags[0] = flags[1] = 0;
        fence_mbar_init();
        if (!S::Q4) {
            prefetch_tmap(&maps.w13);
            prefetch_tmap(&maps.w2);
        }
    }
    pdl_trigger();
    pdl_wait();  // the router's logits
    route_batch(a, r);
    if (a.test_stall && blockIdx.x == 0 && warp >= CONSUMERS / 32) {
        // the test hook: nothing is brought in, the consumers' waits run out
    } else if (warp == CONSUMERS / 32) {
        bring_weights<G, NT>(a, r, maps, segs[1], ring, slot, stages, full, empty, &flags[1]);
    } else if (warp > CONSUMERS / 32) {
        bring_tokens<G, NT>(a, r, segs[2], ring, slot, stages, full, empty);
    } else {
        consume<G, NT>(a, r, segs[0], ring, slot, stages, full, empty, Hs, red, flags);
    }
    if (blockIdx.x == gridDim.x - 1) publish_routing(a, r);
    __syncthreads();
    if (flags[0] && tid == 0) {
        // a wait ran out: see the copies in flight land before the block goes
        const int n = flags[1];
        for (int i = n > stages ? n - stages : 0; i < n; ++i)
            mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1, a.wait_limit_ns);
    }
}

// ---------------------------------------------------------------- combine

// out[t][c] = sum over the uses of token t (choices in order, then the shared
// expert) and their parts of the partial rows.  A block takes 64 columns of one
// token: 16 groups of 16 lanes share the rows, so that a row's 256 bytes are
// one access and many rows are in flight.
constexpr int CB_COLS = 64;

__global__ void __launch_bounds__(256) few_combine_kernel(const __grid_constant__ FewArgs a) {
    __shared__ float4 sums[16][16];
    const int tid = threadIdx.x, col = tid & 15, grp = tid >> 4;
    const int t = blockIdx.y, c = blockIdx.x * CB_COLS + col * 4;
    pdl_wait();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const int uses = a.k + (a.hsum > 0);
    for (int j = 0; j < uses; ++j) {
        const int4 u = a.table[t * (a.k + 1) + j];
#pragma unroll 4
        for (int q = grp; q < u.y; q += 16) {
            const float4 v =
                *reinterpret_cast<const float4*>(a.part + (int64_t)(u.x + q * u.z) * a.d + c);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    sums[grp][col] = s;
    __syncthreads();
    if (tid < 16) {
        float4 o = sums[0][tid];
#pragma unroll
        for (int g = 1; g < 16; ++g) {
            o.x += sums[g][tid].x;
            o.y += sums[g][tid].y;
            o.z += sums[g][tid].z;
            o.w += sums[g][tid].w;
        }
        uint2 w;
        w.x = pack_bf16x2(o.x, o.y);
        w.y = pack_bf16x2(o.z, o.w);
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)t * a.d +
                                  blockIdx.x * CB_COLS + tid * 4) = w;
    }
}

// ---------------------------------------------------------------- router

// z[t][e] for 8 experts and up to TT tokens by a cluster of 8 blocks, each an
// eighth of d; the blocks' sums meet in the first one through its cluster's
// shared memory, in block order.  W_r is read once whatever T, and even E = 8
// spreads over 8 SMs, where one block per token took the latency of reading
// the whole of W_r in turn.
constexpr int RC = 8;

__device__ __forceinline__ float ld_cluster_f32(uint32_t caddr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(caddr) : "memory");
    return v;
}

template <int TT>
__global__ void __cluster_dims__(1, RC, 1) __launch_bounds__(256)
    few_router_kernel(const __nv_bfloat16* __restrict__ x, const float* __restrict__ Wr,
                      float* __restrict__ z, int T, int d, int E, int32_t* status) {
    constexpr int N = TT * 8;
    __shared__ float part[8][N];
    __shared__ float sum[N];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int e0 = blockIdx.x * 8, len = d / RC, c0 = blockIdx.y * len;
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *status = DEV_OK;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int c = c0 + tid; c < c0 + len; c += 256) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e0 + e < E ? Wr[(int64_t)c * E + e0 + e] : 0.f;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float xv = t < T ? __bfloat162float(x[(int64_t)t * d + c]) : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[t * 8 + e] = fmaf(xv, w[e], v[t * 8 + e]);
        }
    }
    // the warp's sums: each exchange halves the values a lane keeps
    int n = N, first = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n /= 2;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float send = up ? v[i] : v[i + n];
                    v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
                }
            if (up) first += n;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    constexpr int LEFT = N >= 32 ? N / 32 : 1;
    if (N >= 32 || (lane & (32 / N - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < LEFT; ++i) part[warp][first + i] = v[i];
    }
    __syncthreads();
    if (tid < N) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part[w][tid];
        sum[tid] = s;
    }
    cluster_sync_all();
    if (cluster_ctarank() == 0 && tid < N) {
        const uint32_t at = smem_addr(&sum[tid]);
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < RC; ++q) s += ld_cluster_f32(map_shared_rank(at, q));
        const int t = tid / 8, e = e0 + tid % 8;
        if (t < T && e < E) z[(int64_t)t * E + e] = s;
    }
    cluster_sync_all();  // the sums are read before their blocks go
}

template <int G, int NT>
int launch_ffn(const FewMaps& m, const FewArgs& a, int smem_limit, cudaStream_t st) {
    using S = Shape<G, NT>;
    const int slot = S::slot(a.T);
    // the kernel's few static bytes count too
    const size_t limit = (size_t)smem_limit - 3 * MAX_SEGS * sizeof(Seg) - 256;
    int stages = (int)((limit - S::fixed()) / slot);
    stages = stages > MAX_STAGES ? MAX_STAGES : stages;
    const size_t smem = S::fixed() + (size_t)slot * stages;
    auto kern = few_ffn_kernel<G, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit) !=
        cudaSuccess)
        return launch_result();
    launch_ex(true, kern, dim3(FEW_CTAS), dim3(FFN_THREADS), smem, st, m, a, slot, stages);
    note_launch();
    return launch_result();
}

template <int NT>
int launch_ffn_group(const FewMaps& m, const FewArgs& a, int smem_limit, cudaStream_t st) {
    switch (a.G) {
        case 0: return launch_ffn<0, NT>(m, a, smem_limit, st);
        case 32: return launch_ffn<32, NT>(m, a, smem_limit, st);
        case 64: return launch_ffn<64, NT>(m, a, smem_limit, st);
        default: return launch_ffn<128, NT>(m, a, smem_limit, st);
    }
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

int launch_few_router(const void* x, const float* Wr, float* z, int T, int d, int E,
                      int32_t* status, cudaStream_t st) {
    const dim3 grid((E + 7) / 8, RC);
    const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(x);
    if (T == 1) few_router_kernel<1><<<grid, 256, 0, st>>>(xb, Wr, z, T, d, E, status);
    else if (T <= 4) few_router_kernel<4><<<grid, 256, 0, st>>>(xb, Wr, z, T, d, E, status);
    else few_router_kernel<16><<<grid, 256, 0, st>>>(xb, Wr, z, T, d, E, status);
    note_launch();
    return launch_result();
}

int launch_few_ffn(const FewMaps& m, const FewArgs& a, int smem_limit, cudaStream_t st) {
    return a.T <= 8 ? launch_ffn_group<1>(m, a, smem_limit, st)
                    : launch_ffn_group<2>(m, a, smem_limit, st);
}

int launch_few_combine(const FewArgs& a, cudaStream_t st) {
    launch_ex(true, few_combine_kernel, dim3(a.d / CB_COLS, a.T), dim3(256), 0, st, a);
    note_launch();
    return launch_result();
}

}  // namespace moe
