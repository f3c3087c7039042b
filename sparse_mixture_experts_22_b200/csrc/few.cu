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
// Eight warps multiply what a ninth brings in through a ring of stages (bulk
// copies, one mbarrier per stage).  Weights are the A operand (16 rows), the
// tokens of one expert the B operand (8 columns a tile), so one instruction
// takes 256 weights from registers whatever the number of tokens.
//
// First half, per tile of up to MA granules of one expert: the 16 rows of a
// granule are the gate and the up rows of its 8 hidden units, so a lane's
// accumulators hold both for the same unit and token.  KW warps share the
// columns of a stage (KA); their sums meet in shared memory at the end of d,
// where H = g silu(a) u is formed in fp32 and stored as two bf16 parts.
// Second half: w2's rows by the part's columns, 128 rows per 8 warps, against
// both parts of H; the products of one expert go to the part's own rows of the
// partial outputs.
//
// Shared-memory rows of the copied tiles are pitched by 16 bytes (bf16 rows) or
// swizzled by the tensor copy (w2), so that ldmatrix meets no bank twice; the
// 4-bit codes arrive in fragment order and are read as they lie.
template <int G, int NT>
struct Shape {
    static constexpr bool Q4 = G > 0;
    static constexpr int KW = Q4 ? 4 : 8;        // warps along the columns
    static constexpr int GW = 8 / KW;            // warps along the granules
    static constexpr int KA = 512;               // columns of a stage
    static constexpr int MA = Q4 ? (NT == 1 ? 8 : 4) : 2;  // granules of a stage
    static constexpr int MW = MA / GW;           // granules of a warp
    static constexpr int XPITCH = KA * 2 + 16;   // bytes of a token's row in a stage
    static constexpr int WPITCH = KA * 2 + 16;   // bytes of a bf16 weight row
    static constexpr int SCALES = MA * 4096;     // 4 bits: where a stage's scales begin
    static constexpr int XOFF = Q4 ? MA * 4608 : MA * 16 * WPITCH;  // where its tokens begin
    static constexpr int RB = Q4 ? MA / 4 : 2;   // blocks of 128 rows of a down stage
    static constexpr int HALIGN = Q4 ? 32 : 16;  // H of one expert is padded to this
    static constexpr int HPITCH = (FEW_HCAP + 64 + 8) * 2;  // bytes of a token's row of H
    static constexpr int HPART = NT * 8 * HPITCH;
    static constexpr int RED = 8 * MW * NT * 8 * 20 * 4;    // bytes of the warps' sums
    static __host__ __device__ int slot(int T) {
        const int b = XOFF + T * XPITCH;
        return (b + 1023) / 1024 * 1024;
    }
    static __host__ __device__ size_t fixed() {
        return 1024 + 2 * HPART + RED + sizeof(Routing) + 256;
    }
};

constexpr int MAX_STAGES = 12;
constexpr int FFN_THREADS = 288;
constexpr int CONSUMERS = 256;

// One expert's share of a part.
struct Seg {
    int item, expert, n;   // expert -1: shared
    int j0, len;           // hidden units j0 .. j0 + len
    int row;               // its first row of the partial outputs
    int hb, front;         // where its H begins; units of padding before j0
    int64_t next;          // granule after it
};

template <int HALIGN>
__device__ __forceinline__ Seg segment(const FewArgs& a, const Routing& r, int v, int64_t s0,
                                       int64_t g1, int hb) {
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int A = r.items - (gS > 0);
    Seg s;
    s.item = (int)min(s0 / gE, (int64_t)A);
    const int64_t is = item_start(s.item, A, gE);
    s.next = min(is + (s.item < A ? gE : gS), g1);
    s.expert = r.expert[s.item];
    s.n = r.n[s.item];
    s.j0 = (int)(s0 - is) * FEW_GRAN;
    s.len = (int)(s.next - s0) * FEW_GRAN;
    s.row = r.row0[s.item] + (v - part_of(is, r.tot, r.V)) * s.n;
    s.hb = hb;
    s.front = HALIGN == 32 ? s.j0 % 32 : 0;
    return s;
}

template <int HALIGN>
__device__ __forceinline__ int padded(const Seg& s) {
    return (s.front + s.len + HALIGN - 1) / HALIGN * HALIGN;
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

template <int G, int NT>
__device__ void produce(const FewArgs& a, const Routing& r, const CUtensorMap* m2,
                        const CUtensorMap* m2s, uint8_t* ring, int slot, int stages,
                        uint64_t* full, uint64_t* empty, int32_t* issued) {
    using S = Shape<G, NT>;
    const int lane = threadIdx.x & 31;
    const int d = a.d;
    const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_normal();
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
    if (a.test_stall && blockIdx.x == 0) return;
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        const int64_t g0 = (int64_t)v * r.tot / r.V, g1 = (int64_t)(v + 1) * r.tot / r.V;
        for (int64_t s0 = g0; s0 < g1;) {
            const Seg s = segment<S::HALIGN>(a, r, v, s0, g1, 0);
            s0 = s.next;
            const bool shared = s.expert < 0;
            const int hid = shared ? a.hsum : a.h;
            const int64_t e = shared ? 0 : s.expert;
            const uint8_t* W = reinterpret_cast<const uint8_t*>(shared ? a.w13s : a.w13);
            const uint8_t* sc = S::Q4 ? W + q13_code_bytes(shared ? 1 : a.E, hid, d) : nullptr;
            const int ng = s.len / FEW_GRAN, tiles = (ng + S::MA - 1) / S::MA;
            for (int tl = 0; tl < tiles; ++tl) {
                const int t0 = tl * ng / tiles, m = (tl + 1) * ng / tiles - t0;
                const int j = s.j0 + t0 * FEW_GRAN;
                for (int k0 = 0; k0 < d; k0 += S::KA) {
                    const int kn = min(S::KA, d - k0);
                    const uint32_t wb = S::Q4 ? kn / 128 * (1024 + 32 * (128 / (G ? G : 128)))
                                              : 16 * kn * 2;
                    if (!open(m * wb + s.n * kn * 2)) return;
                    const uint32_t dst = smem_addr(ring + (size_t)p.stage * slot);
                    if (S::Q4) {
                        constexpr int SB = 32 * (128 / (G ? G : 128));  // scale bytes of a block
                        const int g = lane & 7;
                        const int64_t blk = (e * (hid / 8) + j / 8 + g) * (d / 128) + k0 / 128;
                        if (g < m && lane < 8)
                            bulk_load(dst + g * 4096, W + blk * 1024, kn * 8, &full[p.stage], once);
                        if (g < m && lane >= 8 && lane < 16)
                            bulk_load(dst + S::SCALES + g * 4 * SB, sc + blk * SB, kn / 128 * SB,
                                      &full[p.stage], once);
                        if (lane >= 16 && lane - 16 < s.n)
                            bulk_load(dst + S::XOFF + (lane - 16) * S::XPITCH,
                                      reinterpret_cast<const __nv_bfloat16*>(a.x) +
                                          (int64_t)r.tok[s.item][lane - 16] * d + k0,
                                      kn * 2, &full[p.stage], keep);
                    } else {
                        const int g = lane >> 4, rr = lane & 15, jj = j + g * FEW_GRAN + (rr & 7);
                        const int64_t row = e * 2 * hid + 256 * (jj / 128) + 128 * (rr >> 3) + jj % 128;
                        if (g < m)
                            bulk_load(dst + (g * 16 + rr) * S::WPITCH, W + (row * d + k0) * 2, kn * 2,
                                      &full[p.stage], once);
                        if (lane < s.n)
                            bulk_load(dst + S::XOFF + lane * S::XPITCH,
                                      reinterpret_cast<const __nv_bfloat16*>(a.x) +
                                          (int64_t)r.tok[s.item][lane] * d + k0,
                                      kn * 2, &full[p.stage], keep);
                    }
                    p.next();
                }
            }
        }
        for (int r0 = 0; r0 < d; r0 += 128 * S::RB) {
            const int nb = min(S::RB, (d - r0) / 128);
            for (int64_t s0 = g0; s0 < g1;) {
                const Seg s = segment<S::HALIGN>(a, r, v, s0, g1, 0);
                s0 = s.next;
                const bool shared = s.expert < 0;
                const int hid = shared ? a.hsum : a.h;
                const int64_t e = shared ? 0 : s.expert;
                if (S::Q4) {
                    constexpr int GG = G ? G : 128;
                    const uint8_t* W = reinterpret_cast<const uint8_t*>(shared ? a.w2s : a.w2);
                    const uint8_t* sc = W + q2_code_bytes(shared ? 1 : a.E, hid, d);
                    const int p0 = s.j0 / 32, p1 = (s.j0 + s.len + 31) / 32;
                    for (int pp = p0; pp < p1; pp += 8) {
                        const int np = min(8, p1 - pp);
                        const int q0 = pp * 32 / GG, nq = ((pp + np) * 32 - 1) / GG - q0 + 1;
                        if (!open(nb * (np * 2048 + nq * 256))) return;
                        const uint32_t dst = smem_addr(ring + (size_t)p.stage * slot);
                        if (lane < nb) {
                            const int64_t rb = e * (d / 128) + r0 / 128 + lane;
                            bulk_load(dst + lane * 16384, W + (rb * (hid / 32) + pp) * 2048, np * 2048,
                                      &full[p.stage], once);
                            bulk_load(dst + S::SCALES + lane * 2048, sc + (rb * (hid / GG) + q0) * 256,
                                      nq * 256, &full[p.stage], once);
                        }
                        p.next();
                    }
                } else {
                    for (int c = 0; c < s.len; c += 64) {
                        if (!open(nb * 16384)) return;
                        if (lane < nb)
                            tma_load_2d_hint(ring + (size_t)p.stage * slot + lane * 16384,
                                             shared ? m2s : m2, &full[p.stage], s.j0 + c,
                                             (int)(e * d + r0 + 128 * lane), once);
                        p.next();
                    }
                }
            }
        }
    }
}

template <int G, int NT>
__device__ void consume(const FewArgs& a, const Routing& r, uint8_t* ring, int slot, int stages,
                        uint64_t* full, uint64_t* empty, uint8_t* Hs, float* red, int32_t* dead) {
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
            *dead = 1;
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
        const int64_t g0 = (int64_t)v * r.tot / r.V, g1 = (int64_t)(v + 1) * r.tot / r.V;
        // ---------------------------------------------------- H
        int hb = 0;
        for (int64_t s0 = g0; s0 < g1;) {
            const Seg s = segment<S::HALIGN>(a, r, v, s0, g1, hb);
            s0 = s.next;
            hb += padded<S::HALIGN>(s);
            const int ng = s.len / FEW_GRAN, tiles = (ng + S::MA - 1) / S::MA;
            // rows of tokens past the expert's repeat its last one: their columns
            // of the product are never read
            uint32_t xrow[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                xrow[nt] = S::XOFF + min(nt * 8 + lm, s.n - 1) * S::XPITCH;
            for (int tl = 0; tl < tiles; ++tl) {
                const int t0 = tl * ng / tiles, m = (tl + 1) * ng / tiles - t0;
                float acc[S::MW][NT][4];
#pragma unroll
                for (int i = 0; i < S::MW; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[i][nt][q] = 0.f;
                for (int k0 = 0; k0 < d; k0 += S::KA) {
                    const uint32_t st = wait();
                    constexpr int KP = S::KA / S::KW;  // columns of a warp
                    if (!lost && k0 + kw * KP < d) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (nt * 8 >= s.n) break;
                            uint32_t b[KP / 32][4];
#pragma unroll
                            for (int q = 0; q < KP / 32; ++q)
                                ldmatrix4(st + xrow[nt] + (kw * KP + q * 32 + lq * 8) * 2, b[q]);
                            if (S::Q4) {
                                constexpr int GG = G ? G : 128, SB = 32 * (128 / GG);
#pragma unroll
                                for (int i = 0; i < S::MW; ++i) {
                                    const int g = i * S::GW + gw;
                                    if (g >= m) break;
                                    uint32_t w[8];
                                    const uint4* cw = reinterpret_cast<const uint4*>(
                                        ring + (size_t)p.stage * slot + g * 4096 + kw * 1024);
                                    *reinterpret_cast<uint4*>(w) = cw[lane];
                                    *reinterpret_cast<uint4*>(w + 4) = cw[32 + lane];
                                    const uint32_t sa = st + S::SCALES + (g * 4 + kw) * SB + fg * 2;
#pragma unroll
                                    for (int q = 0; q < 128 / GG; ++q) {
                                        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                        for (int u = 0; u < GG / 16; ++u) {
                                            const int k16 = q * (GG / 16) + u;
                                            uint32_t f[4];
                                            codes_to_frag(w[k16], f);
                                            mma(c, f, b[k16 / 2][2 * (k16 & 1)],
                                                b[k16 / 2][2 * (k16 & 1) + 1]);
                                        }
                                        const float sl = lds_bf16(sa + q * 32);
                                        const float sh = lds_bf16(sa + q * 32 + 16);
                                        acc[i][nt][0] = fmaf(c[0], sl, acc[i][nt][0]);
                                        acc[i][nt][1] = fmaf(c[1], sl, acc[i][nt][1]);
                                        acc[i][nt][2] = fmaf(c[2], sh, acc[i][nt][2]);
                                        acc[i][nt][3] = fmaf(c[3], sh, acc[i][nt][3]);
                                    }
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < S::MW; ++i) {
                                    if (i >= m) break;
                                    const uint32_t wa =
                                        st + (i * 16 + (lq & 1) * 8 + lm) * S::WPITCH +
                                        (kw * KP + (lq >> 1) * 8) * 2;
#pragma unroll
                                    for (int u = 0; u < KP / 16; ++u) {
                                        uint32_t f[4];
                                        ldmatrix4(wa + u * 32, f);
                                        mma(acc[i][nt], f, b[u / 2][2 * (u & 1)],
                                            b[u / 2][2 * (u & 1) + 1]);
                                    }
                                }
                            }
                        }
                    }
                    done();
                }
                named_sync(1, CONSUMERS);  // the last tile's sums have been read
#pragma unroll
                for (int i = 0; i < S::MW; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* q = red + ((warp * S::MW + i) * NT + nt) * 160 + 2 * ft * 20 + fg;
                        q[0] = acc[i][nt][0];
                        q[20] = acc[i][nt][1];
                        q[8] = acc[i][nt][2];
                        q[28] = acc[i][nt][3];
                    }
                named_sync(1, CONSUMERS);
                __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(Hs);
                constexpr int HP = S::HPITCH / 2, HLO = S::HPART / 2;
                for (int i = tid; i < 8 * m * s.n; i += CONSUMERS) {
                    const int jj = i & 7, g = (i >> 3) % m, n = (i >> 3) / m;
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
                    const int at = n * HP + s.hb + s.front + (t0 + g) * FEW_GRAN + jj;
                    H[at] = __float2bfloat16_rn(hi);
                    H[HLO + at] = __float2bfloat16_rn(hv - hi);
                }
                if (tl == 0) {  // zeros in the padding on both sides of the expert's units
                    const int pad = padded<S::HALIGN>(s) - s.len;
                    for (int i = tid; i < pad * s.n; i += CONSUMERS) {
                        const int q = i % pad, n = i / pad;
                        const int at = n * HP + s.hb + (q < s.front ? q : s.len + q);
                        H[at] = __float2bfloat16_rn(0.f);
                        H[HLO + at] = __float2bfloat16_rn(0.f);
                    }
                }
            }
        }
        named_sync(1, CONSUMERS);
        // ---------------------------------------------------- this part of the output
        for (int r0 = 0; r0 < d; r0 += 128 * S::RB) {
            const int nb = min(S::RB, (d - r0) / 128);
            hb = 0;
            for (int64_t s0 = g0; s0 < g1;) {
                const Seg s = segment<S::HALIGN>(a, r, v, s0, g1, hb);
                s0 = s.next;
                hb += padded<S::HALIGN>(s);
                float acc[S::RB][NT][4];
#pragma unroll
                for (int i = 0; i < S::RB; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[i][nt][q] = 0.f;
                // H fragments: matrices (high, k), (high, k + 8), (low, k), (low, k + 8)
                uint32_t hrow[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    hrow[nt] = hs + (lq >> 1) * S::HPART + min(nt * 8 + lm, s.n - 1) * S::HPITCH +
                               (s.hb + (lq & 1) * 8) * 2;
                if (S::Q4) {
                    constexpr int GG = G ? G : 128;
                    const int p0 = s.j0 / 32, p1 = (s.j0 + s.len + 31) / 32;
                    for (int pp = p0; pp < p1; pp += 8) {
                        const int np = min(8, p1 - pp), q0 = pp * 32 / GG;
                        const uint32_t st = wait();
                        if (!lost) {
                            for (int i = 0; i < np; ++i) {
                                const int gq = (pp + i) * 32 / GG - q0;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if (nt * 8 >= s.n) break;
                                    uint32_t b0[4], b1[4];
                                    ldmatrix4(hrow[nt] + (pp - p0 + i) * 64, b0);
                                    ldmatrix4(hrow[nt] + (pp - p0 + i) * 64 + 32, b1);
#pragma unroll
                                    for (int rb = 0; rb < S::RB; ++rb) {
                                        if (rb >= nb) break;
                                        const uint2 w = reinterpret_cast<const uint2*>(
                                            ring + (size_t)p.stage * slot + rb * 16384 +
                                            (i * 8 + warp) * 256)[lane];
                                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                                        uint32_t f[4];
                                        codes_to_frag(w.x, f);
                                        mma(c, f, b0[0], b0[1]);
                                        mma(c, f, b0[2], b0[3]);
                                        codes_to_frag(w.y, f);
                                        mma(c, f, b1[0], b1[1]);
                                        mma(c, f, b1[2], b1[3]);
                                        const uint32_t sa = st + S::SCALES + rb * 2048 + gq * 256 +
                                                            (warp * 16 + fg) * 2;
                                        const float sl = lds_bf16(sa), sh = lds_bf16(sa + 16);
                                        acc[rb][nt][0] = fmaf(c[0], sl, acc[rb][nt][0]);
                                        acc[rb][nt][1] = fmaf(c[1], sl, acc[rb][nt][1]);
                                        acc[rb][nt][2] = fmaf(c[2], sh, acc[rb][nt][2]);
                                        acc[rb][nt][3] = fmaf(c[3], sh, acc[rb][nt][3]);
                                    }
                                }
                            }
                        }
                        done();
                    }
                } else {
                    for (int c0 = 0; c0 < s.len; c0 += 64) {
                        const uint32_t st = wait();
                        if (!lost) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                if (c0 + u * 16 >= s.len) break;
                                uint32_t f[S::RB][4];
#pragma unroll
                                for (int rb = 0; rb < S::RB; ++rb) {
                                    if (rb >= nb) break;
                                    const int row = warp * 16 + (lq & 1) * 8 + lm;
                                    ldmatrix4(st + rb * 16384 + row * 128 +
                                                  (((u * 2 + (lq >> 1)) ^ lm) << 4),
                                              f[rb]);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if (nt * 8 >= s.n) break;
                                    uint32_t b[4];
                                    ldmatrix4(hrow[nt] + (c0 + u * 16) * 2, b);
#pragma unroll
                                    for (int rb = 0; rb < S::RB; ++rb) {
                                        if (rb >= nb) break;
                                        mma(acc[rb][nt], f[rb], b[0], b[1]);
                                        mma(acc[rb][nt], f[rb], b[2], b[3]);
                                    }
                                }
                            }
                        }
                        done();
                    }
                }
#pragma unroll
                for (int rb = 0; rb < S::RB; ++rb) {
                    if (rb >= nb) break;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int n = nt * 8 + 2 * ft;
                        float* q = a.part + (int64_t)(s.row + n) * d + r0 + rb * 128 + warp * 16 + fg;
                        if (n < s.n) {
                            q[0] = acc[rb][nt][0];
                            q[8] = acc[rb][nt][2];
                        }
                        if (n + 1 < s.n) {
                            q[d] = acc[rb][nt][1];
                            q[d + 8] = acc[rb][nt][3];
                        }
                    }
                }
            }
        }
    }
}

template <int G, int NT>
__global__ void __launch_bounds__(FFN_THREADS, 1)
    few_ffn_kernel(const __grid_constant__ CUtensorMap m2, const __grid_constant__ CUtensorMap m2s,
                   const __grid_constant__ FewArgs a, int slot, int stages) {
    using S = Shape<G, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + (-smem_addr(smem_raw) & 1023);
    uint8_t* Hs = ring + (size_t)slot * stages;
    float* red = reinterpret_cast<float*>(Hs + 2 * S::HPART);
    Routing& r = *reinterpret_cast<Routing*>(Hs + 2 * S::HPART + S::RED);
    uint64_t* full = reinterpret_cast<uint64_t*>(
        reinterpret_cast<uint8_t*>(&r) + (sizeof(Routing) + 15) / 16 * 16);
    uint64_t* empty = full + MAX_STAGES;
    int32_t* flags = reinterpret_cast<int32_t*>(empty + MAX_STAGES);  // dead, issued stages
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], CONSUMERS / 32);
        }
        flags[0] = flags[1] = 0;
        fence_mbar_init();
        if (G == 0) {
            prefetch_tmap(&m2);
            if (a.hsum) prefetch_tmap(&m2s);
        }
    }
    pdl_trigger();
    pdl_wait();  // the router's logits
    route_batch(a, r);
    if (tid >= CONSUMERS)
        produce<G, NT>(a, r, &m2, &m2s, ring, slot, stages, full, empty, &flags[1]);
    else
        consume<G, NT>(a, r, ring, slot, stages, full, empty, Hs, red, &flags[0]);
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
int launch_ffn(const CUtensorMap& m2, const CUtensorMap& m2s, const FewArgs& a, int smem_limit,
               cudaStream_t st) {
    using S = Shape<G, NT>;
    const int slot = S::slot(a.T);
    int stages = (int)(((size_t)smem_limit - S::fixed()) / slot);
    stages = stages > MAX_STAGES ? MAX_STAGES : stages;
    const size_t smem = S::fixed() + (size_t)slot * stages;
    auto kern = few_ffn_kernel<G, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_limit) !=
        cudaSuccess)
        return launch_result();
    launch_ex(true, kern, dim3(FEW_CTAS), dim3(FFN_THREADS), smem, st, m2, m2s, a, slot, stages);
    note_launch();
    return launch_result();
}

template <int NT>
int launch_ffn_group(const CUtensorMap& m2, const CUtensorMap& m2s, const FewArgs& a,
                     int smem_limit, cudaStream_t st) {
    switch (a.G) {
        case 0: return launch_ffn<0, NT>(m2, m2s, a, smem_limit, st);
        case 32: return launch_ffn<32, NT>(m2, m2s, a, smem_limit, st);
        case 64: return launch_ffn<64, NT>(m2, m2s, a, smem_limit, st);
        default: return launch_ffn<128, NT>(m2, m2s, a, smem_limit, st);
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

int launch_few_ffn(const CUtensorMap& m2, const CUtensorMap& m2s, const FewArgs& a, int smem_limit,
                   cudaStream_t st) {
    return a.T <= 8 ? launch_ffn_group<1>(m2, m2s, a, smem_limit, st)
                    : launch_ffn_group<2>(m2, m2s, a, smem_limit, st);
}

int launch_few_combine(const FewArgs& a, cudaStream_t st) {
    launch_ex(true, few_combine_kernel, dim3(a.d / CB_COLS, a.T), dim3(256), 0, st, a);
    note_launch();
    return launch_result();
}

}  // namespace moe
