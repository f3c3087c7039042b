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
//
// Measured (a call in a stream of calls, launches included, by box and batch): one token,
// d = 4096, h = 14336, 2 of 8 experts 117-122 us in bf16 (5.8-6.0 TB/s of weights), 50 us
// on 4 bits (3.6 TB/s); eight tokens over 160 experts and two shared ones, d = 5120, h =
// 1536, 319-343 us (6.1-6.5 TB/s) and 151-167 us; sixteen tokens on the first layer 435 us
// (6.4 TB/s) and 219-231 us.  In bf16 HBM bounds it.  On 4 bits no unit is full (issue
// slots 50 to 60 %, HBM 36 to 48 %, 8-bit products 13 to 20 %): what is left is latency
// between the instructions of four multiplying warps a scheduler.  10 to 12 us are the
// router, the routing and the combine.
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "few.h"
#include "kernels.h"
#include "plan.h"

namespace moe {

namespace {

constexpr int FT = FEW_MAX_T;
constexpr int PLANES = FEW_PLANES;

// The routing of the batch, worked out by every CTA for itself (128
// assignments at most) in shared memory.
struct Routing {
    uint32_t tokens[MAX_E];         // tokens that chose an expert, as bits
    uint32_t hit[MAX_E / 32];       // experts some token chose, as bits
    int32_t sel[FT * MAX_K];        // [t * k + j] expert
    float g[FT * MAX_K];            // its gate
    int32_t items;                  // hit experts + the shared one
    int32_t most;                   // tokens of the one that serves most
    int32_t V;                      // parts
    int32_t q, more;                // their weighted granules over V: quotient, remainder
    int32_t expert[FEW_MAX_ITEMS];  // expert of an item, -1: shared
    int32_t n[FEW_MAX_ITEMS];       // tokens it serves
    int32_t cost[FEW_MAX_ITEMS];    // weight of a granule
    int32_t at[FEW_MAX_ITEMS];      // weighted granules before it
    int32_t row0[FEW_MAX_ITEMS];    // first row of its partial outputs
    uint8_t tok[FEW_MAX_ITEMS][FT];
    float gate[FEW_MAX_ITEMS][FT];
};

// Where part v begins, and the part that holds x, on the scale of granules weighted
// by their items' costs: the first r.more parts are r.q + 1 long, the others r.q.
__device__ __forceinline__ int part_start(const Routing& r, int v) { return v * r.q + min(v, r.more); }
__device__ __forceinline__ int part_of(const Routing& r, int x) {
    const int q = r.q, more = r.more, longer = more * (q + 1);
    const bool in = x < longer;  // (one division)
    return (in ? 0 : more) + (x - (in ? 0 : longer)) / (in ? q + 1 : q);
}

// First and last part of an item of g granules.
__device__ __forceinline__ int first_part(const Routing& r, int i) { return part_of(r, r.at[i]); }
__device__ __forceinline__ int last_part(const Routing& r, int i, int g) {
    return part_of(r, r.at[i] + (g - 1) * r.cost[i]);
}

// Sum over this lane and the ones below.
__device__ __forceinline__ int warp_prefix(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

// Number of hit experts below e.
__device__ __forceinline__ int hits_below(const Routing& r, int e) {
    int n = 0;
    for (int w = 0; w < e >> 5; ++w) n += __popc(r.hit[w]);
    return n + __popc(r.hit[e >> 5] & ((1u << (e & 31)) - 1));
}

// fp32 as an unsigned integer of the same order (NaN as -inf, -0 as +0), and back.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint((v != v ? -INFINITY : v) + 0.f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Top-k and gates of token t by one warp, C experts a lane at a time: k rounds of
// a warp-wide maximum over the lanes' keys and, in a lane, what the experts
// before these left (lane j: the j-th best).  Equal keys go to the lower expert.
template <int C>
__device__ __forceinline__ void route_token(const FewArgs& a, int t, Routing& r) {
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k;
    const float* z = a.logits + (int64_t)t * E;
    uint32_t best = 0;              // keys of real experts are above 0
    int expert = 0x7fffffff;
    for (int e0 = 0; e0 < E; e0 += 32 * C) {
        uint32_t key[C + 1];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = e0 + i * 32 + lane;
            key[i] = e < E ? order_key(a.bias ? z[e] + a.bias[e] : z[e]) : 0u;
        }
        key[C] = best;
        const int kept = expert;
        best = 0;
        expert = 0x7fffffff;
        for (int j = 0; j < k; ++j) {
            uint32_t m = key[C];
#pragma unroll
            for (int i = 0; i < C; ++i) m = max(m, key[i]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, m);
            int e = key[C] == top ? kept : 0x7fffffff;
#pragma unroll
            for (int i = C - 1; i >= 0; --i)
                if (key[i] == top) e = min(e, e0 + i * 32 + lane);
            const int win = (int)__reduce_min_sync(0xffffffffu, (unsigned)e);
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (e0 + i * 32 + lane == win) key[i] = 0;
            if (kept == win) key[C] = 0;
            if (lane == j) {
                best = top;
                expert = win;
            }
        }
    }
    const float v = key_value(best);
    const float most = __shfl_sync(0xffffffffu, v, 0);  // by all lanes, outside the choice below
    const float p = lane < k ? expf(v - most) : 0.f;
    float sum = p;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < k) {
        r.sel[t * k + lane] = expert;
        r.g[t * k + lane] = p / sum;
        atomicOr(&r.tokens[expert], 1u << t);
        atomicOr(&r.hit[expert >> 5], 1u << (expert & 31));
    }
}

// Fills r: capacity in token order, the hit experts ascending with their
// tokens and gates, the shared expert last, and the rows of the partial
// outputs.  Called by every thread of the CTA; r.tokens and r.hit are zero.
__device__ void route_batch(const FewArgs& a, Routing& r) {
    const int tid = threadIdx.x, warp = tid >> 5;
    const int N = a.T * a.k, k = a.k;
    if (warp < a.T) {
        if (a.E <= 32) route_token<1>(a, warp, r);
        else route_token<8>(a, warp, r);
    }
    __syncthreads();
    const int A = hits_below(r, a.E - 1) + (r.tokens[a.E - 1] != 0);
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN, items = A + (gS > 0);
    if (tid < N) {
        const int e = r.sel[tid], t = tid / k, at = hits_below(r, e);
        const uint32_t who = r.tokens[e];
        const int rank = __popc(who & ((1u << t) - 1));
        if (rank == 0) {
            r.expert[at] = e;
            r.n[at] = (int)min((int64_t)__popc(who), a.C);
        }
        if (rank < a.C) {
            r.tok[at][rank] = (uint8_t)t;
            r.gate[at][rank] = r.g[tid];
        }
    }
    if (gS > 0 && tid < a.T) {
        r.tok[A][tid] = (uint8_t)tid;
        r.gate[A][tid] = 1.0f;
    }
    if (tid == 0) {
        if (gS) {
            r.expert[A] = -1;
            r.n[A] = a.T;
        }
        r.items = items;
    }
    __syncthreads();
    // two prefixes over the items: weighted granules, then tokens x parts
    if (tid < 32) {
        int before = 0, heaviest = 0, lightest = 1 << 30, most = 0;
        for (int i0 = 0; i0 < items; i0 += 32) {
            const int i = i0 + tid;
            const int cost = i < items ? few_cost(a.G, r.n[i]) : 0;
            const int w = cost * (i < A ? gE : gS);
            const int incl = warp_prefix(w);
            if (i < items) {
                r.cost[i] = cost;
                r.at[i] = before + incl - w;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
            heaviest = max(heaviest, (int)__reduce_max_sync(0xffffffffu, (unsigned)cost));
            lightest = min(lightest,
                           (int)__reduce_min_sync(0xffffffffu, i < items ? (unsigned)cost : 1u << 30));
            most = max(most, (int)__reduce_max_sync(0xffffffffu, i < items ? (unsigned)r.n[i] : 0u));
        }
        if (tid == 0) {
            r.most = most;
            const int V = few_parts(before, lightest, heaviest, gridDim.x);
            r.V = V;
            r.q = before / V;
            r.more = before % V;
        }
        __syncwarp();
        before = 0;
        for (int i0 = 0; i0 < items; i0 += 32) {
            const int i = i0 + tid;
            const int rows =
                i < items ? r.n[i] * (last_part(r, i, i < A ? gE : gS) - first_part(r, i) + 1) : 0;
            const int incl = warp_prefix(rows);
            if (i < items) r.row0[i] = before + incl - rows;
            before += __shfl_sync(0xffffffffu, incl, 31);
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
        const int routed = __popc(r.tokens[e]);
        a.routed[e] = routed;
        a.kept[e] = (int)min((int64_t)routed, a.C);
    }
    for (int i = tid; i < N + a.T; i += nthr) {
        const bool shared = i >= N;
        const int t = shared ? i - N : i / k;
        const int item = shared ? A : hits_below(r, r.sel[i]);
        const int pos = shared ? t : __popc(r.tokens[r.sel[i]] & ((1u << t) - 1));
        int4 row = make_int4(0, 0, 0, 0);
        if (shared ? gS > 0 : pos < a.C) {
            row.x = r.row0[item] + pos;
            row.y = last_part(r, item, shared ? gS : gE) - first_part(r, item) + 1;
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

// Tiled bulk tensor loads to a shared-memory address.
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map,
                                                 uint64_t* bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2),
        "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap* map,
                                                 uint64_t* bar, int c0, int c1, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "l"(policy)
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

// c (16 x 8, int32) += a (16 x 32) b (32 x 8), signed 8-bit
__device__ __forceinline__ void imma(int (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two code words (32 columns) as an A fragment of values 16 q.
__device__ __forceinline__ void codes_to_frag(uint32_t w0, uint32_t w1, uint32_t (&f)[4]) {
    constexpr uint32_t M = 0xF0F0F0F0u;
    f[0] = w0 & M;
    f[1] = (w0 << 4) & M;
    f[2] = w1 & M;
    f[3] = (w1 << 4) & M;
}

// Orders shared memory reached by ordinary accesses and cp.async before bulk copies to it.
__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// An integer of magnitude below 2^22 to fp32 (an addition instead of the slower
// conversion): a group's sum is at most 128 * 112 * 128 = 1.84 million.
__device__ __forceinline__ float small_int(int v) {
    return __int_as_float(v + 0x4B400000) - 12582912.f;
}

__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float((uint32_t)v << 16);
}

// ---------------------------------------------------------------- the expert kernel
//
// Sixteen warps multiply what four others bring in through a ring of stages:
// one issues the weights' copies (tensor maps for bf16, bulk copies for 4 bits),
// three copy the expert's token rows 16 bytes a lane; all signal the stage's
// mbarrier.  Weights are the A operand (16 rows), the tokens of one
// expert the B operand (8 columns a tile), so one instruction takes 256 or 512
// weights from registers whatever the number of tokens.
//
// First half, per granule (32 hidden units): four tiles of 16 rows, the gate and
// the up rows of 8 units each, so that a lane's accumulators hold both for the
// same unit and token.  Four warps share a tile's columns; their sums meet in
// shared memory at the end of d, where H = g silu(a) u is formed in fp32.  The
// four groups of warps wait for nothing of one another.  Second half: 256 rows of
// w2 (16 a warp) by the part's columns against H; the products of one expert go
// to the part's own rows of the partial outputs.
//
// bf16 weights: m16n8k16 products with fp32 sums, H as two bf16 parts: each unit is off by
// 2^-17 of itself at most, where the store of out rounds to 2^-8.  (A third part: one
// token wide 122.6 us against 116.7, and 1.0 instead of 1.5 in 1000 elements of out that
// are not the 64-bit value's rounding; the others are the fp32 sums'.)
//
// 4-bit weights: the products are exact.  A row of x is an integer of 31 bits
// times a power of two (of the row's largest magnitude: the rounding is 2^-30 of
// that at most), held as four planes of signed 8-bit digits; H likewise per expert
// and part.  An element of x keeps its 8 bits down to 2^-22 of the largest one, and
// one of H its 24 down to 2^-6.  (Three planes hold 23 bits: an element 10^4 times the
// others then costs the sums of units whose codes are 0 there 10^-3 of their size, one
// 10^5 times 10^-2, more than the bf16 store.  They take fewer tiles from five tokens
// on, two for five and three for eight: 8 tokens over 160 experts 143 us against 153,
// 16 tokens 206 against 230; below that the same.)  The planes are columns of one 8-bit
// product, which takes the codes after two masks and a shift per 8 codes -- as bf16
// fragments they took three shifts, four masks and four subtractions, and 30 clocks per
// 256 weights and scheduler against 11, where HBM brings 256 in 23; as f16 fragments (a
// nibble is an f16 subnormal as it lies, one column a token) they take twice the
// integer pipe's instructions: one token wide 63 us against 54.  Sums within a group
// are exact in int32; a group's scale multiplies its sum in fp32.
//
// Copied bf16 tiles are swizzled and token rows pitched by an odd multiple of 16
// bytes, so that ldmatrix meets no bank twice; codes arrive in fragment order and
// are read as they lie.
template <int G, int TT>   // group (0: bf16), most tokens
struct Shape {
    static constexpr bool Q4 = G > 0;
    static constexpr int GG = Q4 ? G : 128;
    static constexpr int KW = 4;                           // warps along the columns
    static constexpr int KB = Q4 ? 128 : 64;               // least columns of a warp in a stage
    static constexpr int QB = q13_block_bytes(GG);
    static constexpr int XROWS = Q4 ? PLANES : 1;          // rows of a stage per token
    static constexpr int XBYTES = Q4 ? 1 : 2;              // bytes of an element
    // a stage of the second half: 2 blocks of 128 rows x panels of 32 units, with 4
    // bits then the scales of the groups they meet (one more than they fill, unless a
    // group is a panel)
    static constexpr int PANEL = Q4 ? 2048 : 8192;         // bytes of 128 rows of a panel
    // in bf16 they end where the first half's token rows begin (4 bits: see done())
    static_assert(Q4 || KW * KB * 128 >= 4 * PANEL, "token rows are no bulk copy's target");
    static __device__ __forceinline__ int groups(int panels) {
        return GG == 32 ? panels : panels * 32 / GG + 1;
    }
    static __device__ __forceinline__ int down(int panels) {
        return 2 * panels * PANEL + (Q4 ? 2 * groups(panels) * 256 : 0);
    }
    // H: bf16 high, then low parts of the tokens' rows; 4 bits: a row first fp32, then
    // its planes HPLANE bytes apart (33 and 132 times 16 bytes: the rows of two tokens'
    // planes meet no bank twice)
    static constexpr int HPLANE = FEW_HCAP + 16;
    static constexpr int HPITCH = Q4 ? PLANES * HPLANE : (FEW_HCAP + 8) * 2;
    static_assert(!Q4 || FEW_HCAP * 4 <= HPITCH, "the planes fit the row they replace");
};

// Shared memory of one call: the ring, H and the warps' sums are sized by the most
// tokens an expert of the batch serves, not by the batch.
struct Geometry {
    int blocks;   // blocks of KB columns of a warp in a stage of the first half
    int panels;   // panels of 32 hidden units in a stage of the second
    int ka;       // columns of a stage of the first half
    int xpitch;   // bytes of a token's row in it, and where the rows begin
    int xoff;
    int slot;     // bytes of a stage
    int stages;
    int nt;       // tiles of 8 tokens
    int hpart;    // bytes from H's high to its low parts (bf16)
    int h, red;   // where H and the warps' sums begin, behind the ring
};

constexpr int MAX_STAGES = 12;

// 4 bits: stages of two blocks of columns where two of them fit, else of one: fewer
// stages are fewer waits (one token, d = 4096, h = 14336, 2 of 8 experts: 54.6 us
// against 63.8).  Only where three fit: 16 tokens on that layer 243 us against 228, 8
// over 160 experts 147.5 against 150.  Eight panels always: four were slower at every
// size tried.
template <typename S>
__device__ __forceinline__ Geometry geometry(int tokens, int bytes) {
    Geometry g;
    g.nt = (tokens + 7) / 8;
    g.hpart = g.nt * 8 * S::HPITCH;
    const int h = (S::Q4 ? tokens * S::HPITCH : 2 * g.hpart + 15) / 16 * 16;
    const int red = 2 * 16 * g.nt * 640;   // two granules' sums of 16 warps
    const int ring = bytes - h - red;
#pragma unroll
    for (int blocks = S::Q4 ? 2 : 1; blocks >= 1; --blocks) {
        g.blocks = blocks;
        g.panels = S::Q4 ? 8 : 2;
        g.ka = S::KW * S::KB * blocks;
        g.xpitch = g.ka * S::XBYTES + 16;
        g.xoff = S::Q4 ? g.ka / 128 * S::QB : g.ka * 128;
        const int up = g.xoff + tokens * S::XROWS * g.xpitch;
        g.slot = (max(up, S::down(g.panels)) + 1023) / 1024 * 1024;
        g.stages = min(ring / g.slot, MAX_STAGES);
        if (g.stages >= 2) break;
    }
    g.h = g.stages * g.slot;
    g.red = g.h + h;
    return g;
}

constexpr int CONSUMERS = 512;
constexpr int TOKEN_WARPS = 3;
constexpr int FFN_THREADS = CONSUMERS + 32 + TOKEN_WARPS * 32;
constexpr int MAX_SEGS = FEW_HCAP / 128 + 2;  // experts (at least 128 units each) a part can meet

// One expert's share of a part.
struct Seg {
    int item, expert, n;   // expert -1: shared; tokens
    int j0, len;           // hidden units j0 .. j0 + len
    int row;               // its first row of the partial outputs
    int hb;                // where its H begins

    // Panels of 32 units a stage of the second half takes: as few stages of at most
    // `most` as there can be, of even size.
    __device__ __forceinline__ int step(int most) const {
        const int panels = len / 32, stages = (panels + most - 1) / most;
        return (panels + stages - 1) / stages;
    }
};

// A warp writes part v's shares to segs; returns how many there are.  A granule
// belongs to the part in which it begins.
__device__ __forceinline__ int segments(const FewArgs& a, const Routing& r, int v, Seg* segs) {
    const int lane = threadIdx.x & 31;
    const int gE = a.h / FEW_GRAN, gS = a.hsum / FEW_GRAN;
    const int A = r.items - (gS > 0);
    const int w0 = part_start(r, v), w1 = part_start(r, v + 1);
    int first = -1;  // the last item that begins at or before w0
    for (int i0 = 0; i0 < r.items; i0 += 32)
        first += __popc(__ballot_sync(0xffffffffu, i0 + lane < r.items && r.at[i0 + lane] <= w0));
    const int i = first + lane;
    int s0 = 0, s1 = 0;
    if (lane <= MAX_SEGS && i < r.items) {
        const int at = r.at[i], cost = r.cost[i], g = i < A ? gE : gS;
        s0 = max(0, (w0 - at + cost - 1) / cost);
        s1 = min(g, max(0, (w1 - at + cost - 1) / cost));
    }
    const bool have = s0 < s1;
    const int len = have ? (s1 - s0) * FEW_GRAN : 0;
    const int hb = warp_prefix(len) - len;
    const uint32_t all = __ballot_sync(0xffffffffu, have);
    __syncwarp();
    if (have) {
        Seg s;
        s.item = i;
        s.expert = r.expert[i];
        s.n = r.n[i];
        s.j0 = s0 * FEW_GRAN;
        s.len = len;
        s.row = r.row0[i] + (v - first_part(r, i)) * s.n;
        s.hb = hb;
        segs[__popc(all & ((1u << lane) - 1))] = s;
    }
    __syncwarp();
    return __popc(all);
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

// A bringing warp's side of the ring.
struct Bringer {
    uint8_t* ring;
    uint64_t *full, *empty;
    uint64_t limit;
    Geometry geo;
    Ring p;

    // Waits until the stage is free; false if the wait ran out (the same in all lanes).
    __device__ __forceinline__ bool open() {
        return __all_sync(0xffffffffu, mbar_wait(&empty[p.stage], p.phase ^ 1, limit));
    }
    __device__ __forceinline__ uint32_t at() const { return smem_addr(ring) + p.stage * geo.slot; }
    __device__ __forceinline__ uint64_t* bar() const { return &full[p.stage]; }
};

// The weights' copies, stage by stage: per part the first half (experts, granules,
// columns), then the second (experts, 256 rows of d, panels).  False when a wait
// ran out.
template <int G, int TT>
__device__ __forceinline__ bool bring_weights(const FewArgs& a, const Routing& r,
                                              const FewMaps& maps, Seg* segs, Bringer c,
                                              int32_t* issued) {
    using S = Shape<G, TT>;
    const int lane = threadIdx.x & 31;
    const int d = a.d;
    const uint64_t once = l2_policy_evict_first();
    int count = 0;
    auto announce = [&](uint32_t bytes) {
        if (lane == 0) {
            mbar_arrive_expect_tx(c.bar(), bytes);
            *issued = ++count;
        }
        __syncwarp();
    };
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        const int nseg = segments(a, r, v, segs);
        for (int i = 0; i < nseg; ++i) {
            const Seg s = segs[i];
            const bool shared = s.expert < 0;
            const int hid = shared ? a.hsum : a.h, e = shared ? 0 : s.expert;
            const CUtensorMap* map = shared ? &maps.w13s : &maps.w13;
            // 4 bits: the granules of a share follow one another
            const uint8_t* src = reinterpret_cast<const uint8_t*>(shared ? a.w13s : a.w13) +
                                 ((int64_t)e * (hid / 32) + s.j0 / 32) * (d / 128) * S::QB;
            int block = 2 * (int)(((int64_t)e * hid + s.j0) / 128), row = s.j0 % 128;
            for (int j = 0; j < s.len; j += FEW_GRAN) {
                for (int k0 = 0; k0 < d; k0 += c.geo.ka) {
                    const int kn = min(c.geo.ka, d - k0);
                    if (!c.open()) return false;
                    if (S::Q4) {
                        const uint32_t bytes = kn / 128 * S::QB;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(c.bar(), bytes);
                            bulk_load(c.at(), src, bytes, c.bar(), once);
                            *issued = ++count;
                        }
                        src += bytes;
                    } else {
                        announce(kn * 128);
                        if (lane < kn / 64)
                            tma_load_3d_hint(c.at() + lane * 8192, map, c.bar(), k0 + lane * 64, row,
                                             block, once);
                    }
                    c.p.next();
                }
                row += FEW_GRAN;
                if (row == 128) {
                    row = 0;
                    block += 2;
                }
            }
        }
        for (int i = 0; i < nseg; ++i) {
            const Seg s = segs[i];
            const bool shared = s.expert < 0;
            const int hid = shared ? a.hsum : a.h, e = shared ? 0 : s.expert;
            const CUtensorMap* map = shared ? &maps.w2s : &maps.w2;
            // this lane's copy of a stage: block of rows and, for 4 bits, codes (0) or
            // scales (1), else the panel
            const int b = lane & 1, what = lane >> 1, step = s.step(c.geo.panels);
            const uint8_t* codes = reinterpret_cast<const uint8_t*>(shared ? a.w2s : a.w2);
            const uint8_t* scales = codes + q2_code_bytes(shared ? 1 : a.E, hid, d);
            const int block = c.geo.panels * S::PANEL, scale = S::groups(c.geo.panels) * 256;
            codes += ((int64_t)e * (d / 128) + b) * (hid / 32) * 2048;
            scales += ((int64_t)e * (d / 128) + b) * (hid / S::GG) * 256;
            for (int r0 = 0; r0 < d; r0 += 256) {
                const int nb = min(2, (d - r0) / 128);
                for (int p0 = 0; p0 < s.len / 32; p0 += step) {
                    const int np = min(step, s.len / 32 - p0);
                    const int pp = s.j0 / 32 + p0;
                    if (!c.open()) return false;
                    if (S::Q4) {
                        const int q0 = pp * 32 / S::GG, nq = ((pp + np) * 32 - 1) / S::GG - q0 + 1;
                        announce(nb * (np * 2048 + nq * 256));
                        if (b < nb && what < 2)
                            bulk_load(c.at() + (what ? 2 * block + b * scale : b * block),
                                      what ? scales + q0 * 256 : codes + (int64_t)pp * 2048,
                                      what ? nq * 256 : np * 2048, c.bar(), once);
                    } else {
                        announce(nb * np * 8192);
                        if (b < nb && what < np)
                            tma_load_2d_hint(c.at() + lane * 8192, map, c.bar(),
                                             s.j0 + (p0 + what) * 32, e * d + r0 + 128 * b, once);
                    }
                    c.p.next();
                }
                codes += (int64_t)2 * (hid / 32) * 2048;
                scales += (int64_t)2 * (hid / S::GG) * 256;
            }
        }
    }
    return true;
}

// The token rows of the first half (x, or its planes), 16 bytes a lane, by warp
// `share` of TOKEN_WARPS; every lane arrives on every stage, when its copies have
// landed.
template <int G, int TT>
__device__ __forceinline__ bool bring_tokens(const FewArgs& a, const Routing& r, Seg* segs,
                                             Bringer c, int share) {
    using S = Shape<G, TT>;
    const int rowbytes = c.geo.ka * S::XBYTES;  // of a stage: one copy of every lane, or two
    const int lane = threadIdx.x & 31;
    const int pitch = a.d * S::XBYTES;  // bytes of a row in memory
    const uint8_t* x = reinterpret_cast<const uint8_t*>(S::Q4 ? (const void*)a.xq : a.x) + lane * 16;
    for (int v = blockIdx.x; v < r.V; v += gridDim.x) {
        const int nseg = segments(a, r, v, segs);
        for (int i = 0; i < nseg; ++i) {
            const Seg s = segs[i];
            const int rows = s.n * S::XROWS;
            // lane q keeps where this warp's q-th row begins
            const int mine = share + TOKEN_WARPS * lane;
            const int64_t at = mine < rows ? ((int64_t)r.tok[s.item][mine / S::XROWS] * S::XROWS +
                                              mine % S::XROWS) * pitch
                                           : 0;
            for (int j = 0; j < s.len; j += FEW_GRAN)
                for (int k0 = 0; k0 < pitch; k0 += rowbytes) {
                    if (!c.open()) return false;
                    const uint32_t dst = c.at() + c.geo.xoff + lane * 16;
                    for (int q = 0, row = share; row < rows; ++q, row += TOKEN_WARPS) {
                        const int64_t from = __shfl_sync(0xffffffffu, at, q);
                        const uint8_t* src = x + from + k0;
                        const uint32_t to = dst + row * c.geo.xpitch;
                        if (k0 + lane * 16 < pitch) cp_async16(to, src);
                        if (rowbytes > 512 && k0 + 512 + lane * 16 < pitch)
                            cp_async16(to + 512, src + 512);
                    }
                    cp_async_arrive(c.bar());
                    c.p.next();
                }
        }
        for (int i = 0; i < nseg; ++i) {
            const int step = segs[i].step(c.geo.panels);
            const int stages = (a.d + 255) / 256 * ((segs[i].len / 32 + step - 1) / step);
            for (int q = 0; q < stages; ++q) {
                if (!c.open()) return false;
                mbar_arrive(c.bar());
                c.p.next();
            }
        }
    }
    return true;
}

// What a multiplying warp knows of its place and of the ring.
struct Consumer {
    uint8_t* ring;
    uint64_t *full, *empty;
    int32_t* flags;
    int32_t* status;
    uint64_t limit;
    Geometry geo;
    Ring p;
    bool lost = false;  // a wait ran out: go on without waiting, so that the barriers are met

    __device__ __forceinline__ uint8_t* wait() {
        if (!lost && !mbar_wait(&full[p.stage], p.phase, limit)) {
            lost = true;
            flags[0] = 1;
            report_timeout(status);
        }
        lost = __any_sync(0xffffffffu, lost);
        return ring + (size_t)p.stage * geo.slot;
    }
    // Gives the stage back.  FENCE: it holds token rows, and the stage's next weights may
    // lie over them (4 bits: codes and scales of the second half reach past xoff).  The
    // rows came by cp.async, the weights come by bulk copies, and the barriers alone do not
    // order accesses of the two proxies.
    template <bool FENCE>
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            if (FENCE) fence_proxy_async();
            mbar_arrive(&empty[p.stage]);
        }
        p.next();
    }
};

// First half, bf16: this warp's sums over d of tile gw's rows by the expert's
// tokens.  red: where they go, [NT][8 tokens][20] floats.
template <int TT>
__device__ __forceinline__ void up_bf16(Consumer& c, const Seg& s, int d, float* red) {
    using S = Shape<0, TT>;
    constexpr int NT = (TT + 7) / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kw = warp & 3, gw = warp >> 2;
    const int lm = lane & 7, lq = lane >> 3;         // row and matrix of an ldmatrix address
    // rows of tokens past the expert's repeat its last one: their columns of the
    // product are never read
    uint32_t xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        xrow[nt] = c.geo.xoff + min(nt * 8 + lm, s.n - 1) * c.geo.xpitch + (kw * S::KB + lq * 8) * 2;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[nt][q] = 0.f;
    for (int k0 = 0; k0 < d; k0 += c.geo.ka) {
        const uint32_t st = smem_addr(c.wait());
        if (!c.lost && k0 + kw * S::KB < d) {
            uint32_t b[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt * 8 < s.n) {
                    ldmatrix4(st + xrow[nt], b[nt][0]);
                    ldmatrix4(st + xrow[nt] + 64, b[nt][1]);
                }
            // box of this warp's 64 columns: 32 gate rows, 32 up rows
            const uint32_t wa = st + kw * 8192 + ((lq & 1) * 32 + gw * 8 + lm) * 128;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t f[4];
                ldmatrix4(wa + (((u * 2 + (lq >> 1)) ^ lm) << 4), f);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt * 8 < s.n)
                        mma(acc[nt], f, b[nt][u / 2][2 * (u & 1)], b[nt][u / 2][2 * (u & 1) + 1]);
            }
        }
        c.done<false>();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= s.n) break;
        float* q = red + nt * 160 + 2 * (lane & 3) * 20 + (lane >> 2);
        q[0] = acc[nt][0];
        q[20] = acc[nt][1];
        q[8] = acc[nt][2];
        q[28] = acc[nt][3];
    }
}

// Column c of the 4-bit products is token c / 4, plane c % 4: a tile of 8 columns
// holds two tokens.  Where its second token is past the last one, this lane's ldmatrix
// address is to go back by so many rows: they repeat the last token's, and their
// columns are not used.  (Up to four tiles there are as many as n needs.)
template <int TILES>
__device__ __forceinline__ int rows_back(int t, int n) {
    return (TILES <= 4 && t < TILES - 1) || 2 * t + 1 < n ? 0 : threadIdx.x & 4;
}

// The planes of a tile joined, the highest with weight 1.  A lane holds two planes of
// token ft / 2 (ft = lane & 3; low ones where ft is even) in rows lane / 4 and lane / 4
// + 8; it gets the sum of row lane / 4 + 8 (ft & 1).
__device__ __forceinline__ float join_planes(const float (&v)[4]) {
    constexpr float D = 1.f / 256.f;
    const bool high = threadIdx.x & 1;
    const float up = fmaf(v[0], D, v[1]), down = fmaf(v[2], D, v[3]);
    const float other = __shfl_xor_sync(0xffffffffu, high ? up : down, 1);
    return high ? fmaf(other, D * D, down) : fmaf(up, D * D, other);
}

// The same for 4 bits; TILES: tiles of 8 columns, up to four all computed, so that
// their products overlap.
template <int G, int TT, int TILES>
__device__ __forceinline__ void up_q4(Consumer& c, const Seg& s, int d, float* red) {
    using S = Shape<G, TT>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kw = warp & 3, gw = warp >> 2;
    const uint32_t xrow = c.geo.xoff + (lane & 7) * c.geo.xpitch + kw * c.geo.blocks * 128 + (lane >> 3) * 16;
    float acc[TILES][4];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
    auto block = [&](const uint8_t* stp, int kb) {
        const int blk = kw * c.geo.blocks + kb;
        const uint4* cw = reinterpret_cast<const uint4*>(stp + blk * S::QB + gw * 1024);
        const uint32_t st = smem_addr(stp);
        uint32_t f[4][4];
        {
            const uint4 lo = cw[lane], hi = cw[32 + lane];
            codes_to_frag(lo.x, lo.y, f[0]);
            codes_to_frag(lo.z, lo.w, f[1]);
            codes_to_frag(hi.x, hi.y, f[2]);
            codes_to_frag(hi.z, hi.w, f[3]);
        }
        const uint32_t sa = st + blk * S::QB + 4096 + (gw * 16 + (lane >> 2)) * 2;
        float sl[128 / S::GG], sh[128 / S::GG];
#pragma unroll
        for (int q = 0; q < 128 / S::GG; ++q) {
            sl[q] = lds_bf16(sa + q * 128);
            sh[q] = lds_bf16(sa + q * 128 + 16);
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            if (TILES > 4 && 2 * t >= s.n) break;
            const uint32_t at = st + xrow + (t * 8 - rows_back<TILES>(t, s.n)) * c.geo.xpitch + kb * 128;
            uint32_t b[2][4];
            ldmatrix4(at, b[0]);
            ldmatrix4(at + 64, b[1]);
#pragma unroll
            for (int q = 0; q < 128 / S::GG; ++q) {
                int g[4] = {0, 0, 0, 0};
#pragma unroll
                for (int u = q * (S::GG / 32); u < (q + 1) * (S::GG / 32); ++u)
                    imma(g, f[u], b[u / 2][2 * (u & 1)], b[u / 2][2 * (u & 1) + 1]);
                acc[t][0] = fmaf(small_int(g[0]), sl[q], acc[t][0]);
                acc[t][1] = fmaf(small_int(g[1]), sl[q], acc[t][1]);
                acc[t][2] = fmaf(small_int(g[2]), sh[q], acc[t][2]);
                acc[t][3] = fmaf(small_int(g[3]), sh[q], acc[t][3]);
            }
        }
    };
    for (int k0 = 0; k0 < d; k0 += c.geo.ka) {
        const uint8_t* stp = c.wait();
        const int left = c.lost ? 0 : d - k0 - kw * c.geo.blocks * 128;
        if (c.geo.blocks == 2 && left > 128) {
            block(stp, 0);
            block(stp, 1);
        } else if (left > 0) {
            block(stp, 0);
        }
        c.done<true>();
    }
    // (20 floats a token)
    red += ((lane & 3) >> 1) * 20 + (lane & 1) * 8 + (lane >> 2);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        if (TILES > 4 && 2 * t >= s.n) break;
        red[t * 40] = join_planes(acc[t]);
    }
}

// Second half, bf16: this warp's 16 rows (of 256 from r0) by the part's share of
// one expert.  out: its row of the first token at the lane's row of the tile.
template <int TT>
__device__ __forceinline__ void down_bf16(Consumer& c, const Seg& s, int d, bool mine, uint32_t hs,
                                          float* out) {
    using S = Shape<0, TT>;
    constexpr int NT = (TT + 7) / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rb = warp >> 3, tile = warp & 7;
    const int lm = lane & 7, lq = lane >> 3;
    // H fragments: matrices (high, k), (high, k + 8), (low, k), (low, k + 8); one
    // chain of products for each part
    uint32_t hrow[NT];
    float acc[NT][4], low[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        hrow[nt] = hs + (lq >> 1) * c.geo.hpart + min(nt * 8 + lm, s.n - 1) * S::HPITCH +
                   (s.hb + (lq & 1) * 8) * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[nt][q] = low[nt][q] = 0.f;
    }
    const int step = s.step(c.geo.panels);
    for (int p0 = 0; p0 < s.len / 32; p0 += step) {
        const int np = min(step, s.len / 32 - p0);
        const uint32_t st = smem_addr(c.wait());
        if (!c.lost && mine) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (q >= np) break;
                // box (q, rb): 128 rows of 64 bytes
                const uint32_t wa =
                    st + (q * 2 + rb) * S::PANEL + (tile * 16 + (lq & 1) * 8 + lm) * 64;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t f[4];
                    ldmatrix4(wa + (((u * 2 + (lq >> 1)) ^ ((lm >> 1) & 3)) << 4), f);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (nt * 8 < s.n) {
                            uint32_t b[4];
                            ldmatrix4(hrow[nt] + (p0 + q) * 64 + u * 32, b);
                            mma(acc[nt], f, b[0], b[1]);
                            mma(low[nt], f, b[2], b[3]);
                        }
                }
            }
        }
        c.done<false>();
    }
    if (mine) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = nt * 8 + 2 * (lane & 3);
            float* q = out + (int64_t)n * d;
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

// The same for 4 bits.  hf: what the planes of H are multiplied by, per token.
template <int G, int TT, int TILES>
__device__ __forceinline__ void down_q4(Consumer& c, const Seg& s, int d, bool mine, uint32_t hs,
                                        const float* hf, float* out) {
    using S = Shape<G, TT>;
    constexpr int PG = S::GG / 32;  // panels of a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rb = warp >> 3, tile = warp & 7;
    const uint32_t hrow = hs + (lane & 7) * S::HPLANE + s.hb + (lane >> 3) * 16;
    float acc[TILES][4];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
    const int step = s.step(c.geo.panels);
    for (int p0 = 0; p0 < s.len / 32; p0 += step) {
        const int np = min(step, s.len / 32 - p0);
        const uint8_t* stp = c.wait();
        if (!c.lost && mine) {
            const int first = s.j0 / 32 + p0, q0 = first / PG;
            const int block = c.geo.panels * S::PANEL, scale = S::groups(c.geo.panels) * 256;
            const uint2* cw = reinterpret_cast<const uint2*>(stp + rb * block + tile * 256) + lane;
            const uint32_t sa = smem_addr(stp) + 2 * block + rb * scale +
                                (tile * 16 + (lane >> 2)) * 2;
            // the panels of one group at a time: their sum is exact
            for (int p = 0; p < np;) {
                const int gq = (first + p) / PG - q0;
                const int pe = min(np, (q0 + gq + 1) * PG - first);
                const float sl = lds_bf16(sa + gq * 256), sh = lds_bf16(sa + gq * 256 + 16);
                // tiles side by side as long as their sums fit
                constexpr int N = TILES == 4 ? 2 : TILES > 4 ? 1 : TILES;
#pragma unroll
                for (int t0 = 0; t0 < TILES; t0 += N) {
                    if (TILES > 4 && 2 * t0 >= s.n) break;
                    int g[N][2][4];
#pragma unroll
                    for (int t = 0; t < N; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) g[t][0][q] = g[t][1][q] = 0;
#pragma unroll
                    for (int i = 0; i < PG; i += 2) {  // an H fragment serves two panels
                        if (i > 0 && p + i >= pe) break;
                        uint32_t f[2][4];
                        const uint2 w0 = cw[(p + i) * 256];
                        codes_to_frag(w0.x, w0.y, f[0]);
                        if (PG > 1) {  // (a panel past the group: zero codes)
                            const uint2 w1 = p + i + 1 < pe ? cw[(p + i + 1) * 256] : make_uint2(0, 0);
                            codes_to_frag(w1.x, w1.y, f[1]);
                        }
#pragma unroll
                        for (int t = 0; t < N; ++t) {
                            uint32_t b[4];
                            const int row = (t0 + t) * 8 - rows_back<TILES>(t0 + t, s.n);
                            ldmatrix4(hrow + row * S::HPLANE + (p0 + p + i) * 32, b);
                            imma(g[t][0], f[0], b[0], b[1]);
                            if (PG > 1) imma(g[t][1], f[1], b[2], b[3]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        float* o = acc[t0 + t];
                        o[0] = fmaf(small_int(g[t][0][0] + g[t][1][0]), sl, o[0]);
                        o[1] = fmaf(small_int(g[t][0][1] + g[t][1][1]), sl, o[1]);
                        o[2] = fmaf(small_int(g[t][0][2] + g[t][1][2]), sh, o[2]);
                        o[3] = fmaf(small_int(g[t][0][3] + g[t][1][3]), sh, o[3]);
                    }
                }
                p = pe;
            }
        }
        c.done<false>();
    }
    if (!mine) return;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        if (TILES > 4 && 2 * t >= s.n) break;
        const float y = join_planes(acc[t]);
        const int n = 2 * t + ((lane & 3) >> 1);
        if (n < s.n) out[(int64_t)n * d + (lane & 1) * 8] = y * hf[n];
    }
}

// A value below 2^30 as signed digits of 8 bits, low first.
__device__ __forceinline__ void digits(float scaled, int8_t (&p)[PLANES]) {
    int v = __float2int_rn(scaled);
#pragma unroll
    for (int i = 0; i < PLANES; ++i) {
        p[i] = (int8_t)v;
        v = (v - p[i]) >> 8;
    }
}

// Exponent e that brings magnitudes up to m (finite) to [2^29, 2^30); the smallest end
// lower, where every fp32 is a whole number already.  v 2^e by two products (2^e may not
// be an fp32).
__device__ __forceinline__ int plane_exponent(float m) { return m > 0.f ? min(29 - ilogbf(m), 160) : 0; }
// What the joined planes' products are multiplied by: the codes come as 16 q, and the
// highest plane counts 2^24.
__device__ __forceinline__ float plane_unit(int e) { return scalbnf(1.f, 20 - e); }
__device__ __forceinline__ float2 plane_factors(int e) {
    const int some = min(e, 100);
    return make_float2(scalbnf(1.f, some), scalbnf(1.f, e - some));
}

template <int G, int TT>
__device__ void consume(const FewArgs& a, const Routing& r, Seg* segs, uint8_t* ring,
                        const Geometry& geo, uint64_t* full, uint64_t* empty, uint8_t* Hs,
                        float* red, float (*hf)[FT], int32_t* flags) {
    using S = Shape<G, TT>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gw = warp >> 2, gt = tid & 127;  // group of four warps; thread of the group
    const int d = a.d;
    Consumer c;
    c.ring = ring;
    c.full = full;
    c.empty = empty;
    c.flags = flags;
    c.status = a.status;
    c.limit = a.wait_limit_ns;
    c.geo = geo;
    c.p.stages = geo.stages;
    int turn = 0;  // which half of red
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
            const int jj = gt & 7, n = gt >> 3;  // the unit of the group's 8, and the token
            const float gate = n < s.n ? r.gate[s.item][n] : 0.f;
            const float xf = S::Q4 && n < s.n ? a.xf[r.tok[s.item][n]] : 1.f;
            for (int j = 0; j < s.len; j += FEW_GRAN, turn ^= 1) {
                float* base = red + turn * (16 * geo.nt * 160);
                float* mine = base + warp * (geo.nt * 160);
                if constexpr (!S::Q4)
                    up_bf16<TT>(c, s, d, mine);
                else if (TT <= 2 || s.n <= 2)
                    up_q4<G, TT, 1>(c, s, d, mine);
                else if (s.n <= 4)
                    up_q4<G, TT, TT <= 2 ? 1 : 2>(c, s, d, mine);
                else if (s.n <= 6)
                    up_q4<G, TT, TT <= 2 ? 1 : 3>(c, s, d, mine);
                else if (TT <= 8 || s.n <= 8)
                    up_q4<G, TT, TT <= 2 ? 1 : 4>(c, s, d, mine);
                else
                    up_q4<G, TT, TT <= 2 ? 1 : TT <= 8 ? 4 : 8>(c, s, d, mine);
                named_sync(2 + gw, 128);
                if (n < s.n) {
                    float ga = 0.f, up = 0.f;
#pragma unroll
                    for (int w = 0; w < S::KW; ++w) {
                        // (a tile of 8 tokens is 160 floats)
                        const float* q = base + (gw * 4 + w) * (geo.nt * 160) + n * 20 + jj;
                        ga += q[0];
                        up += q[8];
                    }
                    const int at = s.hb + j + gw * 8 + jj;
                    const float hv = silu_f(ga * xf) * (up * xf) * gate;
                    if (S::Q4) {
                        reinterpret_cast<float*>(Hs + n * S::HPITCH)[at] = hv;
                    } else {
                        __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(Hs + n * S::HPITCH);
                        const float hi = bf16_round(hv);
                        H[at] = __float2bfloat16_rn(hi);
                        H[geo.hpart / 2 + at] = __float2bfloat16_rn(hv - hi);
                    }
                }
            }
        }
        named_sync(1, CONSUMERS);
        if constexpr (S::Q4) {
            // a warp turns a token's row into planes, in place
            if (warp < r.most) {
                const float* row = reinterpret_cast<const float*>(Hs + warp * S::HPITCH);
                float h[FEW_HCAP / 32];
#pragma unroll
                for (int q = 0; q < FEW_HCAP / 32; ++q) h[q] = row[q * 32 + lane];
                __syncwarp();
                for (int i = 0; i < nseg; ++i) {
                    const Seg& s = segs[i];
                    if (warp >= s.n) continue;
                    const int p0 = s.hb / 32, p1 = (s.hb + s.len) / 32;
                    float m = 0.f;
                    bool odd = false;  // infinities and NaN: the token's output is NaN
#pragma unroll
                    for (int q = 0; q < FEW_HCAP / 32; ++q)
                        if (q >= p0 && q < p1) {
                            m = fmaxf(m, fabsf(h[q]));
                            odd |= !(fabsf(h[q]) < INFINITY);
                        }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    odd = __any_sync(0xffffffffu, odd);
                    const int e = odd ? 0 : plane_exponent(m);
                    const float2 by = plane_factors(e);
                    int8_t* dst = reinterpret_cast<int8_t*>(Hs + warp * S::HPITCH) + lane;
#pragma unroll
                    for (int q = 0; q < FEW_HCAP / 32; ++q)
                        if (q >= p0 && q < p1) {
                            int8_t pl[PLANES];
                            digits(odd ? 0.f : h[q] * by.x * by.y, pl);
#pragma unroll
                            for (int k = 0; k < PLANES; ++k) dst[k * S::HPLANE + q * 32] = pl[k];
                        }
                    if (lane == 0) hf[i][warp] = odd ? NAN : plane_unit(e);
                }
            }
            named_sync(1, CONSUMERS);
        }
        // ---------------------------------------------------- this part of the output
        const uint32_t hs = smem_addr(Hs);
        const int rb = warp >> 3, tile = warp & 7;  // this warp's 16 rows of 256
        for (int i = 0; i < nseg; ++i) {
            const Seg s = segs[i];
            float* out = a.part + (int64_t)s.row * d + rb * 128 + tile * 16 + (lane >> 2);
            for (int r0 = 0; r0 < d; r0 += 256, out += 256) {
                const bool mine = r0 + rb * 128 < d;
                if constexpr (!S::Q4)
                    down_bf16<TT>(c, s, d, mine, hs, out);
                else if (TT <= 2 || s.n <= 2)
                    down_q4<G, TT, 1>(c, s, d, mine, hs, hf[i], out);
                else if (s.n <= 4)
                    down_q4<G, TT, TT <= 2 ? 1 : 2>(c, s, d, mine, hs, hf[i], out);
                else if (s.n <= 6)
                    down_q4<G, TT, TT <= 2 ? 1 : 3>(c, s, d, mine, hs, hf[i], out);
                else if (TT <= 8 || s.n <= 8)
                    down_q4<G, TT, TT <= 2 ? 1 : 4>(c, s, d, mine, hs, hf[i], out);
                else
                    down_q4<G, TT, TT <= 2 ? 1 : TT <= 8 ? 4 : 8>(c, s, d, mine, hs, hf[i], out);
            }
        }
    }
}

template <int G, int TT>
__global__ void __launch_bounds__(FFN_THREADS, 1)
    few_ffn_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a,
                   int bytes) {
    using S = Shape<G, TT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + (-smem_addr(smem_raw) & 1023);
    Routing& r = *reinterpret_cast<Routing*>(ring + bytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + bytes + (sizeof(Routing) + 15) / 16 * 16);
    uint64_t* empty = full + MAX_STAGES;
    // a wait ran out; stages issued; shares of the part
    int32_t* flags = reinterpret_cast<int32_t*>(empty + MAX_STAGES);
    __shared__ Seg segs[2 + TOKEN_WARPS][MAX_SEGS];
    __shared__ float hf[MAX_SEGS][FT];
    const int tid = threadIdx.x, warp = tid >> 5;
    for (int e = tid; e < MAX_E; e += FFN_THREADS) r.tokens[e] = 0;
    if (tid < MAX_E / 32) r.hit[tid] = 0;
    if (tid == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            // the weights' announcement and the token warps' lanes
            mbar_init(&full[i], 1 + TOKEN_WARPS * 32);
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
    __syncthreads();
    pdl_wait();  // the router's logits (and planes)
    route_batch(a, r);
    const Geometry geo = geometry<S>(r.most, bytes);
    if (warp < CONSUMERS / 32) {
        consume<G, TT>(a, r, segs[0], ring, geo, full, empty, ring + geo.h,
                       reinterpret_cast<float*>(ring + geo.red), hf, flags);
    } else if (!(a.test_stall && blockIdx.x == 0)) {
        // (with the test hook nothing is brought in: the consumers' waits run out)
        Bringer c;
        c.ring = ring;
        c.full = full;
        c.empty = empty;
        c.limit = a.wait_limit_ns;
        c.geo = geo;
        c.p.stages = geo.stages;
        const int w = warp - CONSUMERS / 32;
        const bool ok = w == 0 ? bring_weights<G, TT>(a, r, maps, segs[1], c, &flags[1])
                               : bring_tokens<G, TT>(a, r, segs[1 + w], c, w - 1);
        if (!ok && (tid & 31) == 0) report_timeout(a.status);
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (blockIdx.x == gridDim.x - 1) publish_routing(a, r);
    __syncthreads();
    if (flags[0] && tid == 0) {
        // a wait ran out: see the copies in flight land before the block goes
        const int n = flags[1], m = geo.stages;
        for (int i = n > m ? n - m : 0; i < n; ++i)
            mbar_wait(&full[i % m], (uint32_t)(i / m) & 1, a.wait_limit_ns);
    }
}

// ---------------------------------------------------------------- combine

// out[t][c] = sum over the uses of token t (choices in order, then the shared
// expert) and their parts of the partial rows.  A block takes 32 columns of one
// token: 16 groups of 8 lanes share the rows, so that many of them are in flight at
// once (a token of a small batch has as many rows as there are parts).  128 threads
// of 32 registers and little shared memory find room beside the expert kernel's
// block, so that they are there when it ends (8 tokens over 160 experts, d = 5120, both
// in one run: the layer 336.7 us with blocks of 256 threads that do not, 324.5 with
// these; 16 tokens and 4 bits, d = 4096: 4 % less).
constexpr int CB_COLS = 32;
constexpr int CB_GROUPS = 16;

__global__ void __launch_bounds__(CB_GROUPS * 8, 16)
    few_combine_kernel(const int4* __restrict__ table, const float* __restrict__ part,
                       __nv_bfloat16* __restrict__ out, int d, int k, int uses) {
    __shared__ float4 sums[CB_GROUPS][9];
    __shared__ int4 use[MAX_K + 2];  // the last one ends the search for a row's use
    const int tid = threadIdx.x, col = tid & 7, grp = tid >> 3;
    const int t = blockIdx.y;
    part += blockIdx.x * CB_COLS + col * 4;
    pdl_wait();
    if (tid <= uses)
        use[tid] = tid < uses ? table[t * (k + 1) + tid] : make_int4(0, 0x7fffffff, 0, 0);
    __syncthreads();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    // this group's rows: its place `at` among those of use j; four loads at a time
    int at = grp, j = 0;
    do {
        float4 v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b, at += CB_GROUPS) {
            while (at >= use[j].y) at -= use[j++].y;
            v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < uses)
                v[b] = *reinterpret_cast<const float4*>(part +
                                                        (int64_t)(use[j].x + at * use[j].z) * d);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            s.x += v[b].x;
            s.y += v[b].y;
            s.z += v[b].z;
            s.w += v[b].w;
        }
    } while (j < uses);
    sums[grp][col] = s;
    __syncthreads();
    if (tid < CB_COLS) {
        const float* q = reinterpret_cast<const float*>(sums) + tid;
        float o = 0.f;
#pragma unroll
        for (int g = 0; g < CB_GROUPS; ++g) o += q[g * 36];
        const float hi = __shfl_down_sync(0xffffffffu, o, 1);
        if ((tid & 1) == 0)
            *reinterpret_cast<uint32_t*>(out + (int64_t)t * d + blockIdx.x * CB_COLS + tid) =
                pack_bf16x2(o, hi);
    }
}

// ---------------------------------------------------------------- router

// z[t][e] for 8 experts and up to TT tokens by a cluster of 8 blocks, each an
// eighth of d; the blocks' sums meet in the first one through its cluster's
// shared memory, in block order.  W_r is read once whatever T, and even E = 8
// spreads over 8 SMs, where one block per token took the latency of reading
// the whole of W_r in turn.  With 4-bit weights one more cluster turns x into
// planes (see the expert kernel).
constexpr int RC = 8;
constexpr int ROUTER_THREADS = 256;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t caddr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
    return v;
}

// Planes of this block's eighth of every token's row; xf[t] is what their sum is
// multiplied by.  Rows with an infinity or NaN get zeros and the factor NaN.
__device__ void split_planes(const FewArgs& a) {
    __shared__ uint32_t top[FT];  // bits of the largest magnitude: ordered as unsigned
    const int tid = threadIdx.x;
    const int d = a.d, vecs = d / RC / 8, v0 = blockIdx.y * vecs;  // 8 elements at a time
    const uint4* x = reinterpret_cast<const uint4*>(a.x);
    const int lane = tid & 31, warp = tid >> 5;
    for (int t = warp; t < a.T; t += ROUTER_THREADS / 32) {
        uint32_t m = 0;
#pragma unroll 4
        for (int c = lane; c < vecs; c += 32) {
            const uint4 v = x[(int64_t)t * (d / 8) + v0 + c];
            const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu,
                                   v.w & 0x7FFF7FFFu};
#pragma unroll
            for (int q = 0; q < 4; ++q) m = max(m, max(w[q] & 0xFFFFu, w[q] >> 16));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) top[t] = m;
    }
    cluster_sync_all();
    for (int t = warp; t < a.T; t += ROUTER_THREADS / 32) {
        uint32_t m = lane < RC ? ld_cluster_u32(map_shared_rank(smem_addr(&top[t]), lane)) : 0u;
        m = __reduce_max_sync(0xffffffffu, m);
        const bool odd = m >= 0x7F80u;
        const int e = odd ? 0 : plane_exponent(__uint_as_float(m << 16));
        const float2 by = plane_factors(e);
#pragma unroll 2
        for (int c = lane; c < vecs; c += 32) {
            const uint4 v = x[(int64_t)t * (d / 8) + v0 + c];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint64_t plane[PLANES] = {};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t bits = q & 1 ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16;
                int8_t p[PLANES];
                digits(odd ? 0.f : __uint_as_float(bits) * by.x * by.y, p);
#pragma unroll
                for (int i = 0; i < PLANES; ++i) plane[i] |= (uint64_t)(uint8_t)p[i] << (8 * q);
            }
#pragma unroll
            for (int i = 0; i < PLANES; ++i)
                *reinterpret_cast<uint64_t*>(a.xq + ((int64_t)t * PLANES + i) * d + (v0 + c) * 8) = plane[i];
        }
        if (lane == 0 && blockIdx.y == 0) a.xf[t] = odd ? NAN : plane_unit(e);
    }
    cluster_sync_all();  // the maxima are read before their blocks go
}

// VEC: rows of W_r are read 16 bytes at a time (E a multiple of 4).
template <int TT, bool VEC>
__global__ void __cluster_dims__(1, RC, 1) __launch_bounds__(ROUTER_THREADS)
    few_router_kernel(const __grid_constant__ FewArgs a, const float* __restrict__ Wr,
                      float* __restrict__ z) {
    constexpr int N = TT * 4;
    __shared__ float part[ROUTER_THREADS / 32][TT * 8];
    __shared__ float sum[TT * 8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int d = a.d, E = a.E, T = a.T;
    pdl_trigger();  // (the expert kernel reads no memory before its own wait)
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *a.status = DEV_OK;
    if ((int)blockIdx.x == (E + 7) / 8) {
        split_planes(a);
        return;
    }
    // two lanes share a row of W_r: four experts each
    const int len = d / RC, c0 = blockIdx.y * len, e0 = blockIdx.x * 8 + (tid & 1) * 4;
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll 4
    for (int c = c0 + tid / 2; c < c0 + len; c += ROUTER_THREADS / 2) {
        float w[4];
        if (VEC) {
            const float4 f = e0 < E ? *reinterpret_cast<const float4*>(Wr + (int64_t)c * E + e0)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            w[0] = f.x; w[1] = f.y; w[2] = f.z; w[3] = f.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = e0 + e < E ? Wr[(int64_t)c * E + e0 + e] : 0.f;
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float xv = t < T ? __bfloat162float(x[(int64_t)t * d + c]) : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[t * 4 + e] = fmaf(xv, w[e], v[t * 4 + e]);
        }
    }
    // sums over the lanes of one parity: each exchange halves the values a lane keeps
    int n = N, first = 0, same = 0;
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) {
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
            same |= o;
        }
    }
    constexpr int LEFT = N >= 16 ? N / 16 : 1;
    if ((lane & same) == 0) {
#pragma unroll
        for (int i = 0; i < LEFT; ++i) {
            const int q = first + i;  // token q / 4, expert q % 4 of this lane's four
            part[warp][q / 4 * 8 + (lane & 1) * 4 + q % 4] = v[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < TT * 8; i += ROUTER_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < ROUTER_THREADS / 32; ++w) s += part[w][i];
        sum[i] = s;
    }
    cluster_sync_all();
    if (cluster_ctarank() == 0)
        for (int i = tid; i < TT * 8; i += ROUTER_THREADS) {
            const uint32_t at = smem_addr(&sum[i]);
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < RC; ++q) s += __uint_as_float(ld_cluster_u32(map_shared_rank(at, q)));
            const int t = i / 8, e = blockIdx.x * 8 + i % 8;
            if (t < T && e < E) z[(int64_t)t * E + e] = s;
        }
    cluster_sync_all();  // the sums are read before their blocks go
}

template <int TT>
void router_launch(const FewArgs& a, const float* Wr, float* z, bool pdl, cudaStream_t st) {
    const dim3 grid((a.E + 7) / 8 + (a.G > 0), RC);
    launch_ex(pdl, a.E % 4 == 0 ? few_router_kernel<TT, true> : few_router_kernel<TT, false>, grid,
              dim3(ROUTER_THREADS), 0, st, a, Wr, z);
}

template <int G, int TT>
int launch_ffn(const FewMaps& m, const FewArgs& a, int smem_limit, bool pdl, cudaStream_t st) {
    // the kernel's few static bytes count too, and a block of the combine finds 4 KB
    const size_t limit = (size_t)smem_limit - 4096 - (2 + TOKEN_WARPS) * MAX_SEGS * sizeof(Seg) -
                         MAX_SEGS * FT * sizeof(float) - 256;
    // (1 KB to align the ring, the routing and the barriers behind the rest)
    const size_t fixed = 1024 + (sizeof(Routing) + 15) / 16 * 16 + 2 * MAX_STAGES * 8 + 16;
    const int bytes = (int)((limit - fixed) / 1024 * 1024);
    auto kern = few_ffn_kernel<G, TT>;
    // once a device (the limit is the device's own)
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return launch_result();
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit) !=
            cudaSuccess)
            return launch_result();
        allowed.fetch_or(bit, std::memory_order_release);
    }
    launch_ex(pdl, kern, dim3(FEW_CTAS), dim3(FFN_THREADS), fixed + bytes, st, m, a, bytes);
    note_launch();
    return launch_result();
}

template <int G>
int launch_ffn_tokens(const FewMaps& m, const FewArgs& a, int smem_limit, bool pdl,
                      cudaStream_t st) {
    if (G && a.T <= 2) return launch_ffn<G, G ? 2 : 8>(m, a, smem_limit, pdl, st);
    if (a.T <= 8) return launch_ffn<G, 8>(m, a, smem_limit, pdl, st);
    return launch_ffn<G, 16>(m, a, smem_limit, pdl, st);
}

}  // namespace

int64_t few_part_rows(int G, int T, int h, int E, int k, int hsum) {
    // A part is W / V long or one more, rounded down, so an item of weight w meets at
    // most w / (W / V) + 2 parts; n tokens then take n w / (W / V) + 2 n rows.  The sum
    // over the items of n w is at most T W, and at most (greatest cost / least cost)
    // times what equal costs would make it.  V follows from the most that A experts with
    // N assignments can weigh.
    const int least = few_cost(G, 1), most = few_cost(G, T);
    const int64_t gE = h / FEW_GRAN, gS = hsum / FEW_GRAN, N = (int64_t)T * k;
    int64_t rows = 0;
    for (int64_t A = k; A <= (E < N ? E : N); ++A) {
        const int64_t tot = A * gE + gS;
        const int64_t W = 8 * tot + (5 * (gE * (N - A) + gS * (T - 1)) + 1) / 2;
        const int64_t V = few_parts((int)W, least, 1, FEW_CTAS);
        const int64_t even = (N * gE + T * gS) * V / tot + 1;  // sum of n w V / W at equal costs
        const int64_t skewed = even * most / least + 1, all = T * V;
        // (rounding W / V down lengthens it by one part in W / V, which is at least 8)
        const int64_t need = (skewed < all ? skewed : all) * 9 / 8 + 2 * (N + T);
        rows = need > rows ? need : rows;
    }
    return rows;
}

int launch_few_router(const FewArgs& a, const float* Wr, float* z, bool pdl, cudaStream_t st) {
    if (a.T == 1) router_launch<1>(a, Wr, z, pdl, st);
    else if (a.T <= 4) router_launch<4>(a, Wr, z, pdl, st);
    else if (a.T <= 8) router_launch<8>(a, Wr, z, pdl, st);
    else router_launch<16>(a, Wr, z, pdl, st);
    note_launch();
    return launch_result();
}

int launch_few_ffn(const FewMaps& m, const FewArgs& a, int smem_limit, bool pdl,
                   cudaStream_t st) {
    switch (a.G) {
        case 0: return launch_ffn_tokens<0>(m, a, smem_limit, pdl, st);
        case 32: return launch_ffn_tokens<32>(m, a, smem_limit, pdl, st);
        case 64: return launch_ffn_tokens<64>(m, a, smem_limit, pdl, st);
        default: return launch_ffn_tokens<128>(m, a, smem_limit, pdl, st);
    }
}

int launch_few_combine(const FewArgs& a, bool pdl, cudaStream_t st) {
    launch_ex(pdl, few_combine_kernel, dim3(a.d / CB_COLS, a.T), dim3(CB_GROUPS * 8), 0, st,
              (const int4*)a.table, (const float*)a.part, reinterpret_cast<__nv_bfloat16*>(a.out), a.d,
              a.k, a.k + (a.hsum > 0));
    note_launch();
    return launch_result();
}

}  // namespace moe
