// few.h -- host interface of the few-token layer (few.cu) and of the 4-bit
// expert weights (q4.cu): parameters, layouts and launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int FEW_MAX_T = 16;       // tokens of one call
constexpr int FEW_CTAS = 148;       // CTAs of the expert kernel (one per SM)
constexpr int FEW_MAX_ITEMS = FEW_MAX_T * 8 + 1;  // experts one batch can hit, and the shared one
constexpr int FEW_GRAN = 32;        // hidden units per granule, the unit the CTAs share work in
constexpr int FEW_HCAP = 512;       // hidden units a part holds in shared memory at most
constexpr int FEW_PLANES = 4;       // 8-bit digits of an element of x or H beside 4-bit weights

// ---------------------------------------------------------------- 4-bit layout
//
// A set is n experts (the routed ones, or the fused shared one) of hidden width
// hid and model width d; weights are codes q in [-7, 7] in two's complement and
// one bf16 scale per group of G along the reduction.  Codes sit in the order in
// which a warp's lanes take them as A fragments of the 8-bit products (m16 x
// k32, lane 4g + t): one 32-bit word holds a lane's eight codes of 16 columns, in
// byte i the code of row g (high nibble) and of row g + 8 (low nibble) at column
// 4t + i.  A nibble in the high half of a byte is 16 q as it lies.
//
// Q13: blocks [n][hid/32][d/128] of 64 rows x 128 of d: four tiles of 16 rows
//      (tile i the gate rows of hidden units 8i..8i+7 of the 32, then their up
//      rows), each [2][32 lanes][4 words] with 16-column step = 4 * half + word;
//      then the scales [128/G][64 rows] bf16.  The columns of one granule follow
//      one another, so a stage of any depth is one copy.
// Q2:  codes [n][d/128][hid/32][8 row tiles][32 lanes][2 words]: 128 rows of d x
//      32 hidden units, tile i its rows 16i..16i+15, word = 16-column step; then
//      the scales [n][d/128][hid/G][128 rows] bf16.
__host__ __device__ constexpr int q13_block_bytes(int G) { return 4096 + 128 * (128 / G); }
__host__ __device__ inline size_t q13_bytes(int64_t n, int hid, int d, int G) {
    return (size_t)n * (hid / 32) * (d / 128) * q13_block_bytes(G);
}
__host__ __device__ inline size_t q2_code_bytes(int64_t n, int hid, int d) {
    return (size_t)n * (d / 128) * (hid / 32) * 2048;
}
__host__ __device__ inline size_t q2_bytes(int64_t n, int hid, int d, int G) {
    return (size_t)n * (d / 128) * ((size_t)(hid / 32) * 2048 + (size_t)(hid / G) * 256);
}

int launch_q4_quantize(const void* W13, const void* W2p, void* Q13, void* Q2, int n, int hid,
                       int d, int G, cudaStream_t st);
int launch_q4_dequantize(const void* Q13, const void* Q2, void* W13, void* W2p, int n, int hid,
                         int d, int G, cudaStream_t st);

// ---------------------------------------------------------------- the layer

// What a granule costs an SM when its expert serves n tokens, in eighths of what it
// costs at one or two: where products take longer than HBM, a part holds fewer
// granules.  With n tokens for every expert (d = 4096, h = 14336) a granule and SM takes,
// in us, bf16 16.7-17.0 (n <= 2), 17.1-18.0 (4), 18.6-18.9 (8), 23.1 (16) and 4 bits
// 5.9-6.9, 7.3-9.7, 13.9-19.1, 35.6-39.5; the costs lie below these ratios, because
// experts with few tokens find more of HBM's rate free beside the others.  4 bits, mean
// of 16 batches in us, with these, with 8 9 12 14 19 24 and with 8 10 13 18 23 28: 8
// tokens over 160 experts and shared ones 147, 160, 151; 16 tokens over 8 experts 243,
// 242, 243; under a skewed router 255, 247, 262; 16 tokens over 32 experts and shared
// ones 153, 155, 156.  At most 8 + 5/2 (n - 1), which few_part_rows counts on.
__host__ __device__ inline int few_cost(int G, int n) {
    if (G == 0) return n <= 8 ? 8 : 10;
    return n <= 2 ? 8 : n <= 4 ? 10 : n <= 6 ? 13 : n <= 8 ? 15 : n <= 12 ? 21 : 26;
}

// Parts the experts' hidden units are cut into: W weighted granules in item order
// (hit experts ascending, then the shared one) over V parts of W / V or one more;
// every CTA of the grid takes the same number of parts within one, none holds more
// than FEW_HCAP hidden units (one granule less, as one may begin at the very end), and
// none is shorter than the costliest granule.
__host__ __device__ inline int few_parts(int W, int lightest, int heaviest, int ctas) {
    const int per = ctas * (FEW_HCAP / FEW_GRAN - 1) * lightest;
    const int V = ctas * ((W + per - 1) / per), most = W / heaviest;
    return V < most ? V : most;
}

struct FewArgs {
    const void* x;              // [T][d] bf16
    int8_t* xq;                 // 4 bits: [T][FEW_PLANES][d] planes of x, and
    float* xf;                  // [T] what they are multiplied by (few_router writes both)
    const float* logits;        // [T][E] router logits without bias
    const float* bias;          // [E] or null
    // routed and shared weights: packed bf16, or codes (scales follow them)
    const void* w13;
    const void* w2;
    const void* w13s;
    const void* w2s;
    int G;                      // 0: bf16, else the group of the 4-bit scales
    int T, d, h, E, k, hsum;
    int64_t C;                  // capacity
    int32_t* topk_idx;          // [T][k]
    float* topk_gate;           // [T][k]
    int32_t* routed;            // [E]
    int32_t* kept;              // [E]
    int4* table;                // [T][k + 1]: first partial row, rows, row stride of each use
    float* part;                // [rows][d] partial outputs
    void* out;                  // [T][d] bf16
    int32_t* status;
    uint64_t wait_limit_ns;
    int test_stall;             // test hook: block 0 brings nothing in
};

// Upper bound on the rows of FewArgs::part for any routing of the batch.
int64_t few_part_rows(int G, int T, int h, int E, int k, int hsum);
// Logits z [T][E] = x Wr; clears the status word; with 4-bit weights (a.G) also
// splits x into its planes.
int launch_few_router(const FewArgs& a, const float* Wr, float* z, bool pdl, cudaStream_t st);
// Tensor maps of the bf16 weights (unused with 4 bits): W13 as [blocks of 128
// rows][128][d] in boxes of 64 columns x 32 rows x 2 blocks (a granule's gate
// and up rows) with the 128-byte swizzle, W2p as rows of the hidden width in
// boxes of 32 columns x 128 rows with the 64-byte swizzle; s: the shared set's.
struct FewMaps {
    CUtensorMap w13, w2, w13s, w2s;
};
int launch_few_ffn(const FewMaps& m, const FewArgs& a, int smem_limit, bool pdl, cudaStream_t st);
int launch_few_combine(const FewArgs& a, bool pdl, cudaStream_t st);

}  // namespace moe
