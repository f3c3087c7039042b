// q4.cu -- packed expert weights to 4 bits with one bf16 scale per group, and
// back (layout: few.h).
//
// Per row and group of G weights along the reduction: a = max |w|,
// s = bf16(a / 7), q = w / s rounded to nearest even and clamped to [-7, 7]
// (0 where s is 0).  The scale is stored in bf16, half of what fp32 would add
// to the 4 bits at G = 32; q is taken against the rounded scale, so a largest
// weight is off by 2^-9 of itself at most.  Read back, q s is exact in fp32 (4
// bits times 8) and rounded once to bf16.
//
// One pass.  A warp takes 16 rows x 128 columns: lane (half, c) reads the eight
// weights 8c.. of row i (half 0) and row i + 8 (half 1) for i = 0..7, so that a row's
// 256 bytes are one access and eight are in flight.  The two halves exchange one word
// of codes for each, which leaves every lane a word in fragment order.  d = 4096, h =
// 14336, 8 experts, group 128 (3.5 GB): packed to 4 bits in 587-654 us by box and back in
// 537-555, 5.5-6.1 and 6.3-6.6 TB/s.  Reading back is bound by memory, packing by memory
// and instructions alike (issue slots 73 %, ALU 68 %, HBM 68 %).
// What counts is bytes in flight (each against 603 and 537 then): a tile a warp (a grid of 8
// blocks an SM that steps over the tiles took 693 and 623), eight rows' loads before the
// first is used (four: 691), and four blocks of 64 registers an SM rather than three of
// 74 (743).
#include "common.cuh"
#include "few.h"
#include "kernels.h"

namespace moe {

namespace {

// max |w| over the lanes of a group (G / 8 neighbours)
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// w / s rounded to nearest even, in the low bits of the result: two additions, no
// division or conversion.  w inv is within 2^-19 of the quotient (|w / s| <= 7.03, the
// fast reciprocal is off by 2 ulp), and the first addition leaves it on a grid of
// 2^-11: as w and s have 8 significant bits, the quotient is n + 1/2 exactly, which it
// stays, or at least 2^-9 away from it, on the same side after.  The second rounds to
// integers.
__device__ __forceinline__ uint32_t code_of(float w, float inv) {
    return __float_as_uint(fmaf(w, inv, 6144.f) + (12582912.f - 6144.f));
}

// The low bytes of four words as one.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of eight weights in the low nibbles of eight bytes: columns 0..3 in x.
__device__ __forceinline__ uint2 codes_of(const float* w, float s) {
    uint32_t q[8];
    if (s >= 1.1754944e-38f && s <= 8.5070592e37f) {  // (the fast reciprocal's range)
        const float inv = __fdividef(1.f, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = code_of(w[e], inv);
    } else {  // no scale, or one at the end of the range
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = (uint32_t)(int)(s > 0.f ? fminf(fmaxf(rintf(w[e] / s), -7.f), 7.f) : 0.f);
    }
    return make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
}

// A lane's codes (row g + 8 half, columns 8c..8c + 7) to a word in fragment order:
// lane (half, c) gets that of fragment lane 4g + 2 (c & 1) + half, 16-column step c >> 1.
__device__ __forceinline__ uint32_t to_fragment(uint2 codes, int half) {
    const uint32_t mine = half ? codes.y : codes.x;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, half ? codes.x : codes.y, 16);
    const uint32_t hi = half ? other : mine, lo = half ? mine : other;  // rows g, g + 8
    return (hi << 4 & 0xF0F0F0F0u) | (lo & 0x0F0F0F0Fu);
}

// The other way; the nibbles' bytes come without their sign.
__device__ __forceinline__ uint2 from_fragment(uint32_t w, int half) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 16);
    const int shift = half ? 0 : 4;
    const uint32_t mine = w >> shift & 0x0F0F0F0Fu, its = other >> shift & 0x0F0F0F0Fu;
    return half ? make_uint2(its, mine) : make_uint2(mine, its);
}

// Codes of two neighbouring columns (bytes 2i, 2i + 1 of n) times s, in bf16: 128 + (q +
// 8) as it lies, less 136, is q, and the product is rounded once.
__device__ __forceinline__ uint32_t value_pair(uint32_t n, int i, __nv_bfloat162 s) {
    const uint32_t b = __byte_perm(n ^ 0x08080808u, 0x43434343u, i ? 0x4342 : 0x4140);
    __nv_bfloat162 v;
    memcpy(&v, &b, 4);
    v = __hmul2(__hsub2(v, __float2bfloat162_rn(136.f)), s);
    uint32_t o;
    memcpy(&o, &v, 4);
    return o;
}

// 16 rows x 128 columns of bf16 weights at W (ld elements a row; row i and row
// i + 8 begin at W + i ld and W + up + i ld) <-> codes and scales.  word(g): where
// this lane keeps its word of rows g, g + 8; scale(q, r): the scale of group q, row r.
template <int G, bool QUANT, typename Word, typename Scale>
__device__ __forceinline__ void block_pass(__nv_bfloat16* W, int64_t ld, int64_t up, Word word,
                                           Scale scale) {
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    __nv_bfloat16* row = W + (half ? up : 0) + c * 8;
    if (QUANT) {
        uint4 raw[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) raw[g] = __ldcs(reinterpret_cast<const uint4*>(row + g * ld));
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint32_t u[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
            float w[8], m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = __uint_as_float(e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
                m = fmaxf(m, fabsf(w[e]));
            }
            // (m / 7 is never within 2^-12 of itself of a midpoint of bf16, so the
            // product by the rounded 1 / 7 rounds to the same value)
            const float s = bf16_round(group_max<G>(m) * (1.f / 7.f));
            if (c % (G / 8) == 0) *scale(c / (G / 8), g + 8 * half) = __float2bfloat16_rn(s);
            *word(g) = to_fragment(codes_of(w, s), half);
        }
    } else {
        uint32_t words[8];
        __nv_bfloat16 s[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            words[g] = *word(g);
            s[g] = *scale(c / (G / 8), g + 8 * half);
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint2 n = from_fragment(words[g], half);
            const __nv_bfloat162 ss = __bfloat162bfloat162(s[g]);
            *reinterpret_cast<uint4*>(row + g * ld) =
                make_uint4(value_pair(n.x, 0, ss), value_pair(n.x, 1, ss), value_pair(n.y, 0, ss),
                           value_pair(n.y, 1, ss));
        }
    }
}

// A set: one warp per 16 rows x 128 columns, first those of W13 (t13 tiles), then of W2p
// (t2).
template <int G, bool QUANT>
__global__ void __launch_bounds__(256, QUANT ? 4 : 5)
    q4_kernel(__nv_bfloat16* W13, uint8_t* Q13, int64_t t13, __nv_bfloat16* W2p, uint32_t* Q2,
              __nv_bfloat16* scales2, int64_t t2, int hid, int d) {
    const int lane = threadIdx.x & 31, c = lane & 15, t = 2 * (c & 1) + (lane >> 4), s = c >> 1;
    int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i < t13) {
        const int64_t b = i >> 2;   // block of 32 hidden units x 128 columns
        const int tile = (int)(i & 3);
        const int kb = (int)(b % (d / 128));
        const int64_t unit = b / (d / 128) * 32 + tile * 8;  // over all experts: e * hid + j
        const int64_t gate = 256 * (unit / 128) + unit % 128;
        uint8_t* blk = Q13 + b * q13_block_bytes(G);
        uint32_t* codes = reinterpret_cast<uint32_t*>(blk) + tile * 256 + (s >> 2) * 128 + (s & 3);
        __nv_bfloat16* sc = reinterpret_cast<__nv_bfloat16*>(blk + 4096) + tile * 16;
        block_pass<G, QUANT>(
            W13 + gate * d + kb * 128, d, (int64_t)128 * d,
            [&](int g) { return codes + (4 * g + t) * 4; },
            [&](int q, int r) { return sc + q * 64 + r; });
    } else if ((i -= t13) < t2) {
        const int kb = (int)(i % (hid / 128));
        const int64_t row = i / (hid / 128) * 16, rb = row / 128;  // over all experts' d rows
        const int tile = (int)(row % 128) / 16;
        uint32_t* codes = Q2 + ((rb * (hid / 32) + kb * 4 + (s >> 1)) * 8 + tile) * 64 + (s & 1);
        __nv_bfloat16* sc = scales2 + (rb * (hid / G) + kb * (128 / G)) * 128 + tile * 16;
        block_pass<G, QUANT>(
            W2p + row * hid + kb * 128, hid, (int64_t)8 * hid,
            [&](int g) { return codes + (4 * g + t) * 2; },
            [&](int q, int r) { return sc + q * 128 + r; });
    }
}

template <int G, bool QUANT>
int launch_q4(const void* W13, const void* W2p, const void* Q13, const void* Q2, int n, int hid,
              int d, cudaStream_t st) {
    uint8_t* q2 = reinterpret_cast<uint8_t*>(const_cast<void*>(Q2));
    const int64_t t13 = (int64_t)n * (hid / 8) * (d / 128), t2 = (int64_t)n * (d / 16) * (hid / 128);
    q4_kernel<G, QUANT><<<(unsigned)((t13 + t2 + 7) / 8), 256, 0, st>>>(
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W13)),
        reinterpret_cast<uint8_t*>(const_cast<void*>(Q13)), t13,
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W2p)), reinterpret_cast<uint32_t*>(q2),
        reinterpret_cast<__nv_bfloat16*>(q2 + q2_code_bytes(n, hid, d)), t2, hid, d);
    note_launch();
    return launch_result();
}

}  // namespace

int launch_q4_quantize(const void* W13, const void* W2p, void* Q13, void* Q2, int n, int hid,
                       int d, int G, cudaStream_t st) {
    return G == 32   ? launch_q4<32, true>(W13, W2p, Q13, Q2, n, hid, d, st)
           : G == 64 ? launch_q4<64, true>(W13, W2p, Q13, Q2, n, hid, d, st)
                     : launch_q4<128, true>(W13, W2p, Q13, Q2, n, hid, d, st);
}

int launch_q4_dequantize(const void* Q13, const void* Q2, void* W13, void* W2p, int n, int hid,
                         int d, int G, cudaStream_t st) {
    return G == 32   ? launch_q4<32, false>(W13, W2p, Q13, Q2, n, hid, d, st)
           : G == 64 ? launch_q4<64, false>(W13, W2p, Q13, Q2, n, hid, d, st)
                     : launch_q4<128, false>(W13, W2p, Q13, Q2, n, hid, d, st);
}

}  // namespace moe
