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
// One pass, bound by memory.  A warp takes 16 rows x 128 columns: lane (half,
// c) reads the eight weights 8c.. of row i (half 0) and row i + 8 (half 1) for i
// = 0..7, so that a row's 256 bytes are one access and eight are in flight.  The
// fragment order gathers a word from four lanes (two rows, two runs of eight
// columns); the lanes exchange their eight codes as one word each.
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

// Codes of eight weights, nibble e = q of element e in two's complement.  q = rint(w
// / s) without divisions or conversions: w inv + 1.5 2^23 leaves the nearest integer
// in the low bits, and w inv is within 2^-19 of the quotient (the fast reciprocal is
// off by 2 ulp).  As w and s have 8 significant bits and |w / s| <= 7.03 (so that
// nothing clips), the quotient is either n + 1/2 exactly or at least 2^-10 away from
// it; the exact remainder tells the half and sends it to the even code.
__device__ __forceinline__ uint32_t codes_of(const float* w, float s) {
    uint32_t out = 0;
    if (s >= 1.1754944e-38f && s <= 8.5070592e37f) {  // (the fast reciprocal's range)
        const float inv = __fdividef(1.f, s), half = 0.5f * s;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = fmaf(w[e], inv, 12582912.f);
            const float rest = fmaf(12582912.f - t, s, w[e]);
            uint32_t code = __float_as_uint(t);
            if (fabsf(rest) == half && (code & 1)) code += rest > 0.f ? 1 : -1;
            out |= (code & 15) << (4 * e);
        }
    } else {  // no scale, or one at the end of the range
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = s > 0.f ? rintf(w[e] / s) : 0.f;
            out |= (uint32_t)((int)fminf(fmaxf(q, -7.f), 7.f) & 15) << (4 * e);
        }
    }
    return out;
}

// Four nibbles (bits 0..15) to the low halves of four bytes, and back.
__device__ __forceinline__ uint32_t spread(uint32_t n) {
    n = (n | n << 8) & 0x00FF00FFu;
    return (n | n << 4) & 0x0F0F0F0Fu;
}
__device__ __forceinline__ uint32_t gather(uint32_t b) {
    b = (b | b >> 4) & 0x00FF00FFu;
    return (b | b >> 8) & 0xFFFFu;
}

// The lanes' codes (lane (half, c): row g + 8 half, columns 8c..) as fragment
// words: lane (t, s) = 8t + s gets the word of fragment lane 4g + t, 16-column
// step s.
__device__ __forceinline__ uint32_t to_fragment(uint32_t codes) {
    const int lane = threadIdx.x & 31, t = lane >> 3, s = lane & 7, c = 2 * s + (t >> 1);
    const uint32_t lo = __shfl_sync(0xffffffffu, codes, c) >> (16 * (t & 1));
    const uint32_t hi = __shfl_sync(0xffffffffu, codes, 16 + c) >> (16 * (t & 1));
    return spread(lo & 0xFFFFu) << 4 | spread(hi & 0xFFFFu);
}

// The other way: fragment words of lanes (t, s) to the eight codes of lane (half, c).
__device__ __forceinline__ uint32_t from_fragment(uint32_t w) {
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    const uint32_t a = __shfl_sync(0xffffffffu, w, 16 * (c & 1) + (c >> 1));
    const uint32_t b = __shfl_sync(0xffffffffu, w, 16 * (c & 1) + 8 + (c >> 1));
    const int shift = half ? 0 : 4;
    return gather(a >> shift & 0x0F0F0F0Fu) | gather(b >> shift & 0x0F0F0F0Fu) << 16;
}

// 16 rows x 128 columns of bf16 weights at W (ld elements a row; row i and row
// i + 8 begin at W + i ld and W + up + i ld) <-> codes and scales.  word(g):
// where lane (t, s) keeps the word of fragment lane 4g + t; scale(q, r): the
// scale of group q, row r.
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
            const float s = bf16_round(group_max<G>(m) / 7.f);
            if (c % (G / 8) == 0) *scale(c / (G / 8), g + 8 * half) = __float2bfloat16_rn(s);
            *word(g) = to_fragment(codes_of(w, s));
        }
    } else {
        uint32_t words[8];
        float s[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            words[g] = *word(g);
            s[g] = __bfloat162float(*scale(c / (G / 8), g + 8 * half));
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint32_t codes = from_fragment(words[g]);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)((int)(codes << (28 - 4 * e)) >> 28) * s[g];
            uint4 o;
            o.x = pack_bf16x2(v[0], v[1]);
            o.y = pack_bf16x2(v[2], v[3]);
            o.z = pack_bf16x2(v[4], v[5]);
            o.w = pack_bf16x2(v[6], v[7]);
            *reinterpret_cast<uint4*>(row + g * ld) = o;
        }
    }
}

// One warp per tile of 16 rows x 128 columns of W13.
template <int G, bool QUANT>
__global__ void __launch_bounds__(256)
    q13_kernel(__nv_bfloat16* W13, uint8_t* Q13, int64_t tiles, int hid, int d) {
    const int lane = threadIdx.x & 31, t = lane >> 3, s = lane & 7;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < tiles;
         i += warps) {
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
    }
}

// One warp per 16 rows x 128 hidden units of W2p.
template <int G, bool QUANT>
__global__ void __launch_bounds__(256)
    q2_kernel(__nv_bfloat16* W2p, uint32_t* Q2, __nv_bfloat16* scales, int64_t tiles, int hid) {
    const int lane = threadIdx.x & 31, t = lane >> 3, s = lane & 7;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < tiles;
         i += warps) {
        const int kb = (int)(i % (hid / 128));
        const int64_t row = i / (hid / 128) * 16, rb = row / 128;  // over all experts' d rows
        const int tile = (int)(row % 128) / 16;
        uint32_t* codes = Q2 + ((rb * (hid / 32) + kb * 4 + (s >> 1)) * 8 + tile) * 64 + (s & 1);
        __nv_bfloat16* sc = scales + (rb * (hid / G) + kb * (128 / G)) * 128 + tile * 16;
        block_pass<G, QUANT>(
            W2p + row * hid + kb * 128, hid, (int64_t)8 * hid,
            [&](int g) { return codes + (4 * g + t) * 2; },
            [&](int q, int r) { return sc + q * 128 + r; });
    }
}

template <int G, bool QUANT>
int launch_q4(const void* W13, const void* W2p, const void* Q13, const void* Q2, int n, int hid,
              int d, cudaStream_t st) {
    auto grid = [](int64_t tiles) { return (int)((tiles + 7) / 8 < 1184 ? (tiles + 7) / 8 : 1184); };
    uint8_t* q2 = reinterpret_cast<uint8_t*>(const_cast<void*>(Q2));
    const int64_t t13 = (int64_t)n * (hid / 8) * (d / 128);
    q13_kernel<G, QUANT><<<grid(t13), 256, 0, st>>>(
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W13)),
        reinterpret_cast<uint8_t*>(const_cast<void*>(Q13)), t13, hid, d);
    note_launch();
    if (launch_result() != 0) return -1;
    const int64_t t2 = (int64_t)n * (d / 16) * (hid / 128);
    q2_kernel<G, QUANT><<<grid(t2), 256, 0, st>>>(
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W2p)), reinterpret_cast<uint32_t*>(q2),
        reinterpret_cast<__nv_bfloat16*>(q2 + q2_code_bytes(n, hid, d)), t2, hid);
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
