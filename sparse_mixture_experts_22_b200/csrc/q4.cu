// q4.cu -- packed expert weights to 4 bits with one bf16 scale per group, and
// back (layout: few.h).
//
// Per row and group of G weights along the reduction: a = max |w|,
// s = bf16(a / 7), q = w / s rounded to nearest even and clamped to [-7, 7]
// (0 where s is 0).  The scale is stored in bf16, half of what fp32 would add
// to the 4 bits at G = 32; q is taken against the rounded scale, so that the
// rounding costs nothing but a largest weight that may clip by 2^-9.  Read
// back, q s is exact in fp32 (4 bits times 8) and rounded once to bf16.
#include "common.cuh"
#include "few.h"
#include "kernels.h"

namespace moe {

namespace {

// Row of the packed matrix that row r of a 16-row block holds: gate rows of
// hidden units 8a.. (r < 8), their up rows, or plainly row base + r.
__device__ __forceinline__ int64_t w13_row(int64_t e, int hid, int a, int r) {
    const int j = a * 8 + r % 8;
    return e * 2 * hid + 256 * (j / 128) + 128 * (r / 8) + j % 128;
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ uint32_t code_of(float w, float s) {
    const float q = s > 0.f ? rintf(w / s) : 0.f;
    return (uint32_t)((int)fminf(fmaxf(q, -7.f), 7.f) + 8);
}

// A lane's fragment of 16 rows x 16 STEPS columns: v[s][2 reg + element].
// lo / hi: rows g and g + 8 of the block at its first column.
template <int STEPS>
__device__ __forceinline__ void load_frag(const __nv_bfloat16* lo, const __nv_bfloat16* hi,
                                          float (*v)[8]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int reg = 0; reg < 4; ++reg) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                (reg & 1 ? hi : lo) + 16 * s + 8 * (reg >> 1) + 2 * t);
            v[s][2 * reg] = __uint_as_float(w << 16);
            v[s][2 * reg + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
}

template <int STEPS>
__device__ __forceinline__ void store_frag(__nv_bfloat16* lo, __nv_bfloat16* hi, float (*v)[8]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int reg = 0; reg < 4; ++reg)
            *reinterpret_cast<uint32_t*>((reg & 1 ? hi : lo) + 16 * s + 8 * (reg >> 1) + 2 * t) =
                pack_bf16x2(v[s][2 * reg], v[s][2 * reg + 1]);
}

// max |w| of a lane's elements of row g (half 0) or g + 8 in step s
__device__ __forceinline__ float step_max(const float* v, int half) {
    return fmaxf(fmaxf(fabsf(v[2 * half]), fabsf(v[2 * half + 1])),
                 fmaxf(fabsf(v[2 * half + 4]), fabsf(v[2 * half + 5])));
}

// Codes of one step; sl, sh: the scales of rows g and g + 8.
__device__ __forceinline__ uint32_t pack_step(const float* v, float sl, float sh) {
    uint32_t w = 0;
#pragma unroll
    for (int reg = 0; reg < 4; ++reg) {
        const float s = reg & 1 ? sh : sl;
        w |= code_of(v[2 * reg], s) << (4 * reg);
        w |= code_of(v[2 * reg + 1], s) << (4 * reg + 16);
    }
    return w;
}

__device__ __forceinline__ void unpack_step(uint32_t w, float sl, float sh, float* v) {
#pragma unroll
    for (int reg = 0; reg < 4; ++reg) {
        const float s = reg & 1 ? sh : sl;
        v[2 * reg] = (float)((int)((w >> (4 * reg)) & 15u) - 8) * s;
        v[2 * reg + 1] = (float)((int)((w >> (4 * reg + 16)) & 15u) - 8) * s;
    }
}

__device__ __forceinline__ float scale_of(float amax) { return bf16_round(amax / 7.f); }

// One warp per 16 x 128 block of W13.
template <int G, bool QUANT>
__global__ void __launch_bounds__(256)
    q13_kernel(__nv_bfloat16* W13, uint32_t* codes, __nv_bfloat16* scales, int64_t blocks, int hid,
               int d) {
    constexpr int SG = G / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t b = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b < blocks;
         b += warps) {
        const int kb = (int)(b % (d / 128));
        const int64_t ea = b / (d / 128);
        const int a = (int)(ea % (hid / 8));
        const int64_t e = ea / (hid / 8);
        __nv_bfloat16* lo = W13 + w13_row(e, hid, a, g) * d + kb * 128;
        __nv_bfloat16* hi = W13 + w13_row(e, hid, a, g + 8) * d + kb * 128;
        uint32_t* cw = codes + b * 256 + lane * 4;
        __nv_bfloat16* sc = scales + b * (128 / G) * 16;
        float v[8][8];
        if (QUANT) {
            load_frag<8>(lo, hi, v);
#pragma unroll
            for (int q = 0; q < 128 / G; ++q) {
                float ml = 0.f, mh = 0.f;
#pragma unroll
                for (int s = 0; s < SG; ++s) {
                    ml = fmaxf(ml, step_max(v[q * SG + s], 0));
                    mh = fmaxf(mh, step_max(v[q * SG + s], 1));
                }
                const float sl = scale_of(quad_max(ml)), sh = scale_of(quad_max(mh));
                if ((lane & 3) == 0) {
                    sc[q * 16 + g] = __float2bfloat16_rn(sl);
                    sc[q * 16 + 8 + g] = __float2bfloat16_rn(sh);
                }
#pragma unroll
                for (int s = 0; s < SG; ++s) {
                    const int st = q * SG + s;
                    cw[(st / 4) * 128 + st % 4] = pack_step(v[st], sl, sh);
                }
            }
        } else {
#pragma unroll
            for (int st = 0; st < 8; ++st) {
                const int q = st / SG;
                unpack_step(cw[(st / 4) * 128 + st % 4], __bfloat162float(sc[q * 16 + g]),
                            __bfloat162float(sc[q * 16 + 8 + g]), v[st]);
            }
            store_frag<8>(lo, hi, v);
        }
    }
}

// One warp per 16 rows x 128 hidden units of W2p.
template <int G, bool QUANT>
__global__ void __launch_bounds__(256)
    q2_kernel(__nv_bfloat16* W2p, uint32_t* codes, __nv_bfloat16* scales, int64_t blocks, int hid,
              int d) {
    constexpr int SG = G / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t b = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b < blocks;
         b += warps) {
        const int kb = (int)(b % (hid / 128));         // 128 hidden units
        const int64_t tile = b / (hid / 128);          // 16 rows of all experts' d
        const int64_t rb = tile / 8;
        const int ti = (int)(tile % 8);
        __nv_bfloat16* lo = W2p + (tile * 16 + g) * hid + kb * 128;
        __nv_bfloat16* hi = lo + (int64_t)8 * hid;
        uint32_t* cw = codes + ((rb * (hid / 32) + kb * 4) * 8 + ti) * 64 + lane * 2;
        __nv_bfloat16* sc = scales + (rb * (hid / G) + kb * (128 / G)) * 128 + ti * 16;
        float v[8][8];
        if (QUANT) {
            load_frag<8>(lo, hi, v);
#pragma unroll
            for (int q = 0; q < 128 / G; ++q) {
                float ml = 0.f, mh = 0.f;
#pragma unroll
                for (int s = 0; s < SG; ++s) {
                    ml = fmaxf(ml, step_max(v[q * SG + s], 0));
                    mh = fmaxf(mh, step_max(v[q * SG + s], 1));
                }
                const float sl = scale_of(quad_max(ml)), sh = scale_of(quad_max(mh));
                if ((lane & 3) == 0) {
                    sc[q * 128 + g] = __float2bfloat16_rn(sl);
                    sc[q * 128 + 8 + g] = __float2bfloat16_rn(sh);
                }
#pragma unroll
                for (int s = 0; s < SG; ++s) {
                    const int st = q * SG + s;
                    cw[(st / 2) * 512 + st % 2] = pack_step(v[st], sl, sh);
                }
            }
        } else {
#pragma unroll
            for (int st = 0; st < 8; ++st) {
                const int q = st / SG;
                unpack_step(cw[(st / 2) * 512 + st % 2], __bfloat162float(sc[q * 128 + g]),
                            __bfloat162float(sc[q * 128 + 8 + g]), v[st]);
            }
            store_frag<8>(lo, hi, v);
        }
    }
}

template <int G, bool QUANT>
int launch_q4(const void* W13, const void* W2p, const void* Q13, const void* Q2, int n, int hid,
              int d, cudaStream_t st) {
    const int64_t blocks = (int64_t)n * (hid / 8) * (d / 128);
    const int grid = (int)((blocks + 7) / 8 < 16384 ? (blocks + 7) / 8 : 16384);
    uint8_t* q13 = reinterpret_cast<uint8_t*>(const_cast<void*>(Q13));
    uint8_t* q2 = reinterpret_cast<uint8_t*>(const_cast<void*>(Q2));
    q13_kernel<G, QUANT><<<grid, 256, 0, st>>>(
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W13)), reinterpret_cast<uint32_t*>(q13),
        reinterpret_cast<__nv_bfloat16*>(q13 + q13_code_bytes(n, hid, d)), blocks, hid, d);
    note_launch();
    if (launch_result() != 0) return -1;
    const int64_t blocks2 = (int64_t)n * (d / 16) * (hid / 128);
    const int grid2 = (int)((blocks2 + 7) / 8 < 16384 ? (blocks2 + 7) / 8 : 16384);
    q2_kernel<G, QUANT><<<grid2, 256, 0, st>>>(
        reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(W2p)), reinterpret_cast<uint32_t*>(q2),
        reinterpret_cast<__nv_bfloat16*>(q2 + q2_code_bytes(n, hid, d)), blocks2, hid, d);
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
