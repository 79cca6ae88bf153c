// What the dense attention kernels share: the queries' scaling to fp16, the
// weights' scaling, the output rows, the tensor map of the codes.
#pragma once

#include <algorithm>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa2 {

constexpr int kDenseCtas = 148;  // CTAs (one per SM) that share a call's work at most
constexpr uint32_t kDenseWaitLimit = 1u << 22;  // polls of a wait for what is in flight (others: DenseArgs::wait_limit)
constexpr float kPBias = 7.f;   // weights are 2^(s - m + 7) (11 is 4 % slower in prefill: m rises more often) ...
constexpr float kPMax = 15.f;   // ... and at most 2^15: m follows a score that exceeds it by 8
constexpr float kScaleLog2e = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)

// Queries are bf16 of any magnitude, K is fp16.  A row (one head) is scaled by a
// power of two that puts its largest value into [2^14, 2^15): every value above
// 2^-28 of the largest is then exact in fp16, and what smaller ones lose is
// below 2^-39 of the largest (fp32 sums round coarser).
__device__ __forceinline__ float q_absmax(const uint4 (&r)[4]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = fmaxf(fmaxf(m, fabsf(bf16_lo(r[i].x))), fmaxf(fabsf(bf16_hi(r[i].x)), fabsf(bf16_lo(r[i].y))));
        m = fmaxf(fmaxf(m, fabsf(bf16_hi(r[i].y))), fmaxf(fabsf(bf16_lo(r[i].z)), fabsf(bf16_hi(r[i].z))));
        m = fmaxf(fmaxf(m, fabsf(bf16_lo(r[i].w))), fabsf(bf16_hi(r[i].w)));
    }
    return m;
}
// the factor f, and c = log2(e) / sqrt(128) / f
__device__ __forceinline__ void q_scale(float absmax, float& f, float& c) {
    int e = (int)(__float_as_uint(absmax) >> 23) - 127;  // absmax in [2^e, 2^(e+1))
    e = absmax == 0.f ? 14 : max(-112, e);
    f = __uint_as_float((uint32_t)(14 - e + 127) << 23);
    c = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * kScaleLog2e;
}
__device__ __forceinline__ uint32_t q_half2(uint32_t w, float f) { return f2_to_h2(bf16_lo(w) * f, bf16_hi(w) * f); }

// maximum over the four lanes of an aligned group
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// two E4M3 bytes (the low half of b2) -> f16x2, byte 0 in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t b2) {
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(b2));
    return d;
}

// fp32 results carry each weight as two fp16 terms, hi + lo * 2^-12, and multiply lo by V * 2^-12.
// V is a multiple of 2^-10, so V * 2^-12 is exact in fp16; a weight is at most 2^15 and
// leaves at most 2^3, so lo does not overflow.  The two terms hold 22 bits of every weight
// from 2^-14 on, which is 2^-20 of the largest or less (that one is held as 2^6 or more);
// smaller ones are rounded by up to 2^-37, 2^-43 of the largest.  (lo without the factor
// would round by 2^-31 of the largest: a million small weights could lose 2^-11 of the sum.)
constexpr float kLoScale = 4096.f;
__device__ __forceinline__ float h2_lo(uint32_t h) {
    __half_raw r;
    r.x = (unsigned short)h;
    return __half2float(__half(r));
}
__device__ __forceinline__ float h2_hi(uint32_t h) { return h2_lo(h >> 16); }
// lo of the pair (a, b) whose fp16 pair is `h`
__device__ __forceinline__ uint32_t rest_h2(float a, float b, uint32_t h) {
    return f2_to_h2((a - h2_lo(h)) * kLoScale, (b - h2_hi(h)) * kLoScale);
}

// 8 dims of output row (token * 16 + head): o / l, and the lse by the thread of dim 0
__device__ __forceinline__ void dense_store(const DenseArgs& a, int64_t row, int d8, const float (&o)[8], float m,
                                            float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.out_bf16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
            memcpy(&w[i], &v, 4);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * kD + d8) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float* p = static_cast<float*>(a.out) + row * kD + d8;
        *reinterpret_cast<float4*>(p) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        *reinterpret_cast<float4*>(p + 4) = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
    }
    if (d8 == 0) a.lse[row] = l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * 0.6931471805599453f;
}

// Tensor map of the code rows: boxes of min(page, 64) rows of 128 bytes, the
// box's innermost coordinate always 0.
constexpr int kDenseBoxShift = 6;
static bool dense_code_map(const csa2_kv_cache& cache, CUtensorMap* map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kCodeBytes, (cuuint64_t)(cache.n_phys_pages * cache.page_size)};
    const cuuint64_t strides[1] = {(cuuint64_t)kCodeBytes};
    const cuuint32_t box[2] = {(cuuint32_t)kCodeBytes, (cuuint32_t)std::min(1 << kDenseBoxShift, cache.page_size)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void*)cache.codes, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csa2
