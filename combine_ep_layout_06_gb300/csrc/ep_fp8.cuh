// Block-scaled E4M3: a block of 128 values has the scale fl32(max|x| / 448) and
// the codes of fl32(x / scale), rounded to nearest even and saturated.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ep_device.cuh"

#ifndef EP_FP8_RECIP_QUOT
#define EP_FP8_RECIP_QUOT 1            // FP8: quotients by reciprocal + one FMA correction
#endif

namespace ep {

// 4 values -> 4 E4M3 codes (byte i = element i) given the block scale.
__device__ __forceinline__ uint32_t quant4(const float *f, float scale) {
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = f[2 * i] / scale;
        const float b = f[2 * i + 1] / scale;
        const __nv_fp8x2_storage_t q =
            __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        packed |= (uint32_t)q << (16 * i);
    }
    return packed;
}

// fl32(x / scale) from r = RN(1 / scale) and one FMA correction of the
// product (Markstein's division step: P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990).  For scale >= 2^-90 the residual x - q0*scale is exact
// for every quotient large enough to give a nonzero code, and the E4M3 code
// of the result equals that of the IEEE quotient for every bf16 x under every
// bf16 block maximum (fp8_quotient_check_kernel in ep_dispatch.cu compares the codes over
// all 1.07e9 pairs; ep_test_fp8_quotient_check runs it); smaller scales
// divide.  The
// residual is formed negated, q0*scale - x (the same magnitude: RN is
// symmetric), and applied with -r, so that for x = +-0 the sums of zeros
// keep the sign of x (the code of -0 is 0x80) with no sign fix-up.
__device__ __forceinline__ float quot_recip(float x, float scale, float r) {
    const float q0 = __fmul_rn(x, r);
    const float nres = __fmaf_rn(q0, scale, -x);
    return __fmaf_rn(nres, -r, q0);
}

// fl32(a / 448) for a block maximum a > 0 (a bf16 magnitude): the product
// with RN(1/448) and the same one-FMA correction.  Equal to the IEEE
// quotient for every finite non-negative bf16 a (proved on the host in exact
// rational arithmetic, and compared on the device for every positive finite
// a by fp8_quotient_check_kernel), and for other a that are far from underflow by
// the theorem of the paper above (1/448 is rounded correctly, the first product is
// within a unit of the quotient); a = inf gives inf.
__device__ __forceinline__ float block_scale(float a) {
#if EP_FP8_RECIP_QUOT
    constexpr float kInv448 = 0x1.24924ap-9f;   // RN(1/448)
    const float q0 = __fmul_rn(a, kInv448);
    const float e = __fmaf_rn(-q0, 448.0f, a);
    const float q = __fmaf_rn(e, kInv448, q0);
    return a <= 0x1.fffffep127f ? q : a;
#else
    return a / 448.0f;
#endif
}

__device__ __forceinline__ uint32_t quant4_recip(const float *f, float scale, float r) {
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = quot_recip(f[2 * i], scale, r);
        const float b = quot_recip(f[2 * i + 1], scale, r);
        const __nv_fp8x2_storage_t q =
            __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        packed |= (uint32_t)q << (16 * i);
    }
    return packed;
}

// 4 values, as two pairs: quot_recip's steps two at a time, on the negated
// quotient: with q = -x r the residual x + q scale and the correction q - res r
// need no value's negative, and zeros keep their sign (x = -0: q = +0, res = +0,
// q - 0 = +0).  The codes' signs are turned at the end.
__device__ __forceinline__ uint32_t quant4_recip(const float2 *f, float scale, float minus_r) {
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 q0 = mul2_rn(f[i], both(minus_r));
        const float2 res = fma2_rn(q0, both(scale), f[i]);
        const __nv_fp8x2_storage_t q =
            __nv_cvt_float2_to_fp8x2(fma2_rn(res, both(minus_r), q0), __NV_SATFINITE, __NV_E4M3);
        packed |= (uint32_t)q << (16 * i);
    }
    return packed ^ 0x80808080u;
}
// The largest magnitude; NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// A lane's N times 8 values of a block whose largest magnitude is a: their codes (byte i =
// value i); returns the block's scale.  A block with a NaN or an infinity is NaN as a
// whole.
template <int N> __device__ __forceinline__ float scaled_codes(const float2 *f, float a, uint2 *q) {
    if (a >= 0x1p-80f && a <= 0x1.fffffep127f) { // so that the scale is past 2^-90
        const float s = block_scale(a), r = -__frcp_rn(s);
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = make_uint2(quant4_recip(f + 4 * i, s, r), quant4_recip(f + 4 * i + 2, s, r));
        return s;
    }
    if (!(a <= 0x1.fffffep127f)) {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        return __uint_as_float(0x7fffffffu);
    }
    const float s = __fdiv_rn(a, 448.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 *g = f + 4 * i;
        const float v[8] = {g[0].x, g[0].y, g[1].x, g[1].y, g[2].x, g[2].y, g[3].x, g[3].y};
        q[i] = s == 0.f ? make_uint2(0u, 0u) : make_uint2(quant4(v, s), quant4(v + 4, s));
    }
    return s;
}
// A block of 128 values over 16 neighbouring lanes, 4 pairs a lane.  By whole warps.
__device__ __forceinline__ uint2 block_codes(const float2 *f, float *scale) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max_nan(a, f[i].x, f[i].y);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o), 0.f);
    uint2 q;
    *scale = scaled_codes<1>(f, a, &q);
    return q;
}
// 8 codes -> 8 values, code * scale.
__device__ __forceinline__ void block_values(float2 *v, const uint2 &q, float scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        v[i] = mul2_rn(__half22float2(__half2(h)), both(scale));
    }
}
__device__ __forceinline__ void block_values(float *v, const uint2 &q, float scale) {
    float2 f[4];
    block_values(f, q, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = f[i].x;
        v[2 * i + 1] = f[i].y;
    }
}

}  // namespace ep
