// Rows of 16-bit (and 32-bit) values as the products, norms and checkpoints see
// them: their groups, conversions, activations and the checks of their layout.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "ep_device.cuh"

namespace ep {

// ---------------------------------------------------------------- groups

struct Groups {
    const int32_t *count, *offset;
    int R, per, rows;
};

// First row and number of rows of group g within its segment.
__device__ __forceinline__ void group_range(const Groups &gr, int g, int *first, int *n) {
    if (!gr.count) {
        *first = 0;
        *n = gr.rows;
        return;
    }
    const int o = gr.offset[g], c = gr.count[g];
    const bool none = o < 0 || o >= gr.rows || c <= 0;
    *first = none ? 0 : o;
    *n = none ? 0 : min(c, gr.rows - o);
}

// ----------------------------------------------------------- conversions

template <typename T> __device__ __forceinline__ float f32(T v);
template <> __device__ __forceinline__ float f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ __nv_bfloat16 rounded(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rounded(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float rounded(float v) { return v; }

// Two floats as two 16-bit values.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
// Two 16-bit values as two floats.
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t q);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t q) {
    return make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t q) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&q));
}
template <typename T> __device__ __forceinline__ void unpack8(float *v, const uint4 &r) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f32(e[i]);
}

// ----------------------------------------------------------- activations

// Within a few units of the last place of fp32 (more of 2^-24 |v|): far below
// the 16-bit rounding of every result it goes into.
__device__ __forceinline__ float sigmoidf(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// v sigmoid(v) of two values, with the same error.
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 t = mul2_rn(v, both(-1.4426950408889634f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = add2_rn(e, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    return mul2_rn(v, e);
}

// v Phi(v) of two values, Phi(v) = erfc(-v / sqrt(2)) / 2 by the rational approximation
// 7.1.26 of Abramowitz and Stegun (erf within 1.5e-7).
__device__ __forceinline__ float2 gelu2(float2 v) {
    const float2 x = make_float2(fabsf(v.x), fabsf(v.y));
    float2 t = fma2_rn(x, both(0.3275911f * 0.70710678118654752f), both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(t.y));
    float2 q = fma2_rn(t, both(1.061405429f), both(-1.453152027f));
    q = fma2_rn(q, t, both(1.421413741f));
    q = fma2_rn(q, t, both(-0.284496736f));
    q = fma2_rn(q, t, both(0.254829592f));
    const float2 a = mul2_rn(mul2_rn(v, v), both(-0.72134752044448170f));       // -v^2 / 2 in powers of two
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(a.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(a.y));
    q = mul2_rn(mul2_rn(q, mul2_rn(t, both(0.5f))), e);                         // Phi(-|v|)
    return mul2_rn(v, make_float2(v.x < 0.f ? q.x : 1.0f - q.x, v.y < 0.f ? q.y : 1.0f - q.y));
}

__device__ __forceinline__ void activate8(int act, float *v) {
    switch (act) {
    case EP_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i];     // NaN stays (fmaxf would drop it)
        break;
    case EP_ACT_GELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(v[i] * 0.70710678118654752f));
        break;
    case EP_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sigmoidf(v[i]);
        break;
    default: break;
    }
}

// grad * act'(v).  A closed unit of ReLU takes nothing, an infinite gradient included.
__device__ __forceinline__ float act_grad(int act, float grad, float v) {
    if (act == EP_ACT_RELU) return v > 0.f ? grad : 0.f;
    if (act == EP_ACT_GELU)      // Phi(v) + v phi(v), phi(v) = exp(-v^2/2) / sqrt(2 pi)
        return grad * (0.5f * (1.0f + erff(v * 0.70710678118654752f)) + v * expf(-0.5f * v * v) * 0.39894228040143268f);
    if (act == EP_ACT_SILU) {
        const float s = sigmoidf(v);
        return grad * (s * (1.0f + v * (1.0f - s)));
    }
    return grad;
}

// ------------------------------------------------------------- host side

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of `width` elements: 16-byte aligned, dense rows that do not overlap.
inline bool valid_rows(const ep_rows_t &r, int64_t width, bool many) {
    return r.ptr && aligned(r.ptr, 16) && r.row_stride >= width && r.row_stride % 8 == 0 &&
           (!many || (r.rank_stride > 0 && r.rank_stride % 8 == 0));
}

// 8-bit rows of `width` codes, 8-byte aligned, and their blocks' scales.
inline bool valid_codes(const ep_rows_t &codes, const ep_rows_t &scales, int64_t width, bool many) {
    return codes.ptr && aligned(codes.ptr, 8) && codes.row_stride >= width && codes.row_stride % 8 == 0 &&
           (!many || (codes.rank_stride > 0 && codes.rank_stride % 8 == 0)) && scales.ptr && aligned(scales.ptr, 4) &&
           scales.row_stride >= (width + 127) / 128 && (!many || scales.rank_stride > 0);
}

template <typename F> void with_type(int dtype, F f) {
    if (dtype == EP_DT_BF16) f(__nv_bfloat16());
    else f(__half());
}

inline ep_status_t launched() { return cudaGetLastError() == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP; }

constexpr int kMaxDevices = 64;

inline int sm_count(int dev) {
    static std::atomic<int> cached[kMaxDevices];
    int n = cached[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace ep
