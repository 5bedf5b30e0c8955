// The experts of a few tokens: both products and the weighted sum, in two
// kernels.
#include "ep_rows.cuh"

namespace ep {
namespace {

struct FewParams {
    int T, E, k, H, F, wide, act;
    ep_rows_t up, down, x, residual, out;
    const void *up_bias, *down_bias;
    const float *w;
    const int32_t *idx;
    float *h;                        // [T * k][F]
    uint32_t *error;
};

template <typename T> __device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b) {
    float x[8], y[8], s = 0.f;
    unpack8<T>(x, a);
    unpack8<T>(y, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * y[i];
    return s;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A warp for each choice and feature.
template <typename T> __global__ void __launch_bounds__(256) few_up_kernel(const FewParams p) {
    const int lane = threadIdx.x & 31, f = blockIdx.x * 8 + (threadIdx.x >> 5), pair = blockIdx.y;
    if (f >= p.F) return;
    const int e = p.idx[pair];
    if (e < 0 || e >= p.E) {
        if (e >= p.E && f == 0 && lane == 0 && p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
        return;
    }
    const T *x = static_cast<const T *>(p.x.ptr) + (pair / p.k) * p.x.row_stride;
    const T *w = static_cast<const T *>(p.up.ptr) + e * p.up.rank_stride;
    const bool gated = p.act == EP_ACT_SWIGLU;
    float v[2] = {};
    for (int g = 0; g < (gated ? 2 : 1); ++g) {
        const int64_t row = f + (int64_t)g * p.F;
        for (int c = lane * 8; c < p.H; c += 256)
            v[g] += dot8<T>(*reinterpret_cast<const uint4 *>(x + c),
                            ld_stream16(w + row * p.up.row_stride + c));
        v[g] = warp_sum(v[g]);
        if (p.up_bias) v[g] += f32(static_cast<const T *>(p.up_bias)[(int64_t)e * p.wide + row]);
    }
    float a[8] = {v[0]};
    if (gated) a[0] = v[0] * sigmoidf(v[0]) * v[1];
    else activate8(p.act, a);
    if (lane == 0) p.h[(int64_t)pair * p.F + f] = a[0];
}

// A warp for each token and output.
template <typename T> __global__ void __launch_bounds__(256) few_down_kernel(const FewParams p) {
    const int lane = threadIdx.x & 31, m = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
    if (m >= p.H) return;
    float sum = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const int pair = t * p.k + j, e = p.idx[pair];
        if (e < 0 || e >= p.E) continue;
        const T *w = static_cast<const T *>(p.down.ptr) + e * p.down.rank_stride + m * p.down.row_stride;
        const float *h = p.h + (int64_t)pair * p.F;
        float v = 0.f;
        for (int c = lane * 8; c < p.F; c += 256) {
            float f[8];
            unpack8<T>(f, ld_stream16(w + c));
#pragma unroll
            for (int i = 0; i < 8; ++i) v += f[i] * h[c + i];
        }
        v = warp_sum(v);
        if (p.down_bias) v += f32(static_cast<const T *>(p.down_bias)[(int64_t)e * p.H + m]);
        sum += p.w[pair] * v;
    }
    if (lane == 0) {
        if (p.residual.ptr) sum += f32(static_cast<const T *>(p.residual.ptr)[t * p.residual.row_stride + m]);
        static_cast<T *>(p.out.ptr)[t * p.out.row_stride + m] = rounded<T>(sum);
    }
}

int64_t wide_of(const ep_few_desc_t &d) { return d.activation == EP_ACT_SWIGLU ? 2 * (int64_t)d.inner : d.inner; }

bool valid(const ep_few_desc_t *d) {
    if (!d || d->tokens < 0 || d->tokens > EP_MAX_FEW_TOKENS) return false;
    if (d->experts < 1 || d->experts > EP_MAX_ROUTE_EXPERTS || d->topk < 1 || d->topk > 32) return false;
    if (d->hidden < 8 || d->hidden % 8 || d->hidden > 1 << 20) return false;
    if (d->inner < 8 || d->inner % 8 || d->inner > 1 << 20) return false;
    if (d->dtype != EP_DT_BF16 && d->dtype != EP_DT_FP16) return false;
    if (d->activation < EP_ACT_NONE || d->activation > EP_ACT_SWIGLU || d->reserved) return false;
    return aligned(d->up_bias, 16) && aligned(d->down_bias, 16) && valid_rows(d->up, d->hidden, d->experts > 1) &&
           valid_rows(d->down, d->inner, d->experts > 1);
}

size_t workspace(const ep_few_desc_t &d) { return (size_t)d.tokens * d.topk * d.inner * 4; }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_moe_few_workspace(const ep_few_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = workspace(*d);
    return EP_SUCCESS;
}

ep_status_t ep_moe_few(const ep_few_desc_t *d, const ep_rows_t *x, const float *d_w, const int32_t *d_idx,
                       const ep_rows_t *residual, const ep_rows_t *out, void *d_workspace, size_t workspace_bytes,
                       uint32_t *d_error, void *stream) {
    EP_RANGE("ep_moe_few");
    if (!valid(d) || !x || !residual || !out || !aligned(d_workspace, 256) || !aligned(d_error, 4))
        return EP_ERR_INVALID_ARGS;
    if (d->tokens == 0) return EP_SUCCESS;
    if (!d_w || !d_idx || !aligned(d_w, 4) || !aligned(d_idx, 4) || !d_workspace || workspace_bytes < workspace(*d) ||
        !valid_rows(*x, d->hidden, false) || !valid_rows(*out, d->hidden, false) ||
        (residual->ptr && !valid_rows(*residual, d->hidden, false)))
        return EP_ERR_INVALID_ARGS;
    const FewParams p = {d->tokens, d->experts, d->topk, d->hidden, d->inner, (int)wide_of(*d), d->activation,
                         d->up, d->down, *x, *residual, *out, d->up_bias, d->down_bias, d_w, d_idx,
                         static_cast<float *>(d_workspace), d_error};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    with_type(d->dtype, [&](auto type) {
        using T = decltype(type);
        few_up_kernel<T><<<dim3((p.F + 7) / 8, p.T * p.k), 256, 0, st>>>(p);
        few_down_kernel<T><<<dim3((p.H + 7) / 8, p.T), 256, 0, st>>>(p);
    });
    return launched();
}

}  // extern "C"
