// Expert products: one matrix product per group of rows, with bias,
// activation and residual in its epilogue, and its gradient.
//
// Every product here is  out[n][m] = sum_k A[m][k] * B[n][k]  over one group:
//   forward   m = feature, n = row,   k = input    A = weight,    B = x
//   grad_x    m = input,   n = row,   k = feature  A = weight^T,  B = d
//   grad_w    m = input,   n = feature, k = row    A = x^T,       B = d^T
// The output's contiguous dimension is always m.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "ep_device.cuh"

namespace ep {
namespace {

constexpr int kTile = 64, kTileK = 16;

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

struct Operand {           // element (i, k) of a group's operand at ptr + base + i * si + k * sk
    const void *ptr;
    int64_t group_stride;  // by group (weights) or by segment (rows)
    int64_t si, sk;
    bool rows_i, rows_k;   // index i / k counts the group's rows
};

struct ProductParams {
    Groups gr;
    Operand a, b;
    int M, N, K;           // N or K < 0: the group's number of rows
    int wide_half;         // SWIGLU: features of one half, else 0
    int act;
    bool out_by_rows;      // n counts rows (else out is per group)
    const void *bias;
    ep_rows_t residual, out, pre;
};

template <typename T> __device__ __forceinline__ float f32(T v);
template <> __device__ __forceinline__ float f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ __nv_bfloat16 rounded(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rounded(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float sigmoidf(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
    case EP_ACT_RELU: return fmaxf(v, 0.f);
    case EP_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case EP_ACT_SILU: return v * sigmoidf(v);
    default: return v;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) product_kernel(const ProductParams p) {
    __shared__ float sa[2][kTileK][kTile + 1], sb[kTileK][kTile + 1];
    const int G = p.gr.R * p.gr.per;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int mt = (p.M + kTile - 1) / kTile;
    int64_t before = 0;
    int64_t tile = blockIdx.x;
    for (int g = 0; g < G; ++g) {
        int first, rows;
        group_range(p.gr, g, &first, &rows);
        const int N = p.N < 0 ? rows : p.N, K = p.K < 0 ? rows : p.K;
        const int64_t tiles = (int64_t)mt * ((N + kTile - 1) / kTile);
        const int seg = g / p.gr.per;
        const T *A = static_cast<const T *>(p.a.ptr) +
                     (p.a.rows_i || p.a.rows_k ? seg : g) * p.a.group_stride +
                     (p.a.rows_k ? first * p.a.sk : 0);
        const T *B = static_cast<const T *>(p.b.ptr) + seg * p.b.group_stride +
                     first * (p.b.rows_i ? p.b.si : p.b.sk);
        for (; tile < before + tiles; tile += gridDim.x) {
            const int m0 = (int)((tile - before) % mt) * kTile, n0 = (int)((tile - before) / mt) * kTile;
            float acc[2][4][4] = {};
            for (int k0 = 0; k0 < K; k0 += kTileK) {
                for (int i = tid; i < kTile * kTileK; i += 256) {
                    const int r = i / kTileK, c = i % kTileK;
                    const bool kin = k0 + c < K;
                    sa[0][c][r] = kin && m0 + r < p.M ? f32(A[(m0 + r) * p.a.si + (k0 + c) * p.a.sk]) : 0.f;
                    if (p.wide_half)
                        sa[1][c][r] = kin && m0 + r < p.M
                                          ? f32(A[(p.wide_half + m0 + r) * p.a.si + (k0 + c) * p.a.sk]) : 0.f;
                    sb[c][r] = kin && n0 + r < N ? f32(B[(n0 + r) * p.b.si + (k0 + c) * p.b.sk]) : 0.f;
                }
                __syncthreads();
                for (int c = 0; c < kTileK; ++c)
                    for (int u = 0; u < 4; ++u)
                        for (int v = 0; v < 4; ++v) {
                            acc[0][u][v] += sb[c][ty + 16 * u] * sa[0][c][tx + 16 * v];
                            if (p.wide_half) acc[1][u][v] += sb[c][ty + 16 * u] * sa[1][c][tx + 16 * v];
                        }
                __syncthreads();
            }
            const int wide = p.wide_half ? 2 * p.wide_half : p.M;
            for (int u = 0; u < 4; ++u)
                for (int v = 0; v < 4; ++v) {
                    const int n = n0 + ty + 16 * u, m = m0 + tx + 16 * v;
                    if (n >= N || m >= p.M) continue;
                    const int64_t row = p.out_by_rows ? first + n : n;
                    const int64_t own = p.out_by_rows ? seg : g;
                    float h0 = acc[0][u][v], h1 = acc[1][u][v];
                    if (p.bias) {
                        const T *bias = static_cast<const T *>(p.bias) + (int64_t)g * wide;
                        h0 += f32(bias[m]);
                        if (p.wide_half) h1 += f32(bias[p.wide_half + m]);
                    }
                    if (p.pre.ptr) {
                        T *pre = static_cast<T *>(p.pre.ptr) + own * p.pre.rank_stride + row * p.pre.row_stride;
                        pre[m] = rounded<T>(h0);
                        if (p.wide_half) pre[p.wide_half + m] = rounded<T>(h1);
                    }
                    float y = p.wide_half ? h0 * sigmoidf(h0) * h1 : activate(p.act, h0);
                    if (p.residual.ptr)
                        y += f32(static_cast<const T *>(p.residual.ptr)[own * p.residual.rank_stride +
                                                                        row * p.residual.row_stride + m]);
                    static_cast<T *>(p.out.ptr)[own * p.out.rank_stride + row * p.out.row_stride + m] =
                        rounded<T>(y);
                }
        }
        before += tiles;
    }
}

// d = grad * act'(pre) over every group's rows, rounded once for the
// products, and its column sums before that rounding.  One block takes 256
// features of one group, thread t feature t, rows in order.
struct ActGradParams {
    Groups gr;
    int N, act;
    ep_rows_t grad, pre, d;
    void *grad_bias;        // [G][wide] or null
    bool write;
};

template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(const ActGradParams p) {
    const int g = blockIdx.y, seg = g / p.gr.per;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.N) return;
    int first, rows;
    group_range(p.gr, g, &first, &rows);
    const bool gated = p.act == EP_ACT_SWIGLU;
    float s0 = 0.f, s1 = 0.f;
    for (int i = first; i < first + rows; ++i) {
        const float gy = f32(static_cast<const T *>(p.grad.ptr)[seg * p.grad.rank_stride + i * p.grad.row_stride + c]);
        float d0 = gy, d1 = 0.f;
        if (p.act != EP_ACT_NONE) {
            const T *pre = static_cast<const T *>(p.pre.ptr) + seg * p.pre.rank_stride + i * p.pre.row_stride;
            const float v = f32(pre[c]);
            if (p.act == EP_ACT_RELU) {
                d0 = v > 0.f ? gy : 0.f;
            } else if (p.act == EP_ACT_GELU) {
                // Phi(v) + v phi(v), phi(v) = exp(-v^2/2) / sqrt(2 pi)
                d0 = gy * (0.5f * (1.0f + erff(v * 0.70710678118654752f)) +
                           v * expf(-0.5f * v * v) * 0.39894228040143268f);
            } else {
                const float s = sigmoidf(v), slope = s * (1.0f + v * (1.0f - s));
                if (gated) {
                    const float up = f32(pre[p.N + c]);
                    d0 = gy * up * slope;
                    d1 = gy * v * s;
                } else {
                    d0 = gy * slope;
                }
            }
        }
        if (p.write) {
            T *d = static_cast<T *>(p.d.ptr) + seg * p.d.rank_stride + i * p.d.row_stride;
            d[c] = rounded<T>(d0);
            if (gated) d[p.N + c] = rounded<T>(d1);
        }
        s0 += d0;
        s1 += d1;
    }
    if (p.grad_bias) {
        T *gb = static_cast<T *>(p.grad_bias) + (int64_t)g * (gated ? 2 * p.N : p.N);
        gb[c] = rounded<T>(s0);
        if (gated) gb[p.N + c] = rounded<T>(s1);
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of `width` elements: 16-byte aligned, dense rows that do not overlap.
bool valid_rows(const ep_rows_t &r, int64_t width, bool many) {
    return r.ptr && aligned(r.ptr, 16) && r.row_stride >= width && r.row_stride % 8 == 0 &&
           (!many || (r.rank_stride >= 0 && r.rank_stride % 8 == 0));
}

int64_t wide_of(const ep_product_desc_t &d) {
    return d.activation == EP_ACT_SWIGLU ? 2 * (int64_t)d.out_features : d.out_features;
}

bool valid(const ep_product_desc_t *d) {
    if (!d || d->ranks < 1 || d->groups < 1 || (int64_t)d->ranks * d->groups > 65535) return false;
    if (d->rows < 0 || d->rows > 1 << 30) return false;
    if (d->in_features < 8 || d->in_features % 8 || d->in_features > 1 << 24) return false;
    if (d->out_features < 8 || d->out_features % 8 || d->out_features > 1 << 24) return false;
    if (d->dtype != EP_DT_BF16 && d->dtype != EP_DT_FP16) return false;
    if (d->activation < EP_ACT_NONE || d->activation > EP_ACT_SWIGLU || d->reserved) return false;
    if ((d->d_count == nullptr) != (d->d_offset == nullptr)) return false;
    if (!d->d_count && d->groups != 1) return false;
    if (!aligned(d->d_count, 4) || !aligned(d->d_offset, 4)) return false;
    const bool many = d->ranks > 1;
    return valid_rows(d->weight, d->in_features, (int64_t)d->ranks * d->groups > 1) &&
           (d->rows == 0 || valid_rows(d->x, d->in_features, many));
}

Groups groups_of(const ep_product_desc_t &d) {
    return Groups{d.d_count, d.d_offset, d.ranks, d.groups, d.rows};
}

template <typename F> void with_type(int dtype, F f) {
    if (dtype == EP_DT_BF16) f(__nv_bfloat16());
    else f(__half());
}

ep_status_t launched() { return cudaGetLastError() == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP; }

void launch_product(const ep_product_desc_t &d, const ProductParams &p, cudaStream_t st) {
    with_type(d.dtype, [&](auto type) { product_kernel<decltype(type)><<<152 * 4, 256, 0, st>>>(p); });
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_expert_product(const ep_product_desc_t *d, const void *d_bias,
                              const ep_rows_t *residual, const ep_rows_t *y, const ep_rows_t *pre,
                              uint32_t *d_error, void *stream) {
    EP_RANGE("ep_expert_product");
    if (!valid(d) || !residual || !y || !pre || !aligned(d_bias, 16) || !aligned(d_error, 4))
        return EP_ERR_INVALID_ARGS;
    if (d->rows == 0) return EP_SUCCESS;
    const bool many = d->ranks > 1;
    if (!valid_rows(*y, d->out_features, many) ||
        (residual->ptr && !valid_rows(*residual, d->out_features, many)) ||
        (pre->ptr && !valid_rows(*pre, wide_of(*d), many)))
        return EP_ERR_INVALID_ARGS;
    ProductParams p = {};
    p.gr = groups_of(*d);
    p.a = Operand{d->weight.ptr, d->weight.rank_stride, d->weight.row_stride, 1, false, false};
    p.b = Operand{d->x.ptr, d->x.rank_stride, d->x.row_stride, 1, true, false};
    p.M = d->out_features;
    p.N = -1;
    p.K = d->in_features;
    p.wide_half = d->activation == EP_ACT_SWIGLU ? d->out_features : 0;
    p.act = d->activation;
    p.out_by_rows = true;
    p.bias = d_bias;
    p.residual = *residual;
    p.out = *y;
    p.pre = *pre;
    launch_product(*d, p, static_cast<cudaStream_t>(stream));
    return launched();
}

ep_status_t ep_expert_product_workspace(const ep_product_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = d->activation == EP_ACT_NONE
                 ? 0 : align256((size_t)d->ranks * d->rows * (size_t)wide_of(*d) * 2);
    return EP_SUCCESS;
}

ep_status_t ep_expert_product_backward(const ep_product_desc_t *d, const ep_rows_t *grad,
                                       const ep_rows_t *pre, const ep_rows_t *grad_x, void *d_grad_w,
                                       void *d_grad_bias, void *d_workspace, size_t workspace_bytes,
                                       uint32_t *d_error, void *stream) {
    EP_RANGE("ep_expert_product_backward");
    if (!valid(d) || !grad || !pre || !grad_x || !aligned(d_grad_w, 16) || !aligned(d_grad_bias, 16) ||
        !aligned(d_workspace, 256) || !aligned(d_error, 4))
        return EP_ERR_INVALID_ARGS;
    const bool many = d->ranks > 1, act = d->activation != EP_ACT_NONE;
    const int64_t wide = wide_of(*d);
    size_t need = 0;
    ep_expert_product_workspace(d, &need);
    if (workspace_bytes < need || (need && !d_workspace)) return EP_ERR_INVALID_ARGS;
    if (d->rows > 0 && (!valid_rows(*grad, d->out_features, many) ||
                        (act && !valid_rows(*pre, wide, many)) ||
                        (grad_x->ptr && !valid_rows(*grad_x, d->in_features, many))))
        return EP_ERR_INVALID_ARGS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Groups gr = groups_of(*d);
    const ep_rows_t dd = act ? ep_rows_t{d_workspace, d->rows * wide, wide} : *grad;
    if (act || d_grad_bias) {
        ActGradParams a = {gr, d->out_features, d->activation, *grad, *pre, dd, d_grad_bias, act};
        const dim3 grid((d->out_features + 255) / 256, gr.R * gr.per);
        with_type(d->dtype, [&](auto type) { act_grad_kernel<decltype(type)><<<grid, 256, 0, st>>>(a); });
    }
    if (grad_x->ptr && d->rows > 0) {
        ProductParams p = {};
        p.gr = gr;
        p.a = Operand{d->weight.ptr, d->weight.rank_stride, 1, d->weight.row_stride, false, false};
        p.b = Operand{dd.ptr, dd.rank_stride, dd.row_stride, 1, true, false};
        p.M = d->in_features;
        p.N = -1;
        p.K = (int)wide;
        p.out_by_rows = true;
        p.out = *grad_x;
        launch_product(*d, p, st);
    }
    if (d_grad_w) {
        ProductParams p = {};
        p.gr = gr;
        p.a = Operand{d->x.ptr, d->x.rank_stride, 1, d->x.row_stride, false, true};
        p.b = Operand{dd.ptr, dd.rank_stride, 1, dd.row_stride, false, true};
        p.M = d->in_features;
        p.N = (int)wide;
        p.K = -1;
        p.out = ep_rows_t{d_grad_w, wide * d->in_features, d->in_features};
        launch_product(*d, p, st);
    }
    return launched();
}

}  // extern "C"
