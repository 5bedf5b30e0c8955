// Top-k routing, the balance and z losses, and the gradient of both by the
// router logits.
//
// One warp per token: the row of E logits lies in registers, lane l holding
// experts l, l + 32, ...  Softmax statistics are warp reductions in fp32.
// Top-k is k rounds of a warp-wide maximum over order-preserving integer
// keys; a tie goes to the lowest expert id by a second, minimum reduction.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "ep_device.cuh"

namespace ep {
namespace {

constexpr int kRouteWarps = 4;
constexpr int kLossWarps = 8;

struct RouteParams {
    const void *logits;
    int64_t row_stride, rank_stride;
    TokenCounts nt;
    int W, T, E, k;
    float scale;
    const float *bias;       // forward
    float *w;                // forward
    int32_t *idx_out;        // forward
    const float *grad_w;     // backward
    const int32_t *idx;      // loss, backward
    const float *grad_loss;  // backward
    const int32_t *counts;   // backward
    void *grad_logits;       // backward
    float balance_coef, z_coef, inv_n;
    float *part;             // loss: [blocks][E + 1] partial sums
    int32_t *part_count;     // loss: [blocks][E]
    float *loss, *probs;
    int32_t *counts_out;
    uint32_t *error;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// NaN reads as -inf (closed), +inf as the largest finite number, so that
// differences of logits are never inf - inf between open experts.
__device__ __forceinline__ float sane_logit(float v) {
    return v != v ? -INFINITY : fminf(v, FLT_MAX);
}

// Unsigned integers in the order of the floats (-0 counts as +0).  Every
// value, -inf included, maps above 0, which marks "no candidate".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename T>
__device__ __forceinline__ const T *logit_row(const RouteParams &p, int s, int t) {
    return static_cast<const T *>(p.logits) + s * p.rank_stride + t * p.row_stride;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_row(const RouteParams &p, const T *row, int lane, float *x) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < p.E ? sane_logit(to_f32(row[e])) : -INFINITY;
    }
}

// Softmax statistics of a row: the largest logit and 1 / sum exp(x - max).
// Probabilities are taken from the pair: m + log(sum) in one number would
// lose the sum's digits where |m| is large.
struct RowStats {
    float m, inv_sum;
    bool open;                   // some expert is open
    __device__ float prob(float x) const { return open ? expf(x - m) * inv_sum : 0.f; }
    __device__ float lse() const { return open ? m - logf(inv_sum) : 0.f; }
};

// Softmax over the warp's row: probabilities in place of x (all 0 when no
// expert is open).
template <int VPL>
__device__ __forceinline__ RowStats softmax_row(float *x) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    if (m == -INFINITY) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = 0.f;
        return RowStats{0.f, 1.f, false};
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        x[i] = expf(x[i] - m);
        sum += x[i];
    }
    sum = warp_sum(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] *= inv;
    return RowStats{m, inv, true};
}

// Softmax over the chosen experts (lane j < k holds x_j of choice j).
__device__ __forceinline__ float chosen_softmax(float xj, bool mine) {
    const float m = warp_max(mine ? xj : -INFINITY);
    const float e = mine && m > -INFINITY ? expf(xj - m) : 0.f;
    const float sum = warp_sum(e);
    return sum > 0.f ? e / sum : 0.f;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p, bool softmax,
                                                                 bool renorm) {
    const int lane = threadIdx.x & 31;
    const int64_t tok = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (tok >= (int64_t)p.W * p.T) return;
    const int s = (int)(tok / p.T), t = (int)(tok - (int64_t)s * p.T);
    if (t >= p.nt.n[s]) {
        if (lane < p.k) {
            p.w[tok * p.k + lane] = 0.f;
            p.idx_out[tok * p.k + lane] = -1;
        }
        return;
    }
    float x[VPL];
    uint32_t key[VPL];
    load_row<T, VPL>(p, logit_row<T>(p, s, t), lane, x);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < p.E ? order_key(p.bias ? x[i] + p.bias[e] : x[i]) : 0u;
    }
    int mine_e = 0;
    float mine_x = -INFINITY;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int be = 0;
        float bx = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                be = lane + 32 * i;
                bx = x[i];
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)be : 0xffffffffu);
        const float xe = __shfl_sync(0xffffffffu, bx, e & 31);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((uint32_t)(lane + 32 * i) == e) key[i] = 0;
        if (lane == j) {
            mine_e = (int)e;
            mine_x = xe;
        }
    }
    const bool mine = lane < p.k;
    float v;
    if (softmax && renorm) {
        v = chosen_softmax(mine_x, mine);
    } else if (softmax) {
        const RowStats st = softmax_row<VPL>(x);
        v = mine ? st.prob(mine_x) : 0.f;
    } else {
        v = mine ? sigmoid(mine_x) : 0.f;
        if (renorm) {
            const float sum = warp_sum(v);
            v = sum > 0.f ? v / sum : 0.f;
        }
    }
    if (mine) {
        p.w[tok * p.k + lane] = v * p.scale;
        p.idx_out[tok * p.k + lane] = mine_e;
    }
}

template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const RouteParams p, bool softmax, bool renorm) {
    const int lane = threadIdx.x & 31;
    const int64_t tok = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (tok >= (int64_t)p.W * p.T) return;
    const int s = (int)(tok / p.T), t = (int)(tok - (int64_t)s * p.T);
    T *out = static_cast<T *>(p.grad_logits) + tok * p.E;
    if (t >= p.nt.n[s]) {
        for (int e = lane; e < p.E; e += 32) out[e] = from_f32<T>(0.f);
        return;
    }
    const T *row = logit_row<T>(p, s, t);
    float d[VPL], pr[VPL];
    RowStats st = {0.f, 1.f, false};
    const bool dense = p.grad_loss || (p.grad_w && softmax && !renorm);
    if (dense) {
        load_row<T, VPL>(p, row, lane, pr);
        st = softmax_row<VPL>(pr);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.f;
    if (p.grad_w) {
        int id = -1;
        float g = 0.f, xj = -INFINITY;
        if (lane < p.k) {
            id = p.idx[tok * p.k + lane];
            if ((uint32_t)id < (uint32_t)p.E) {
                g = p.grad_w[tok * p.k + lane] * p.scale;
                xj = sane_logit(to_f32(row[id]));
            } else {
                id = -1;
                if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
            }
        }
        const bool mine = id >= 0;
        float dj, inner = 0.f;
        if (softmax && renorm) {
            const float v = chosen_softmax(xj, mine);
            dj = v * (g - warp_sum(g * v));
        } else if (softmax) {
            const float v = mine ? st.prob(xj) : 0.f;
            inner = warp_sum(g * v);
            dj = v * g;
        } else {
            const float v = mine ? sigmoid(xj) : 0.f;
            float dv = g;
            if (renorm) {
                const float sum = warp_sum(v), dot = warp_sum(g * v);
                dv = sum > 0.f ? (g - dot / sum) / sum : 0.f;
            }
            dj = dv * v * (1.0f - v);
        }
        for (int j = 0; j < p.k; ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float de = __shfl_sync(0xffffffffu, dj, j);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e == lane + 32 * i) d[i] += de;
        }
        if (softmax && !renorm) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) d[i] -= pr[i] * inner;
        }
    }
    if (p.grad_loss) {
        const float gl = *p.grad_loss * p.inv_n, lse = st.lse();
        const float share = p.inv_n * ((float)p.E / (float)p.k);
        float f[VPL], dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i;
            f[i] = e < p.E ? (float)p.counts[e] * share : 0.f;
            dot += pr[i] * f[i];
        }
        dot = warp_sum(dot);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            d[i] += pr[i] * ((f[i] - dot) * p.balance_coef + 2.0f * p.z_coef * lse) * gl;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E) out[e] = from_f32<T>(d[i]);
    }
}

// Losses, pass 1: every block sums softmax probabilities and lse^2 of its
// tokens (a warp's tokens in registers, then the warps in order) and counts
// choices in shared memory.
template <typename T, int VPL>
__global__ void __launch_bounds__(kLossWarps * 32) balance_partial_kernel(const RouteParams p) {
    extern __shared__ float sh[];                 // [kLossWarps][E + 1], then [E] counts
    int32_t *cnt = reinterpret_cast<int32_t *>(sh + kLossWarps * (p.E + 1));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    float acc[VPL], z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
    const int64_t total = (int64_t)p.W * p.T;
    for (int64_t tok = (int64_t)blockIdx.x * kLossWarps + warp; tok < total;
         tok += (int64_t)gridDim.x * kLossWarps) {
        const int s = (int)(tok / p.T), t = (int)(tok - (int64_t)s * p.T);
        if (t >= p.nt.n[s]) continue;
        if (lane < p.k) {
            const int id = p.idx[tok * p.k + lane];
            if ((uint32_t)id < (uint32_t)p.E) atomicAdd(&cnt[id], 1);
            else if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
        }
        float x[VPL];
        load_row<T, VPL>(p, logit_row<T>(p, s, t), lane, x);
        const float lse = softmax_row<VPL>(x).lse();
        z += lse * lse;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += x[i];
    }
    float *mine = sh + warp * (p.E + 1);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < p.E) mine[lane + 32 * i] = acc[i];
    if (lane == 0) mine[p.E] = z;
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
        float sum = 0.f;
        for (int w = 0; w < kLossWarps; ++w) sum += sh[w * (p.E + 1) + e];
        p.part[(int64_t)blockIdx.x * (p.E + 1) + e] = sum;
        if (e < p.E) p.part_count[(int64_t)blockIdx.x * p.E + e] = cnt[e];
    }
}

// Losses, pass 2: one block joins the blocks' sums; lanes are experts, warp w
// takes blocks w, w + 32, ..., and the warps' sums are added in order.
__global__ void __launch_bounds__(1024) balance_final_kernel(const RouteParams p, int blocks) {
    __shared__ float sh[32][33];
    __shared__ int32_t sc[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float balance = 0.f, z = 0.f;                 // warp 0's
    for (int e0 = 0; e0 <= p.E; e0 += 32) {
        const int e = e0 + lane;
        float sum = 0.f;
        int32_t c = 0;
        if (e <= p.E)
            for (int b = warp; b < blocks; b += 32) {
                sum += p.part[(int64_t)b * (p.E + 1) + e];
                if (e < p.E) c += p.part_count[(int64_t)b * p.E + e];
            }
        sh[warp][lane] = sum;
        sc[warp][lane] = c;
        __syncthreads();
        if (warp == 0 && e <= p.E) {
            sum = 0.f;
            c = 0;
            for (int w = 0; w < 32; ++w) {
                sum += sh[w][lane];
                c += sc[w][lane];
            }
            sum *= p.inv_n;
            if (e < p.E) {
                p.probs[e] = sum;
                p.counts_out[e] = c;
                balance += (float)c * (p.inv_n * ((float)p.E / (float)p.k)) * sum;
            } else {
                z = sum;
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        balance = warp_sum(balance);
        z = warp_sum(z);
        if (lane == 0) {
            p.loss[0] = p.balance_coef * balance + p.z_coef * z;
            p.loss[1] = balance;
            p.loss[2] = z;
        }
    }
}

int loss_blocks(const ep_route_desc_t &d) {
    const int64_t tokens = (int64_t)d.world_size * d.tokens;
    const int64_t want = (tokens + kLossWarps - 1) / kLossWarps;
    return (int)(want < 152 ? want : 152);
}

// Calls f(T(), integral VPL) for the logits' type and the row length.
template <int V> struct Int { static constexpr int value = V; };
template <typename T, typename F> void with_row(int E, F f) {
    if (E <= 32) f(T(), Int<1>());
    else if (E <= 64) f(T(), Int<2>());
    else if (E <= 128) f(T(), Int<4>());
    else if (E <= 256) f(T(), Int<8>());
    else if (E <= 512) f(T(), Int<16>());
    else f(T(), Int<32>());
}
template <typename F> void with_types(int dtype, int E, F f) {
    if (dtype == EP_DT_BF16) with_row<__nv_bfloat16>(E, f);
    else if (dtype == EP_DT_FP16) with_row<__half>(E, f);
    else with_row<float>(E, f);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid(const ep_route_desc_t *d) {
    if (!d) return false;
    if (d->world_size < 1 || d->world_size > EP_MAX_WORLD || d->tokens < 1) return false;
    if ((int64_t)d->world_size * d->tokens > (int64_t)1 << 30) return false;
    if (d->num_experts < 1 || d->num_experts > EP_MAX_ROUTE_EXPERTS) return false;
    if (d->topk < 1 || d->topk > EP_MAX_TOPK || d->topk > d->num_experts) return false;
    if (d->dtype != EP_DT_BF16 && d->dtype != EP_DT_FP16 && d->dtype != EP_DT_FP32) return false;
    if (d->score != EP_SCORE_SOFTMAX && d->score != EP_SCORE_SIGMOID) return false;
    if (d->row_stride < d->num_experts) return false;
    return d->world_size == 1 || d->rank_stride >= 0;
}

bool make_params(const ep_route_desc_t *d, const void *logits, const int32_t *h_nt, RouteParams *p) {
    if (!valid(d) || !logits || !h_nt) return false;
    if (!aligned(logits, d->dtype == EP_DT_FP32 ? 4 : 2)) return false;
    *p = RouteParams{};
    int64_t n = 0;
    for (int s = 0; s < d->world_size; ++s) {
        if (h_nt[s] < 0 || h_nt[s] > d->tokens) return false;
        p->nt.n[s] = h_nt[s];
        n += h_nt[s];
    }
    p->logits = logits;
    p->row_stride = d->row_stride;
    p->rank_stride = d->world_size == 1 ? 0 : d->rank_stride;
    p->W = d->world_size;
    p->T = d->tokens;
    p->E = d->num_experts;
    p->k = d->topk;
    p->scale = d->scale;
    p->balance_coef = d->balance_coef;
    p->z_coef = d->z_coef;
    p->inv_n = n > 0 ? 1.0f / (float)n : 0.f;
    return true;
}

ep_status_t launched() { return cudaGetLastError() == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP; }

unsigned token_blocks(const RouteParams &p) {
    return (unsigned)(((int64_t)p.W * p.T + kRouteWarps - 1) / kRouteWarps);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_route(const ep_route_desc_t *d, const void *d_logits, const float *d_bias,
                     const int32_t *h_num_tokens, float *d_w, int32_t *d_idx, void *stream) {
    EP_RANGE("ep_route");
    RouteParams p;
    if (!make_params(d, d_logits, h_num_tokens, &p)) return EP_ERR_INVALID_ARGS;
    if (!d_w || !d_idx || !aligned(d_w, 4) || !aligned(d_idx, 4) || !aligned(d_bias, 4))
        return EP_ERR_INVALID_ARGS;
    p.bias = d_bias;
    p.w = d_w;
    p.idx_out = d_idx;
    const bool softmax = d->score == EP_SCORE_SOFTMAX, renorm = d->renormalize != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    with_types(d->dtype, p.E, [&](auto type, auto vpl) {
        route_kernel<decltype(type), decltype(vpl)::value>
            <<<token_blocks(p), kRouteWarps * 32, 0, st>>>(p, softmax, renorm);
    });
    return launched();
}

ep_status_t ep_route_backward(const ep_route_desc_t *d, const void *d_logits,
                              const float *d_grad_w, const int32_t *d_idx,
                              const float *d_grad_loss, const int32_t *d_counts,
                              const int32_t *h_num_tokens, void *d_grad_logits,
                              uint32_t *d_error, void *stream) {
    EP_RANGE("ep_route_backward");
    RouteParams p;
    if (!make_params(d, d_logits, h_num_tokens, &p)) return EP_ERR_INVALID_ARGS;
    if ((d_grad_w == nullptr) != (d_idx == nullptr) ||
        (d_grad_loss == nullptr) != (d_counts == nullptr) || (!d_grad_w && !d_grad_loss))
        return EP_ERR_INVALID_ARGS;
    if (!d_grad_logits || !aligned(d_grad_logits, d->dtype == EP_DT_FP32 ? 4 : 2) ||
        !aligned(d_grad_w, 4) || !aligned(d_idx, 4) || !aligned(d_grad_loss, 4) ||
        !aligned(d_counts, 4) || !aligned(d_error, 4))
        return EP_ERR_INVALID_ARGS;
    p.grad_w = d_grad_w;
    p.idx = d_idx;
    p.grad_loss = d_grad_loss;
    p.counts = d_counts;
    p.grad_logits = d_grad_logits;
    p.error = d_error;
    const bool softmax = d->score == EP_SCORE_SOFTMAX, renorm = d->renormalize != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    with_types(d->dtype, p.E, [&](auto type, auto vpl) {
        route_backward_kernel<decltype(type), decltype(vpl)::value>
            <<<token_blocks(p), kRouteWarps * 32, 0, st>>>(p, softmax, renorm);
    });
    return launched();
}

ep_status_t ep_balance_loss_workspace(const ep_route_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = (size_t)loss_blocks(*d) * (2 * (size_t)d->num_experts + 1) * 4;
    return EP_SUCCESS;
}

ep_status_t ep_balance_loss(const ep_route_desc_t *d, const void *d_logits, const int32_t *d_idx,
                            const int32_t *h_num_tokens, float *d_loss, int32_t *d_counts,
                            float *d_probs, void *d_workspace, size_t workspace_bytes,
                            uint32_t *d_error, void *stream) {
    EP_RANGE("ep_balance_loss");
    RouteParams p;
    size_t need = 0;
    if (!make_params(d, d_logits, h_num_tokens, &p)) return EP_ERR_INVALID_ARGS;
    if (!d_idx || !d_loss || !d_counts || !d_probs || !d_workspace || !aligned(d_idx, 4) ||
        !aligned(d_loss, 4) || !aligned(d_counts, 4) || !aligned(d_probs, 4) ||
        !aligned(d_workspace, 16) || !aligned(d_error, 4))
        return EP_ERR_INVALID_ARGS;
    ep_balance_loss_workspace(d, &need);
    if (workspace_bytes < need) return EP_ERR_INVALID_ARGS;
    const int blocks = loss_blocks(*d);
    p.idx = d_idx;
    p.loss = d_loss;
    p.counts_out = d_counts;
    p.probs = d_probs;
    p.error = d_error;
    p.part = static_cast<float *>(d_workspace);
    p.part_count = reinterpret_cast<int32_t *>(p.part + (size_t)blocks * (p.E + 1));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t sh = ((size_t)kLossWarps * (p.E + 1) + p.E) * 4;    // 36 KB at most
    with_types(d->dtype, p.E, [&](auto type, auto vpl) {
        balance_partial_kernel<decltype(type), decltype(vpl)::value>
            <<<blocks, kLossWarps * 32, sh, st>>>(p);
    });
    balance_final_kernel<<<1, 1024, 0, st>>>(p, blocks);
    return launched();
}

}  // extern "C"
