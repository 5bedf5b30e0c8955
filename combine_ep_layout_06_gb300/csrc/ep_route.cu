// Top-k routing, the balance and z losses, and the gradient of both by the
// router logits.
//
// A token's row of E logits lies in the registers of LANES neighbouring lanes,
// 8 (or, past 256 experts, 16 or 32) neighbouring experts each, so that lane
// order is expert order and a warp holds 32 / LANES tokens: with 8 experts a
// thread has a token to itself.  Softmax statistics are fp32 reductions over
// those lanes.  Top-k takes the largest remaining key k times over; a lane
// keeps its two best keys at hand and looks through its own again when both
// are taken.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "ep_device.cuh"

namespace ep {
namespace {

constexpr int kRouteWarps = 4;
constexpr int kLossWarps = 32;

struct RouteParams {
    const void *logits;
    int64_t row_stride, rank_stride;
    TokenCounts nt;
    int W, T, E, k;
    bool vec;                // rows of logits (and of their gradient) in 16-byte pieces
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

// Reductions over the LANES lanes of a token.
template <int LANES> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES> __device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int LANES> __device__ __forceinline__ uint32_t row_max_key(uint32_t v) {
    if constexpr (LANES == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// exp of a difference of logits, within 2^-22 (1 + |d| / 2) of it: the callers'
// sums and 1e-5 tolerances are far above.
__device__ __forceinline__ float exp_diff(float d) { return __expf(d); }

template <typename T>
__device__ __forceinline__ const T *logit_row(const RouteParams &p, int s, int t) {
    return static_cast<const T *>(p.logits) + s * p.rank_stride + t * p.row_stride;
}

// Experts l * VPL .. l * VPL + VPL - 1 of a row; -inf past the last expert.
template <typename T, int VPL>
__device__ __forceinline__ void load_row(const RouteParams &p, const T *row, int l, float *x) {
    constexpr int kPer = 16 / sizeof(T);
    if (p.vec) {             // E is a multiple of 8: every piece is inside or outside
#pragma unroll
        for (int c = 0; c < VPL; c += kPer) {
            const int e = l * VPL + c;
            if (e < p.E) {
                const uint4 v = ld_stream16(row + e);
                const T *s = reinterpret_cast<const T *>(&v);
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[c + i] = sane_logit(to_f32(s[i]));
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[c + i] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = l * VPL + i;
            x[i] = e < p.E ? sane_logit(to_f32(row[e])) : -INFINITY;
        }
    }
}
template <typename T, int VPL>
__device__ __forceinline__ void store_row(const RouteParams &p, T *row, int l, const float *d) {
    constexpr int kPer = 16 / sizeof(T);
    if (p.vec) {
#pragma unroll
        for (int c = 0; c < VPL; c += kPer) {
            const int e = l * VPL + c;
            __align__(16) T s[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[i] = from_f32<T>(d[c + i]);
            if (e < p.E) *reinterpret_cast<uint4 *>(row + e) = *reinterpret_cast<const uint4 *>(s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (l * VPL + i < p.E) row[l * VPL + i] = from_f32<T>(d[i]);
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

// Softmax over a token's row: probabilities in place of x (all 0 when no
// expert is open).
template <int LANES, int VPL>
__device__ __forceinline__ RowStats softmax_row(float *x) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = row_max<LANES>(m);
    const bool open = m > -INFINITY;
    if (!open) m = 0.f;                      // every exponential is then 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        x[i] = exp_diff(x[i] - m);
        sum += x[i];
    }
    sum = row_sum<LANES>(sum);
    const float inv = open ? 1.0f / sum : 1.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] *= inv;
    return RowStats{m, inv, open};
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A token's place: lane l of its LANES, token t of rank blockIdx.y.
template <int LANES> struct Place {
    int l, s, t;
    int64_t tok;
    bool in, present;
    __device__ explicit Place(const RouteParams &p, int warps) {
        constexpr int kTokens = 32 / LANES;              // of a warp
        const int lane = threadIdx.x & 31;
        l = lane % LANES;
        s = blockIdx.y;
        t = (blockIdx.x * warps + (threadIdx.x >> 5)) * kTokens + lane / LANES;
        tok = (int64_t)s * p.T + t;
        in = t < p.T;
        present = t < p.nt.n[s];
    }
};

// Choice j of a token is held by lane j % LANES of its lanes, in slot
// j / LANES; with 32 choices at most and at most 8 * LANES experts below 32
// lanes, min(8, 32 / LANES) slots are enough.
template <int LANES> __host__ __device__ constexpr int slots_of() { return 32 / LANES < 8 ? 32 / LANES : 8; }

// Scores of the chosen experts from their logits c[] (mine: slot is a choice)
// and the row's statistics.  v[]: scale 1.  For the sigmoid *sum is what
// renormalising divides by.
template <int LANES, int SLOTS>
__device__ __forceinline__ void chosen_scores(bool softmax, bool renorm, const RowStats &st, const float *c,
                                              const bool *mine, float *v, float *sum) {
    *sum = 0.f;
    if (softmax && renorm) {
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) m = fmaxf(m, mine[q] ? c[q] : -INFINITY);
        m = row_max<LANES>(m);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            v[q] = mine[q] && m > -INFINITY ? expf(c[q] - m) : 0.f;
            *sum += v[q];
        }
        *sum = row_sum<LANES>(*sum);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) v[q] = *sum > 0.f ? v[q] / *sum : 0.f;
    } else if (softmax) {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) v[q] = mine[q] ? st.prob(c[q]) : 0.f;
    } else {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            v[q] = mine[q] ? sigmoid(c[q]) : 0.f;
            *sum += v[q];
        }
        if (renorm) *sum = row_sum<LANES>(*sum);
    }
}

template <typename T, int LANES, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p, bool softmax,
                                                                 bool renorm) {
    constexpr int SLOTS = slots_of<LANES>();
    const Place<LANES> at(p, kRouteWarps);
    const T *row = logit_row<T>(p, at.s, at.present ? at.t : 0);
    float x[VPL];
    if (at.present) {
        load_row<T, VPL>(p, row, at.l, x);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = -INFINITY;
    }
    // this lane's best and second best key: the larger one, or the earlier expert
    uint32_t key[VPL], best = 0, second = 0;
    int be = 0, se = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = at.l * VPL + i;
        key[i] = e < p.E ? order_key(p.bias ? x[i] + p.bias[e] : x[i]) : 0u;
        const bool first = key[i] > best, next = key[i] > second;
        second = first ? best : next ? key[i] : second;
        se = first ? be : next ? i : se;
        best = first ? key[i] : best;
        be = first ? i : be;
    }
    const uint32_t lanes = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << ((threadIdx.x & 31) & ~(LANES - 1));
    int id[SLOTS];
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) id[q] = -1;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t top = row_max_key<LANES>(best);
        const uint32_t who = __ballot_sync(0xffffffffu, best == top) & lanes;
        const int winner = __ffs(who) - 1;               // the first lane has the first expert
        const int e = __shfl_sync(0xffffffffu, at.l * VPL + be, winner);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q)
            if (j == q * LANES + at.l) id[q] = e;
        bool again = false;
        if ((threadIdx.x & 31) == winner) {
            again = second == 0;
            if (!again) {
                best = second;
                be = se;
                second = 0;
            }
        }
        if (__any_sync(0xffffffffu, again)) {
            // both keys are taken: the best two after the one taken last (equal
            // keys in the order of the experts)
            if (again) {
                const uint32_t last = best;
                const int le = be;
                best = second = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    const bool open = key[i] < last || (key[i] == last && i > le);
                    const uint32_t v = open ? key[i] : 0u;
                    const bool first = v > best, next = v > second;
                    second = first ? best : next ? v : second;
                    se = first ? be : next ? i : se;
                    best = first ? v : best;
                    be = first ? i : be;
                }
            }
        }
    }
    float c[SLOTS], v[SLOTS], sum;
    bool mine[SLOTS];
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
        mine[q] = at.present && q * LANES + at.l < p.k;
        c[q] = mine[q] ? sane_logit(to_f32(row[id[q]])) : -INFINITY;
    }
    RowStats st = {0.f, 1.f, false};
    if (softmax && !renorm) st = softmax_row<LANES, VPL>(x);
    chosen_scores<LANES, SLOTS>(softmax, renorm, st, c, mine, v, &sum);
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
        const int j = q * LANES + at.l;
        if (!softmax && renorm) v[q] = sum > 0.f ? v[q] / sum : 0.f;
        if (at.in && j < p.k) {
            p.w[at.tok * p.k + j] = mine[q] ? v[q] * p.scale : 0.f;
            p.idx_out[at.tok * p.k + j] = mine[q] ? id[q] : -1;
        }
    }
}

// The weights' gradient is nonzero at the chosen experts (and, for a softmax
// that is not renormalised, dense): the row meets in shared memory, where the
// chosen experts' terms are added to the dense part, one choice after the
// other where an expert was chosen twice.
template <typename T, int LANES, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const RouteParams p, bool softmax, bool renorm) {
    constexpr int SLOTS = slots_of<LANES>();
    constexpr int kTokens = 32 / LANES, kRow = LANES * VPL;
    __shared__ __align__(16) float rows[kRouteWarps * kTokens][kRow + 4];
    const Place<LANES> at(p, kRouteWarps);
    const T *row = logit_row<T>(p, at.s, at.present ? at.t : 0);
    float d[VPL], pr[VPL];
    RowStats st = {0.f, 1.f, false};
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.f;
    if (p.grad_loss || (softmax && !renorm)) {
        if (at.present) {
            load_row<T, VPL>(p, row, at.l, pr);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) pr[i] = -INFINITY;
        }
        st = softmax_row<LANES, VPL>(pr);
    }
    if (p.grad_loss) {
        const float gl = *p.grad_loss * p.inv_n, lse = st.lse();
        const float share = p.inv_n * ((float)p.E / (float)p.k);
        float f[VPL], dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = at.l * VPL + i;
            f[i] = e < p.E ? (float)p.counts[e] * share : 0.f;
            dot += pr[i] * f[i];
        }
        dot = row_sum<LANES>(dot);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            d[i] = pr[i] * ((f[i] - dot) * p.balance_coef + 2.0f * p.z_coef * lse) * gl;
    }
    if (p.grad_w) {
        int id[SLOTS];
        float g[SLOTS], c[SLOTS], v[SLOTS], dv[SLOTS], sum, dot = 0.f;
        bool mine[SLOTS];
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int j = q * LANES + at.l;
            id[q] = -1;
            g[q] = 0.f;
            c[q] = -INFINITY;
            if (at.present && j < p.k) {
                id[q] = p.idx[at.tok * p.k + j];
                if ((uint32_t)id[q] < (uint32_t)p.E) {
                    g[q] = p.grad_w[at.tok * p.k + j] * p.scale;
                    c[q] = sane_logit(to_f32(row[id[q]]));
                } else {
                    id[q] = -1;
                    if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
                }
            }
            mine[q] = id[q] >= 0;
        }
        chosen_scores<LANES, SLOTS>(softmax, renorm, st, c, mine, v, &sum);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) dot += g[q] * v[q];
        if (softmax || renorm) dot = row_sum<LANES>(dot);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            if (softmax) {
                dv[q] = renorm ? v[q] * (g[q] - dot) : v[q] * g[q];
            } else {
                float s = g[q];
                if (renorm) s = sum > 0.f ? (g[q] - dot / sum) / sum : 0.f;
                dv[q] = s * v[q] * (1.0f - v[q]);
            }
        }
        if (softmax && !renorm) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) d[i] -= pr[i] * dot;
        }
        float *r = rows[threadIdx.x / LANES];
#pragma unroll
        for (int i = 0; i < VPL; i += 4)
            *reinterpret_cast<float4 *>(r + at.l * VPL + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
        __syncwarp();
        // one lane a token: in order.  32: at once, unless an expert comes twice.
        bool twice = LANES < 32;
        if (LANES == 32) {
            const uint32_t same = __match_any_sync(0xffffffffu, mine[0] ? id[0] : -1 - (int)(threadIdx.x & 31));
            twice = __any_sync(0xffffffffu, (same & (same - 1u)) != 0);
        }
        if (!twice) {
            if (mine[0]) r[id[0]] += dv[0];
        } else {
            for (int j = 0; j < p.k; ++j) {
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    if (j == q * LANES + at.l && mine[q]) r[id[q]] += dv[q];
                __syncwarp();
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(r + at.l * VPL + i);
            d[i] = f.x;
            d[i + 1] = f.y;
            d[i + 2] = f.z;
            d[i + 3] = f.w;
        }
    }
    if (!at.in) return;
    if (!at.present) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = 0.f;
    }
    store_row<T, VPL>(p, static_cast<T *>(p.grad_logits) + at.tok * p.E, at.l, d);
}

// Losses, pass 1: every block sums softmax probabilities and lse^2 of its
// tokens (a lane's tokens in registers, then lanes and warps in order) and
// counts choices in shared memory.  Bound by instructions (about 100 a warp
// and token of 256 experts), so one block of 32 warps per SM.
template <typename T, int LANES, int VPL>
__global__ void __launch_bounds__(kLossWarps * 32) balance_partial_kernel(const RouteParams p, int tokens_per_warp) {
    extern __shared__ float sh[];                 // [kLossWarps][E + 1], then [E] counts
    constexpr int kTokens = 32 / LANES;
    int32_t *cnt = reinterpret_cast<int32_t *>(sh + kLossWarps * (p.E + 1));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    float acc[VPL], z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
    // this warp's tokens: a run of all ranks' tokens
    const int64_t total = (int64_t)p.W * p.T;
    const int64_t tok0 = ((int64_t)blockIdx.x * kLossWarps + warp) * tokens_per_warp;
    int s = (int)(tok0 / p.T), t0 = (int)(tok0 - (int64_t)s * p.T);
    for (int i0 = 0; i0 < tokens_per_warp; i0 += kTokens) {
        int t = t0 + i0 + lane / LANES, r = s;
        while (t >= p.T && r < p.W) {
            t -= p.T;
            ++r;
        }
        const bool present = i0 + lane / LANES < tokens_per_warp && tok0 + i0 + lane / LANES < total && t < p.nt.n[r];
        float x[VPL];
        if (present) {
            const int64_t tok = (int64_t)r * p.T + t;
            for (int j = l; j < p.k; j += LANES) {
                const int id = p.idx[tok * p.k + j];
                if ((uint32_t)id < (uint32_t)p.E) atomicAdd(&cnt[id], 1);
                else if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
            }
            load_row<T, VPL>(p, logit_row<T>(p, r, t), l, x);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) x[i] = -INFINITY;
        }
        const float lse = softmax_row<LANES, VPL>(x).lse();
        z += l == 0 ? lse * lse : 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += x[i];
    }
    // the warp's tokens of other lanes with the same experts
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    z = row_sum<32>(z);
    float *mine = sh + warp * (p.E + 1);
    if (lane < LANES) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (l * VPL + i < p.E) mine[l * VPL + i] = acc[i];
    }
    if (lane == 0) mine[p.E] = z;
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
        float sum = 0.f;
#pragma unroll 8
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
        balance = row_sum<32>(balance);
        z = row_sum<32>(z);
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

// Calls f(T(), Int<LANES>, Int<VPL>) for the logits' type and the row length.
template <int V> struct Int { static constexpr int value = V; };
template <typename T, typename F> void with_row(int E, F f) {
    if (E <= 8) f(T(), Int<1>(), Int<8>());
    else if (E <= 32) f(T(), Int<4>(), Int<8>());
    else if (E <= 64) f(T(), Int<8>(), Int<8>());
    else if (E <= 128) f(T(), Int<16>(), Int<8>());
    else if (E <= 256) f(T(), Int<32>(), Int<8>());
    else if (E <= 512) f(T(), Int<32>(), Int<16>());
    else f(T(), Int<32>(), Int<32>());
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
    const int size = d->dtype == EP_DT_FP32 ? 4 : 2;
    p->vec = d->num_experts % 8 == 0 && aligned(logits, 16) && d->row_stride * size % 16 == 0 &&
             p->rank_stride * size % 16 == 0;
    return true;
}

ep_status_t launched() { return cudaGetLastError() == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP; }

// One block per 4 warps of tokens of a rank.
template <int LANES> dim3 token_grid(const RouteParams &p) {
    constexpr int kTokens = kRouteWarps * (32 / LANES);
    return dim3((unsigned)((p.T + kTokens - 1) / kTokens), (unsigned)p.W);
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
    with_types(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        constexpr int kLanes = decltype(lanes)::value;
        route_kernel<decltype(type), kLanes, decltype(vpl)::value>
            <<<token_grid<kLanes>(p), kRouteWarps * 32, 0, st>>>(p, softmax, renorm);
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
    p.vec = p.vec && aligned(d_grad_logits, 16);
    with_types(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        constexpr int kLanes = decltype(lanes)::value;
        route_backward_kernel<decltype(type), kLanes, decltype(vpl)::value>
            <<<token_grid<kLanes>(p), kRouteWarps * 32, 0, st>>>(p, softmax, renorm);
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
    const size_t sh = ((size_t)kLossWarps * (p.E + 1) + p.E) * 4;    // 135 KB at most
    const int64_t warps = (int64_t)blocks * kLossWarps;
    const int per_warp = (int)(((int64_t)p.W * p.T + warps - 1) / warps);
    cudaError_t e = cudaSuccess;
    with_types(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        auto kernel = balance_partial_kernel<decltype(type), decltype(lanes)::value, decltype(vpl)::value>;
        if (sh > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e == cudaSuccess) kernel<<<blocks, kLossWarps * 32, sh, st>>>(p, per_warp);
    });
    if (e != cudaSuccess) return EP_ERR_GPU_OP;
    balance_final_kernel<<<1, 1024, 0, st>>>(p, blocks);
    return launched();
}

}  // extern "C"
