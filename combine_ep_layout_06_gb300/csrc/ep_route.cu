// Top-k routing, the balance and z losses, and the gradient of both by the
// router logits.
//
// A token's row of E logits lies in the registers of LANES neighbouring lanes,
// 8 to 32 neighbouring experts each, so that lane
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
constexpr int kSms = 152;        // of a GB300
// Warps of a block of the losses, one block per SM: what the registers and 48
// KB of shared memory allow (32768 x 256: 24 warps of 16 lanes a token 13.4 us
// a call, 16 warps 15.0).
__host__ __device__ constexpr int loss_warps(int lanes, int experts_per_lane) {
    return experts_per_lane == 8 ? 32 : experts_per_lane == 16 ? (lanes < 32 ? 24 : 16) : 8;
}

struct RouteParams {
    const void *logits;
    int64_t row_stride, rank_stride;
    TokenCounts nt;
    int W, T, E, k;
    bool vec;                // rows of logits (and of their gradient) in 16-byte pieces
    bool vec_e;              // per-expert inputs in 16-byte pieces
    int rounds;              // backward: runs of tokens of a warp
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
    float *part;             // loss: [clusters][E + 1] partial sums
    int32_t *part_count;     // loss: [clusters][E]
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
    return fminf(fmaxf(v, -INFINITY), FLT_MAX);     // fmaxf drops a NaN
}

// Unsigned integers in the order of the floats (-0 counts as +0).  Every
// value, -inf included, maps above 0, which marks "no candidate".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Reductions over the LANES lanes of a token.
template <int LANES> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES> __device__ __forceinline__ float row_max(float v) {
    if constexpr (LANES == 32) {
        float r;
        asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    }
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
template <int LANES> __device__ __forceinline__ uint32_t row_min(uint32_t v) {
    if constexpr (LANES == 32) return __reduce_min_sync(0xffffffffu, v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
constexpr float kLog2e = 1.44269504088896341f;
// 2^v within 2^-22, results below 2^-126 are 0.
__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// exp of a difference of logits (<= 0): relative error below 2^-22 + |d| 2^-23.
// Terms with a large |d| weigh exp(d) of the largest one.
__device__ __forceinline__ float exp_diff(float d) { return exp2_approx(d * kLog2e); }

template <typename T>
__device__ __forceinline__ const T *logit_row(const RouteParams &p, int s, int t) {
    return static_cast<const T *>(p.logits) + s * p.rank_stride + t * p.row_stride;
}

// Experts l * VPL .. l * VPL + VPL - 1 of a row, as they lie in memory, and
// as fp32 with -inf past the last expert.  Two steps, so that the next row's
// load can be on its way while a row is worked on.
template <typename T, int VPL> struct RawRow {
    static constexpr int kPer = 16 / sizeof(T);
    uint4 v[VPL / kPer];

    __device__ __forceinline__ void load(const RouteParams &p, const T *row, int l, bool present) {
        if (!present) {
            const T shut = from_f32<T>(-INFINITY);
            T *s = reinterpret_cast<T *>(v);
#pragma unroll
            for (int i = 0; i < VPL; ++i) s[i] = shut;
        } else if (p.vec) {  // E is a multiple of 8: every piece is inside or outside
#pragma unroll
            for (int c = 0; c < VPL / kPer; ++c)
                if (l * VPL + c * kPer < p.E) v[c] = ld_stream16(row + l * VPL + c * kPer);
        } else {
            T *s = reinterpret_cast<T *>(v);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (l * VPL + i < p.E) s[i] = row[l * VPL + i];
        }
    }
    __device__ __forceinline__ void values(const RouteParams &p, int l, float *x) const {
        const T *s = reinterpret_cast<const T *>(v);
        if ((l + 1) * VPL <= p.E) {
            float odd = 0.f;                     // a NaN as soon as one logit is not finite
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                x[i] = to_f32(s[i]);
                odd = fmaf(x[i], 0.f, odd);
            }
            if (odd != odd) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) x[i] = sane_logit(x[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) x[i] = l * VPL + i < p.E ? sane_logit(to_f32(s[i])) : -INFINITY;
        }
    }
};
// Two values as they lie in memory, in 32 bits (16-bit types).
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(__half, float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T, int VPL>
__device__ __forceinline__ void store_row(const RouteParams &p, T *row, int l, const float *d) {
    if (p.vec) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                if (l * VPL + c < p.E)
                    *reinterpret_cast<float4 *>(row + l * VPL + c) = make_float4(d[c], d[c + 1], d[c + 2], d[c + 3]);
        } else {
#pragma unroll
            for (int c = 0; c < VPL; c += 8)
                if (l * VPL + c < p.E)
                    *reinterpret_cast<uint4 *>(row + l * VPL + c) =
                        make_uint4(pack2(T(), d[c], d[c + 1]), pack2(T(), d[c + 2], d[c + 3]),
                                   pack2(T(), d[c + 4], d[c + 5]), pack2(T(), d[c + 6], d[c + 7]));
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
    float m, scaled, inv_sum;    // scaled: m log2(e)
    bool open;                   // some expert is open

    // With |m| <= 2^16, exp(x - m) is taken as 2^(x log2(e) - scaled), one
    // multiply-add.  What rounding m log2(e) to `scaled` left out, 2^-8 at most
    // there, is in every term's exponent: a factor that probabilities share, and
    // in lse() an error of 2^-24 |m|.  It grows with |m| (512 at 2^33: sums of 0
    // or infinity), so rows further out subtract first, exact at the maximum.
    __device__ bool near() const { return fabsf(m) <= 65536.f; }
    __device__ float prob(float x) const {
        if (!open) return 0.f;
        return (near() ? exp2_approx(fmaf(x, kLog2e, -scaled)) : exp_diff(x - m)) * inv_sum;
    }
    // error of the logarithm: 2^-21.4 where the sum is below 2, else 3 units in the last place of a value of 7 at most
    __device__ float lse() const { return open ? m - __logf(inv_sum) : 0.f; }
};

// Statistics of a token's row but for the sum; exp(x - max) in place of x (all
// 0 when no expert is open).
template <int LANES, int VPL>
__device__ __forceinline__ RowStats row_exps(float *x) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = row_max<LANES>(m);
    RowStats st = {m, 0.f, 1.f, m > -INFINITY};
    if (!st.open) st.m = 0.f;                // every exponential is then 0
    st.scaled = st.m * kLog2e;
    if (st.near()) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = exp2_approx(fmaf(x[i], kLog2e, -st.scaled));
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = exp_diff(x[i] - st.m);
    }
    return st;
}
// Of an open row, whose largest term is 1 within 2^-8: 0.99 <= sum <= 1.01 E.
__device__ __forceinline__ float inverse(const RowStats &st, float sum) {
    return st.open ? __fdividef(1.0f, sum) : 1.f;
}
template <int VPL> __device__ __forceinline__ float lane_sum(const float *x) {
    float sum = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) sum += x[i];
    return sum;
}
// The whole: exponentials in place of x, their inverse sum in the statistics.
template <int LANES, int VPL>
__device__ __forceinline__ RowStats softmax_row(float *x) {
    RowStats st = row_exps<LANES, VPL>(x);
    st.inv_sum = inverse(st, row_sum<LANES>(lane_sum<VPL>(x)));
    return st;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A token's place: lane l of its LANES, token t of rank blockIdx.y.  A warp
// takes `rounds` runs of 32 / LANES tokens; this is the first.
template <int LANES> struct Place {
    static constexpr int kTokens = 32 / LANES;           // of a warp and round
    int l, s, t;
    int64_t tok;
    bool in, present;
    __device__ Place(const RouteParams &p, int warps, int rounds) {
        const int lane = threadIdx.x & 31;
        l = lane % LANES;
        s = blockIdx.y;
        t = (blockIdx.x * warps + (threadIdx.x >> 5)) * rounds * kTokens + lane / LANES;
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
// renormalising divides by.  Where that sum is below 2^-32 the scores are e^c
// within 2^-32 of themselves, down to below fp32's range, and only their ratios
// matter: they are taken relative to the largest instead (the return value).  A
// token whose largest is below e^-745, the least that 64 bits hold (all at a
// mask's fill value), has no score.
template <int LANES, int SLOTS>
__device__ __forceinline__ bool chosen_scores(bool softmax, bool renorm, const RowStats &st, const float *c,
                                              const bool *mine, float *v, float *sum) {
    bool relative = false;
    *sum = 0.f;
    if (softmax && renorm) {
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) m = fmaxf(m, mine[q] ? c[q] : -INFINITY);
        m = row_max<LANES>(m);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            v[q] = mine[q] && m > -INFINITY ? exp_diff(c[q] - m) : 0.f;
            *sum += v[q];
        }
        *sum = row_sum<LANES>(*sum);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) v[q] = *sum > 0.f ? __fdividef(v[q], *sum) : 0.f;     // 1 <= sum <= k
    } else if (softmax) {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) v[q] = mine[q] ? st.prob(c[q]) : 0.f;
    } else {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            v[q] = mine[q] ? sigmoid(c[q]) : 0.f;
            *sum += v[q];
        }
        if (renorm) {
            *sum = row_sum<LANES>(*sum);
            const bool low = *sum < 2.3283064e-10f;      // 2^-32
            if (__any_sync(0xffffffffu, low)) {
                float m = -INFINITY, total = 0.f;
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) m = fmaxf(m, mine[q] ? c[q] : -INFINITY);
                m = row_max<LANES>(m);
                relative = low && m > -745.f;
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) {
                    if (low) v[q] = relative && mine[q] ? exp_diff(c[q] - m) : 0.f;
                    total += v[q];
                }
                total = row_sum<LANES>(total);
                if (low) *sum = total;
            }
        }
    }
    return relative;
}

// The scores, each in kernels of its own; and a gradient of the loss alone.
enum Part { kLossOnly, kSoftmaxChosen, kSoftmaxAll, kSigmoid };

template <typename T, int LANES, int VPL, Part PART>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p, bool renorm) {
    constexpr int SLOTS = slots_of<LANES>();
    const Place<LANES> at(p, kRouteWarps, 1);
    grid_dependency_wait();
    grid_dependents_may_launch();     // the next kernel may count on all before this one
    if (!__any_sync(0xffffffffu, at.present)) {          // nobody here
        for (int j = at.l; at.in && j < p.k; j += LANES) {
            p.w[at.tok * p.k + j] = 0.f;
            p.idx_out[at.tok * p.k + j] = -1;
        }
        return;
    }
    const T *row = logit_row<T>(p, at.s, at.present ? at.t : 0);
    RawRow<T, VPL> raw;
    raw.load(p, row, at.l, at.present);
    float x[VPL], y[VPL];
    const int e0 = at.l * VPL;
    if (p.bias && p.vec_e) {          // E is a multiple of 8: every piece is inside or outside
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
            float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e0 + i < p.E) b = *reinterpret_cast<const float4 *>(p.bias + e0 + i);
            y[i] = b.x; y[i + 1] = b.y; y[i + 2] = b.z; y[i + 3] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) y[i] = p.bias && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
    }
    raw.values(p, at.l, x);
    // this lane's best and second best key: the larger one, or the earlier expert
    uint32_t key[VPL], best = 0, second = 0;
    int be = 0, se = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = order_key(x[i] + y[i]);
    if (e0 + VPL > p.E) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e0 + i >= p.E) key[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool first = key[i] > best, next = key[i] > second;
        second = max(second, min(best, key[i]));
        se = first ? be : next ? i : se;
        best = max(best, key[i]);
        be = first ? i : be;
    }
    int id[SLOTS];
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) id[q] = 0;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t top = row_max_key<LANES>(best);
        const int mine = e0 + be;                        // of equal keys the first expert's
        const int e = (int)row_min<LANES>(best == top ? (uint32_t)mine : 0xffffffffu);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q)
            if (j == q * LANES + at.l) id[q] = e;
        bool again = false;
        if (e == mine && best == top) {
            again = second == 0 && j + 1 < p.k;
            if (!again) {
                best = second;
                be = se;
                second = 0;
            }
        }
        if (__any_sync(0xffffffffu, again)) {
            // both keys are taken: the best one after the one taken last (equal
            // keys in the order of the experts)
            if (again) {
                const uint32_t last = best;
                const int le = be;
                best = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    const bool open = key[i] < last || (key[i] == last && i > le);
                    if (open && key[i] > best) {
                        best = key[i];
                        be = i;
                    }
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
    RowStats st = {0.f, 0.f, 1.f, false};
    if (PART == kSoftmaxAll) st = softmax_row<LANES, VPL>(x);
    chosen_scores<LANES, SLOTS>(PART != kSigmoid, PART == kSoftmaxChosen || (PART == kSigmoid && renorm), st, c, mine, v,
                                &sum);
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
        const int j = q * LANES + at.l;
        if (PART == kSigmoid && renorm) v[q] = sum > 0.f ? v[q] / sum : 0.f;
        if (at.in && j < p.k) {
            p.w[at.tok * p.k + j] = mine[q] ? v[q] * p.scale : 0.f;
            p.idx_out[at.tok * p.k + j] = mine[q] ? id[q] : -1;
        }
    }
}

// The weights' gradient is nonzero at the chosen experts (and, for a softmax
// that is not renormalised, dense): the row meets in shared memory, where the
// chosen experts' terms are added to the dense part, one choice after the
// other where an expert was chosen twice.  The experts' loads, the same for
// all tokens, stay in registers over a warp's tokens.
template <typename T, int LANES, int VPL, Part PART>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const RouteParams p, bool renorm) {
    constexpr bool WEIGHTS = PART != kLossOnly, softmax = PART != kSigmoid;
    constexpr int SLOTS = slots_of<LANES>();
    constexpr int kTokens = 32 / LANES, kRow = LANES * VPL;
    __shared__ __align__(16) float rows[WEIGHTS ? kRouteWarps * kTokens : 1][kRow + 4];
    const bool dense = PART == kLossOnly || PART == kSoftmaxAll || p.grad_loss;
    const int e0 = (int)(threadIdx.x & 31) % LANES * VPL;
    float f[VPL], gl = 0.f;
    grid_dependency_wait();
    grid_dependents_may_launch();     // the next kernel may count on all before this one
    if (!WEIGHTS || p.grad_loss) {
        gl = *p.grad_loss * p.inv_n;
        const float share = p.inv_n * ((float)p.E / (float)p.k) * p.balance_coef;
#pragma unroll
        for (int i = 0; i < VPL; ++i) f[i] = e0 + i < p.E ? (float)p.counts[e0 + i] * share : 0.f;
    }
    // one round ahead: the rows, the choices and their weights' gradients
    const Place<LANES> at(p, kRouteWarps, p.rounds);
    const int present = p.nt.n[at.s];
    const T *row = logit_row<T>(p, at.s, 0) + at.t * p.row_stride;
    T *out = static_cast<T *>(p.grad_logits) + at.tok * p.E;
    const int32_t *idx = p.idx + at.tok * p.k;
    const float *gw = p.grad_w + at.tok * p.k;
    RawRow<T, VPL> raw;
    int id_next[SLOTS];
    float g_next[SLOTS];
    auto fetch = [&](int t) {                 // token t of the rank, at row, idx and gw
        if (dense) raw.load(p, row, at.l, t < present);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int j = q * LANES + at.l;
            const bool mine = WEIGHTS && t < present && j < p.k;
            id_next[q] = mine ? idx[j] : 0;
            g_next[q] = mine ? gw[j] : 0.f;
        }
    };
    int t = at.t;
    fetch(t);
    for (int round = 0; round < p.rounds; ++round, t += kTokens, out += (int64_t)kTokens * p.E) {
        float d[VPL], pr[VPL], g[SLOTS];
        int id[SLOTS];
        const T *here = row;
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = 0.f;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            id[q] = id_next[q];
            g[q] = g_next[q] * p.scale;
        }
        if (dense) raw.values(p, at.l, pr);
        if (round + 1 < p.rounds) {
            row += kTokens * p.row_stride;
            idx += kTokens * p.k;
            gw += kTokens * p.k;
            fetch(t + kTokens);
        }
        if (__any_sync(0xffffffffu, t < present)) {
            const bool is = t < present;
            RowStats st = {0.f, 0.f, 1.f, false};
            float *r = rows[WEIGHTS ? threadIdx.x / LANES : 0];
            float c[SLOTS];
            bool mine[SLOTS];
#pragma unroll
            for (int q = 0; q < SLOTS; ++q) {
                mine[q] = WEIGHTS && is && q * LANES + at.l < p.k;
                if (mine[q] && (uint32_t)id[q] >= (uint32_t)p.E) {
                    mine[q] = false;
                    g[q] = 0.f;
                    if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
                }
                c[q] = -INFINITY;
            }
            // the chosen logits: from the row where it is at hand
            if (WEIGHTS && dense) {
#pragma unroll
                for (int i = 0; i < VPL; i += 4)
                    *reinterpret_cast<float4 *>(r + e0 + i) = make_float4(pr[i], pr[i + 1], pr[i + 2], pr[i + 3]);
                __syncwarp();
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    if (mine[q]) c[q] = r[id[q]];
                __syncwarp();
            } else if (WEIGHTS) {
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    if (mine[q]) c[q] = sane_logit(to_f32(here[id[q]]));
            }
            if (!WEIGHTS || p.grad_loss) {
                // p (f - <p, f> + 2 z lse), with p = exp / sum: both sums at once
                st = row_exps<LANES, VPL>(pr);
                float sum = lane_sum<VPL>(pr), dot = 0.f;
#pragma unroll
                for (int i = 0; i < VPL; ++i) dot = fmaf(pr[i], f[i], dot);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                st.inv_sum = inverse(st, sum);
                const float shift = 2.0f * p.z_coef * st.lse() - dot * st.inv_sum, factor = st.inv_sum * gl;
#pragma unroll
                for (int i = 0; i < VPL; ++i) d[i] = pr[i] * fmaf(f[i], factor, shift * factor);
            } else if (dense) {
                st = softmax_row<LANES, VPL>(pr);
            }
            if constexpr (WEIGHTS) {
                float v[SLOTS], dv[SLOTS], sum, dot = 0.f;
                const bool relative = chosen_scores<LANES, SLOTS>(
                    softmax, PART == kSoftmaxChosen || (PART == kSigmoid && renorm), st, c, mine, v, &sum);
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) dot += g[q] * v[q];
                if (PART != kSigmoid || renorm) dot = row_sum<LANES>(dot);
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) {
                    if (softmax) {
                        dv[q] = PART == kSoftmaxChosen ? v[q] * (g[q] - dot) : v[q] * g[q];
                    } else {
                        float s = g[q];
                        if (renorm) s = sum > 0.f ? (g[q] - dot / sum) / sum : 0.f;
                        dv[q] = s * v[q] * (relative ? 1.0f : 1.0f - v[q]);
                    }
                }
                if (PART == kSoftmaxAll) {
                    const float slope = dot * st.inv_sum;
#pragma unroll
                    for (int i = 0; i < VPL; ++i) d[i] = fmaf(-pr[i], slope, d[i]);
                }
                // several choices a lane: in order.  One choice a lane: at once,
                // unless two lanes find each other at an expert's place.
                bool twice = p.k > LANES;
                if (!twice) {
                    int *mark = reinterpret_cast<int *>(r);
                    if (mine[0]) mark[id[0]] = at.l;
                    __syncwarp();
                    twice = __any_sync(0xffffffffu, mine[0] && mark[id[0]] != at.l);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < VPL; i += 4)
                    *reinterpret_cast<float4 *>(r + e0 + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                __syncwarp();
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
                    const float4 b = *reinterpret_cast<const float4 *>(r + e0 + i);
                    d[i] = b.x; d[i + 1] = b.y; d[i + 2] = b.z; d[i + 3] = b.w;
                }
                __syncwarp();
            }
            if (!is) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) d[i] = 0.f;
            }
        }
        if (t < p.T) store_row<T, VPL>(p, out, at.l, d);
    }
}

// Without the z loss its size, past fp32 for |lse| > 2^64, has no part in the
// total: 0 * infinity would be NaN.
__device__ __forceinline__ void store_loss(const RouteParams &p, float balance, float z) {
    p.loss[0] = p.balance_coef * balance + (p.z_coef != 0.f ? p.z_coef * z : 0.f);
    p.loss[1] = balance;
    p.loss[2] = z;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(addr), "f"(v) : "memory");
}

// Losses, pass 1: every block sums softmax probabilities and lse^2 of its
// tokens (a lane's tokens in registers, then lanes and warps in order) and
// counts choices in shared memory; the 4 blocks of a cluster join their sums,
// each a quarter of the experts, through distributed shared memory.  Few tokens
// are one cluster's, which also finishes the losses.  Bound by instructions and
// the rows' latency: one block per SM, each lane with its next row on the way.
constexpr int kLossCluster = 4;

template <typename T, int LANES, int VPL>
__global__ void __cluster_dims__(kLossCluster, 1, 1) __launch_bounds__(loss_warps(LANES, VPL) * 32)
    balance_partial_kernel(const RouteParams p, int tokens_per_warp) {
    extern __shared__ float sh[];                 // [kLossWarps][E + 1], then [E] counts
    constexpr int kTokens = 32 / LANES, kLossWarps = loss_warps(LANES, VPL), SLOTS = slots_of<LANES>();
    __shared__ float shares[32], joined[kLossCluster + 1];   // of the loss by warp, by block; z
    int32_t *cnt = reinterpret_cast<int32_t *>(sh + kLossWarps * (p.E + 1));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    grid_dependency_wait();
    grid_dependents_may_launch();     // the next kernel may count on all before this one
    __syncthreads();
    float acc[VPL], z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
    // this warp's tokens: a run of all ranks' tokens
    const int64_t total = (int64_t)p.W * p.T;
    const int64_t tok0 = ((int64_t)blockIdx.x * kLossWarps + warp) * tokens_per_warp;
    int r = (int)(tok0 / p.T), t = (int)(tok0 - (int64_t)r * p.T) + lane / LANES, i = lane / LANES;
    RawRow<T, VPL> raw, ahead;
    int ids[SLOTS];                              // -1: no choice of a present token here
    auto fetch = [&] {                           // the row of this lane's token i; then on to the next
        while (t >= p.T && r < p.W) {
            t -= p.T;
            ++r;
        }
        const bool present = i < tokens_per_warp && tok0 + i < total && t < p.nt.n[r];
        ahead.load(p, present ? logit_row<T>(p, r, t) : nullptr, l, present);
        const int64_t first = ((int64_t)r * p.T + t) * p.k;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int j = q * LANES + l;
            ids[q] = -1;
            if (present && j < p.k) {
                ids[q] = p.idx[first + j];
                if ((uint32_t)ids[q] >= (uint32_t)p.E) ids[q] = p.E;
            }
        }
        t += kTokens;
        i += kTokens;
    };
    fetch();
    for (int i0 = 0; i0 < tokens_per_warp; i0 += kTokens) {
        raw = ahead;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            if (ids[q] < 0) continue;
            if (ids[q] < p.E) atomicAdd(&cnt[ids[q]], 1);
            else if (p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
        }
        if (i0 + kTokens < tokens_per_warp) fetch();
        float x[VPL];
        raw.values(p, l, x);
        const RowStats st = softmax_row<LANES, VPL>(x);
        const float lse = st.lse();
        z += l == 0 ? lse * lse : 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) acc[j] = fmaf(x[j], st.inv_sum, acc[j]);
    }
    // the warp's tokens of other lanes with the same experts
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    }
    z = row_sum<32>(z);
    float *mine = sh + warp * (p.E + 1);
    if (lane < LANES) {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (l * VPL + j < p.E) mine[l * VPL + j] = acc[j];
    }
    if (lane == 0) mine[p.E] = z;
    __syncthreads();
    // the block's sums, in the first warp's place
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
        float sum = 0.f;
#pragma unroll 8
        for (int w = 0; w < kLossWarps; ++w) sum += sh[w * (p.E + 1) + e];
        sh[e] = sum;
    }
    __syncwarp();
    cluster_sync();
    const uint32_t rank = cluster_rank();
    const int per = (p.E + kLossCluster) / kLossCluster;     // of E + 1 sums
    const int e1 = min(p.E + 1, (int)(rank + 1) * per);
    const bool whole = gridDim.x == kLossCluster;
    const int64_t part = blockIdx.x / kLossCluster;
    float balance = 0.f;
    for (int e = rank * per + threadIdx.x; e < e1; e += blockDim.x) {
        float sum = 0.f;
        int32_t c = 0;
#pragma unroll
        for (uint32_t b = 0; b < kLossCluster; ++b) {
            sum += ld_cluster_f32(in_cta(smem_u32(sh + e), b));
            if (e < p.E) c += ld_cluster_s32(in_cta(smem_u32(cnt + e), b));
        }
        if (!whole) {
            p.part[part * (p.E + 1) + e] = sum;
            if (e < p.E) p.part_count[part * p.E + e] = c;
        } else if (e < p.E) {
            sum *= p.inv_n;
            p.probs[e] = sum;
            p.counts_out[e] = c;
            balance += (float)c * (p.inv_n * ((float)p.E / (float)p.k)) * sum;
        } else {
            st_cluster_f32(in_cta(smem_u32(joined + kLossCluster), 0), sum * p.inv_n);
        }
    }
    if (whole) {
        __syncwarp();
        balance = row_sum<32>(balance);
        if (lane == 0) shares[warp] = balance;
        __syncthreads();
        if (warp == 0) {
            balance = row_sum<32>(lane < kLossWarps ? shares[lane] : 0.f);
            if (lane == 0) st_cluster_f32(in_cta(smem_u32(joined + rank), 0), balance);
        }
    }
    __syncwarp();
    cluster_sync();                              // no block's shared memory is read any more
    if (whole && rank == 0 && threadIdx.x == 0) {
        balance = 0.f;
        for (int b = 0; b < kLossCluster; ++b) balance += joined[b];
        store_loss(p, balance, joined[kLossCluster]);
    }
}

// Losses, pass 2: one cluster of 8 blocks joins the parts, each block an
// eighth of the experts (128 at most) by 8 slices of the parts, sums in order;
// the loss's shares meet in the first block.
constexpr int kFinalCluster = 8, kFinalColumns = EP_MAX_ROUTE_EXPERTS / kFinalCluster;

__global__ void __cluster_dims__(kFinalCluster, 1, 1) __launch_bounds__(1024)
    balance_final_kernel(const RouteParams p, int parts) {
    constexpr int kSlices = 1024 / kFinalColumns;
    __shared__ float sh[kSlices][kFinalColumns], shares[kFinalColumns / 32], joined[kFinalCluster + 1];
    __shared__ int32_t sc[kSlices][kFinalColumns];
    const uint32_t rank = cluster_rank();
    const int column = threadIdx.x % kFinalColumns, slice = threadIdx.x / kFinalColumns;
    const int per = (p.E + kFinalCluster - 1) / kFinalCluster;
    const int e = column < per && (int)rank * per + column < p.E ? (int)rank * per + column : -1;
    cluster_sync();              // all 8 blocks run: their shared memory may be written
    grid_dependency_wait();
    float sum = 0.f, z = 0.f;
    int32_t c = 0;
    if (e >= 0) {
#pragma unroll 5
        for (int b = slice; b < parts; b += kSlices) {
            sum += p.part[(int64_t)b * (p.E + 1) + e];
            c += p.part_count[(int64_t)b * p.E + e];
        }
    }
    if (rank == 0 && threadIdx.x < 32) {
        for (int b = threadIdx.x; b < parts; b += 32) z += p.part[(int64_t)b * (p.E + 1) + p.E];
        z = row_sum<32>(z) * p.inv_n;
    }
    sh[slice][column] = sum;
    sc[slice][column] = c;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
        for (int s = 1; s < kSlices; ++s) {
            sum += sh[s][column];
            c += sc[s][column];
        }
        float balance = 0.f;
        if (e >= 0) {
            sum *= p.inv_n;
            p.probs[e] = sum;
            p.counts_out[e] = c;
            balance = (float)c * (p.inv_n * ((float)p.E / (float)p.k)) * sum;
        }
        balance = row_sum<32>(balance);
        if (threadIdx.x % 32 == 0) shares[threadIdx.x / 32] = balance;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float balance = 0.f;
        for (int w = 0; w < kFinalColumns / 32; ++w) balance += shares[w];
        st_cluster_f32(in_cta(smem_u32(joined + rank), 0), balance);
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        float balance = 0.f;
        for (int b = 0; b < kFinalCluster; ++b) balance += joined[b];
        store_loss(p, balance, z);
    }
}

// Clusters of the losses' first pass.  One, without a second pass, up to 2^17
// logits; else one per 128 tokens, up to the 36 that run at a time (a block per
// SM: what cudaOccupancyMaxActiveClusters gives on the 152 SMs).
int loss_clusters(const ep_route_desc_t &d) {
    const int64_t tokens = (int64_t)d.world_size * d.tokens;
    const int64_t want = tokens * d.num_experts <= 1 << 17 ? 1 : (tokens + 127) / 128;
    return (int)(want < 36 ? want : 36);
}

// Calls f(T(), Int<LANES>, Int<VPL>) for the logits' type and the row length.
// Reductions cost a warp the same for one token or several, so for the losses
// (WIDE) a lane takes 16 experts of a long row (32768 x 256: 13.7 against 15.0
// us a call); top-k, which searches a lane's experts, and the gradient, which needs the
// registers, take 8 (against 16: top-k 14.5 and 15.4 us, gradient of the loss
// alone 9.1 and 10.1, with the weights' 15.7 and 24.3).
template <int V> struct Int { static constexpr int value = V; };
template <bool WIDE, typename T, typename F> void with_row(int E, F f) {
    if (E <= 8) f(T(), Int<1>(), Int<8>());
    else if (E <= 32) f(T(), Int<4>(), Int<8>());
    else if (E <= 64) f(T(), Int<8>(), Int<8>());
    else if (E <= 128) f(T(), Int<WIDE ? 8 : 16>(), Int<WIDE ? 16 : 8>());
    else if (E <= 256) f(T(), Int<WIDE ? 16 : 32>(), Int<WIDE ? 16 : 8>());
    else if (E <= 512) f(T(), Int<32>(), Int<16>());
    else f(T(), Int<32>(), Int<32>());
}
template <bool WIDE, typename F> void with_types(int dtype, int E, F f) {
    if (dtype == EP_DT_BF16) with_row<WIDE, __nv_bfloat16>(E, f);
    else if (dtype == EP_DT_FP16) with_row<WIDE, __half>(E, f);
    else with_row<WIDE, float>(E, f);
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

// Launches as a programmatic dependent of the kernel before where the kernel
// is long enough to gain by it (32768 x 256: top-k 14.5 instead of 16.5 us a
// call, both gradients 15.7 instead of 17.3; 131072 x 8 the same either way); a
// one-token call's time goes by the host, whose launch it makes a microsecond
// longer.
template <typename... Params, typename... Args>
cudaError_t launch(const RouteParams &p, void (*kernel)(Params...), dim3 blocks, unsigned threads, size_t dyn,
                   cudaStream_t st, Args &&...args) {
    if ((int64_t)p.W * p.T * p.E >= 1 << 18)
        return launch_after_previous(kernel, blocks, threads, dyn, st, static_cast<Args &&>(args)...);
    kernel<<<blocks, threads, dyn, st>>>(static_cast<Args &&>(args)...);
    return cudaGetLastError();
}

// One block per 4 warps of tokens of a rank.
template <int LANES> dim3 token_grid(const RouteParams &p, int rounds) {
    const int tokens = kRouteWarps * (32 / LANES) * rounds;
    return dim3((unsigned)((p.T + tokens - 1) / tokens), (unsigned)p.W);
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
    p.vec_e = p.E % 8 == 0 && aligned(d_bias, 16);
    p.w = d_w;
    p.idx_out = d_idx;
    const bool softmax = d->score == EP_SCORE_SOFTMAX, renorm = d->renormalize != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    with_types<false>(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        constexpr int kLanes = decltype(lanes)::value;
        constexpr int kVpl = decltype(vpl)::value;
        using T = decltype(type);
        e = launch(p, !softmax ? route_kernel<T, kLanes, kVpl, kSigmoid>
                      : renorm ? route_kernel<T, kLanes, kVpl, kSoftmaxChosen>
                               : route_kernel<T, kLanes, kVpl, kSoftmaxAll>,
                   token_grid<kLanes>(p, 1), kRouteWarps * 32, 0, st, p, renorm);
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
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
    cudaError_t e = cudaSuccess;
    p.vec = p.vec && aligned(d_grad_logits, 16);
    with_types<false>(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        constexpr int kLanes = decltype(lanes)::value;
        // enough warps for all SMs (32 each) before a warp takes a second run
        constexpr int64_t kFull = kSms * 32;
        const int64_t runs = (int64_t)p.W * p.T * kLanes / 32;
        p.rounds = (int)(runs < kFull ? 1 : runs < 4 * kFull ? runs / kFull : 4);
        constexpr int kVpl = decltype(vpl)::value;
        using T = decltype(type);
        e = launch(p, !d_grad_w          ? route_backward_kernel<T, kLanes, kVpl, kLossOnly>
                      : !softmax         ? route_backward_kernel<T, kLanes, kVpl, kSigmoid>
                      : renorm           ? route_backward_kernel<T, kLanes, kVpl, kSoftmaxChosen>
                                         : route_backward_kernel<T, kLanes, kVpl, kSoftmaxAll>,
                   token_grid<kLanes>(p, p.rounds), kRouteWarps * 32, 0, st, p, renorm);
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

ep_status_t ep_balance_loss_workspace(const ep_route_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    // parts of the sums and counts
    *bytes = (size_t)loss_clusters(*d) * (2 * (size_t)d->num_experts + 1) * 4;
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
    const int clusters = loss_clusters(*d);
    p.idx = d_idx;
    p.loss = d_loss;
    p.counts_out = d_counts;
    p.probs = d_probs;
    p.error = d_error;
    p.part = static_cast<float *>(d_workspace);
    p.part_count = reinterpret_cast<int32_t *>(p.part + (size_t)clusters * (p.E + 1));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    with_types<true>(d->dtype, p.E, [&](auto type, auto lanes, auto vpl) {
        constexpr int kWarps = loss_warps(decltype(lanes)::value, decltype(vpl)::value);
        const size_t sh = ((size_t)kWarps * (p.E + 1) + p.E) * 4;    // 37 KB at most
        const int64_t warps = (int64_t)clusters * kLossCluster * kWarps;
        const int per_warp = (int)(((int64_t)p.W * p.T + warps - 1) / warps);
        e = launch_after_previous(
            balance_partial_kernel<decltype(type), decltype(lanes)::value, decltype(vpl)::value>,
            clusters * kLossCluster, kWarps * 32, sh, st, p, per_warp);
    });
    if (e != cudaSuccess) return EP_ERR_GPU_OP;
    if (clusters == 1) return EP_SUCCESS;
    e = launch_after_previous(balance_final_kernel, kFinalCluster, 1024, 0, st, p, clusters);
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

}  // extern "C"
