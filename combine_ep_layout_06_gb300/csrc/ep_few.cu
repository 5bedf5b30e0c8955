// The experts of a few tokens: both products and the weighted sum, in two
// kernels.
//
//   up    h[row][f] = act(x[t] up_e^T + b),  a row for every (expert, token) that meet
//   down  out[t] = residual[t] + sum over e of w[t][e] (h[row] down_e^T + c)
//
// The weights of the experts that were chosen are read once and everything
// else is small, so the kernels are built to keep memory busy.  The weights are the
// 128-wide operand of the matrix instructions and the tokens the other
// (16 columns at least), so that few tokens cost narrow instructions.  One
// CTA per SM: two warps in turn load 128-deep slices of weights and tokens by TMA
// into a ring in shared memory, tile after tile without a pause; one thread issues
// the instructions; four warps finish one accumulator while the other fills.
//
// Up takes all tokens as columns and keeps those that chose the expert: no
// gather.  Down has a CTA go through all experts for its outputs, which it sums in
// shared memory in ascending order of experts: no atomics, no partial outputs.
// h stands grouped by expert, in two 16-bit halves (a value and what its rounding
// left) that are columns of their own, because 16 columns cost what 8 do.
//
// Down is launched programmatically: its CTAs start as up's end, and fill their
// rings with weights before they wait for h.
#include <cuda.h>

#include "ep_rows.cuh"
#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kSlice = 128;                  // k of a slice: two halves of 64, 128 bytes each
constexpr int kMaxStages = 12;
constexpr int kLoaders = 2, kFinishers = 4;    // warps
constexpr int kMostRows = 32;                // of h in an accumulator of down
constexpr int kThreads = (kLoaders + 1 + kFinishers) * 32;
constexpr int kSmemMost = 227 * 1024 - 1024; // of a CTA, less what is static

struct FewParams {
    int T, E, k, M, K;           // M: outputs of this product (gated: of a half); K: its depth
    int act, rows;               // rows of weights a tile
    int box;                     // up: token rows a copy brings
    int stages, stage_bytes, columns;
    int split;                   // down: CTAs that share a tile, each a part of K
    int off_acc, off_mask, off_weight, off_first, off_list, off_token;    // in shared memory, after the ring
    const float *w;
    const int32_t *idx;
    const void *bias;            // [E][features]
    void *h;                     // [2][T * k][F]
    int64_t h_half;
    ep_rows_t residual, out;
    uint32_t *error;
};
struct FewWork {
    CUtensorMap a, b;
    FewParams p;
};

struct __align__(8) FewBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], joined, drained;
    uint32_t tmem;
    int present;
    Watch watch;
};

// Which tokens chose which expert.  Experts that were chosen stand in `list`, in
// ascending order; the rows of expert e are first[e] and on, its tokens in
// order.
struct Plan {
    unsigned long long *mask;    // [E] tokens
    float *weight;               // [rows], down only
    uint16_t *first, *list;      // [E]
    uint8_t *token;              // [rows], down only
    int present;
};

__device__ __forceinline__ int bits_below(unsigned long long mask, int t) { return __popcll(mask & ((1ull << t) - 1)); }

template <bool DOWN> __device__ void make_plan(const FewParams &p, unsigned char *smem, int *present, Plan *plan) {
    plan->mask = reinterpret_cast<unsigned long long *>(smem + p.off_mask);
    plan->weight = reinterpret_cast<float *>(smem + p.off_weight);
    plan->first = reinterpret_cast<uint16_t *>(smem + p.off_first);
    plan->list = reinterpret_cast<uint16_t *>(smem + p.off_list);
    plan->token = reinterpret_cast<uint8_t *>(smem + p.off_token);
    for (int e = threadIdx.x; e < p.E; e += kThreads) plan->mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {
        const int e = p.idx[i];
        if ((unsigned)e < (unsigned)p.E) atomicOr(&plan->mask[e], 1ull << (i / p.k));      // the order does not show
        else if (!DOWN && e >= p.E && blockIdx.x == 0 && p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int rows = 0, n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int mine = e0 + lane < p.E ? __popcll(plan->mask[e0 + lane]) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (mine) {
                plan->first[e0 + lane] = (uint16_t)(rows + upto - mine);
                plan->list[n + __popc(some & ((1u << lane) - 1))] = (uint16_t)(e0 + lane);
            }
            rows += __shfl_sync(0xffffffffu, upto, 31);
            n += __popc(some);
        }
        if (lane == 0) *present = n;
        if (DOWN)
            for (int r = lane; r < rows; r += 32) plan->weight[r] = 0.f;
    }
    __syncthreads();
    plan->present = *present;
    if (DOWN && threadIdx.x < p.T) {         // a thread for each token: one that names an expert twice adds in order
        const int t = threadIdx.x;
        for (int j = 0; j < p.k; ++j) {
            const int e = p.idx[t * p.k + j];
            if ((unsigned)e >= (unsigned)p.E) continue;
            const int row = plan->first[e] + bits_below(plan->mask[e], t);
            plan->weight[row] += p.w[t * p.k + j];
            plan->token[row] = (uint8_t)t;
        }
    }
    if (DOWN) __syncthreads();
}

// The accumulators that a CTA fills, one after the other.  Up: tile m of the
// i-th chosen expert.  Down: tile m of the outputs for all experts, at most
// kMostRows rows of h at a time (an expert with more has its weights come again, from
// L2), so that the ring need not be laid out for all tokens.
template <bool DOWN> struct Walk {
    const FewParams &p;
    const Plan &plan;
    int tiles, u, i, m, row;     // row: first of the expert's rows
    __device__ Walk(const FewParams &params, const Plan &pl)
        : p(params), plan(pl), tiles((params.M + per_tile(params) - 1) / per_tile(params)),
          u(DOWN ? blockIdx.x / params.split : blockIdx.x), i(0), m(0), row(0) {
        place();
    }
    static __device__ int per_tile(const FewParams &p) { return !DOWN && p.act == EP_ACT_SWIGLU ? p.rows / 2 : p.rows; }
    __device__ void place() {
        if constexpr (DOWN) {
            m = u;
        } else {
            i = u / tiles;
            m = u - i * tiles;
        }
    }
    __device__ bool more() const { return DOWN ? u < tiles && plan.present > 0 : u < tiles * plan.present; }
    __device__ int expert() const { return plan.list[i]; }
    __device__ int rows_from(int at) const { return __popcll(plan.mask[expert()]) - at; }
    __device__ int rows() const { return min(rows_from(row), kMostRows); }
    __device__ bool last_of_tile() const { return i + 1 == plan.present && rows_from(row) <= kMostRows; }
    __device__ void next() {
        if constexpr (DOWN) {
            if (rows_from(row) > kMostRows) {
                row += kMostRows;
                return;
            }
            row = 0;
            if (++i < plan.present) return;
            i = 0;
            u += gridDim.x / p.split;
        } else {
            u += gridDim.x;
        }
        place();
    }
};

// This CTA's part of K, in slices.
template <bool DOWN> struct Depth {
    int first, n;
    __device__ explicit Depth(const FewParams &p) {
        const int all = (p.K + kSlice - 1) / kSlice;
        if constexpr (DOWN) {
            const int r = blockIdx.x % p.split;          // the CTA's rank in its cluster
            first = r * all / p.split;
            n = (r + 1) * all / p.split - first;
        } else {
            first = 0;
            n = all;
        }
    }
};

// Columns of an accumulator.  Up: all tokens.  Down: for every 8 rows of h 8 of
// upper and 8 of lower halves.
template <bool DOWN> __device__ __forceinline__ int columns_of(const FewParams &p, const Walk<DOWN> &at) {
    return DOWN ? (at.rows() + 7) / 8 * 16 : (p.T + 15) & ~15;
}

// Tensor memory for two accumulators: a power of two of at least 32 columns.
__device__ __forceinline__ uint32_t tmem_columns(int columns) {
    uint32_t n = 32;
    while (n < 2u * columns) n *= 2;
    return n;
}

// ---- the first warps: copies

template <bool DOWN, bool GATED> struct FewLoader {
    const FewWork &w;
    const Plan &plan;
    FewBarriers &bars;
    uint32_t ring;

    __device__ uint32_t stage(uint32_t s) const { return ring + s * w.p.stage_bytes; }
    __device__ void weights(uint32_t s, const Walk<DOWN> &at, int k) const {
        const FewParams &p = w.p;
        const uint32_t bar = smem_u32(&bars.full[s]), half = p.rows * 128;
        const int e = at.expert();
        for (int h = 0; h < (p.K - k > 64 ? 2 : 1); ++h) {
            if constexpr (GATED) tma_load5<false>(stage(s) + h * half, &w.a, bar, k + h * 64, 0, 0, at.m * (p.rows / 16), e);
            else tma_load3<false>(stage(s) + h * half, &w.a, bar, k + h * 64, at.m * p.rows, e);
        }
    }
    // Boxes of tokens in a half slice, and where the halves start.
    __device__ int boxes(const Walk<DOWN> &at) const { return DOWN ? (at.rows() + 7) / 8 : 1; }
    __device__ void tokens(uint32_t s, const Walk<DOWN> &at, int k, int n) const {
        const FewParams &p = w.p;
        const uint32_t bar = smem_u32(&bars.full[s]), to = stage(s) + p.rows * 256;
        const int first = DOWN ? plan.first[at.expert()] + at.row : 0;
        for (int h = 0; h < (p.K - k > 64 ? 2 : 1); ++h)
            for (int j = 0; j < n; ++j)
                tma_load3<false>(to + (h * n + j) * p.box * 128, &w.b, bar, k + h * 64, first + j * 8, 0);
    }
    __device__ void expect(uint32_t s, int k, int n) const {
        const FewParams &p = w.p;
        mbar_expect(smem_u32(&bars.full[s]), (p.K - k > 64 ? 2 : 1) * (p.rows + n * p.box) * 128);
    }

    // This warp's slices: every kLoaders-th one, from its own number on.
    struct Slices {
        Walk<DOWN> at;
        Depth<DOWN> depth;
        int n, ks;                                       // slice, its place in the accumulator
        __device__ Slices(const FewParams &p, const Plan &plan, int mine) : at(p, plan), depth(p), n(mine), ks(mine) { settle(); }
        __device__ void settle() {
            for (; at.more() && ks >= depth.n; at.next()) ks -= depth.n;
        }
        __device__ bool more() const { return at.more(); }
        __device__ int k() const { return (depth.first + ks) * kSlice; }
        __device__ void next() {
            n += kLoaders;
            ks += kLoaders;
            settle();
        }
    };

    __device__ void run(int mine) {
        const FewParams &p = w.p;
        const bool elected = elect_one();
        const int S = p.stages;
        bool ok = true;
        if constexpr (DOWN) {                            // weights for a whole ring, ahead of h
            for (Slices it(p, plan, mine); it.more() && it.n < S; it.next()) {
                if (elected) {
                    expect(it.n, it.k(), boxes(it.at));
                    weights(it.n, it.at, it.k());
                }
                __syncwarp();
            }
            grid_dependency_wait();
        }
        int s = mine % S, last = -1;
        uint32_t phase = mine / S & 1u;
        Slices it(p, plan, mine);
        for (; it.more(); it.next()) {
            // by the whole warp, which stays together: a lane that fell two
            // rounds behind would wait for a phase that has passed
            ok = warp_wait(smem_u32(&bars.empty[s]), phase ^ 1u, &bars.watch);
            if (!ok) break;
            if (elected) {
                const int n = boxes(it.at);
                if (!DOWN || it.n >= S) {
                    expect(s, it.k(), n);
                    weights(s, it.at, it.k());
                }
                tokens(s, it.at, it.k(), n);
                *(volatile uint32_t *)&bars.watch.loaded = it.n + 1;
            }
            __syncwarp();
            last = it.n;
            for (s += kLoaders; s >= S; s -= S) phase ^= 1u;
        }
        // The CTA ends no earlier than its copies and its stages' last signals (of
        // the last S slices of all warps: earlier ones' phases have passed);
        // after a wait that ran out, as far as they come within another wait each.
        if ((threadIdx.x & 31) == 0) {
            Watch ignore = {};
            volatile Watch *watch = ok ? (volatile Watch *)&bars.watch : &ignore;
            const int all = ok ? it.n - it.ks : last + 1;
            for (int n = last; n >= 0 && n >= all - S; n -= kLoaders) {
                const uint32_t q = n % S, round = n / S & 1u;
                if (!ok) tensor_wait(smem_u32(&bars.full[q]), round, watch);
                tensor_wait(smem_u32(&bars.empty[q]), round, watch);
            }
        }
        __syncwarp();
    }
};

// ---- the next warp: matrix instructions

template <typename T, bool DOWN>
__device__ void few_multiply(const FewParams &p, const Plan &plan, FewBarriers &bars, uint32_t ring, uint32_t tmem) {
    const bool elected = elect_one();
    constexpr uint32_t kIdesc = f16_idesc(std::is_same<T, __nv_bfloat16>::value, false, false, 128);
    uint32_t s = 0, phase = 0, acc = 0;
    bool ok = true;
    const Depth<DOWN> depth(p);
    for (Walk<DOWN> at(p, plan); ok && at.more(); at.next()) {
        const int n = columns_of<DOWN>(p, at), boxes = DOWN ? n / 16 : 1;
        const uint32_t idesc = kIdesc | idesc_n(n), d = tmem + (acc & 1u) * p.columns;
        ok = warp_wait(smem_u32(&bars.acc_empty[acc & 1u]), ((acc >> 1) & 1u) ^ 1u, &bars.watch);
        tcgen_after_sync();
        for (int ks = 0; ks < depth.n; ++ks) {
            const int k = (depth.first + ks) * kSlice;
            ok = ok && warp_wait(smem_u32(&bars.full[s]), phase, &bars.watch);
            if (!ok) break;
            if (elected) {
                // rows of weights past p.rows are whatever follows in shared
                // memory: their lanes of the accumulator are not read
                const uint32_t base = ring + s * p.stage_bytes;
                const uint64_t a0 = smem_desc(base, 16, 1024), a1 = smem_desc(base + p.rows * 128, 16, 1024);
                const uint64_t b0 = smem_desc(base + p.rows * 256, 16, 1024);
                const uint64_t b1 = smem_desc(base + p.rows * 256 + boxes * p.box * 128, 16, 1024);
#pragma unroll
                for (int j = 0; j < kSlice / 16; ++j)
                    if (j == 0 || k + j * 16 < p.K)
                        mma_f16_single(d, (j < 4 ? a0 : a1) + j % 4 * 2, (j < 4 ? b0 : b1) + j % 4 * 2, idesc, ks > 0 || j > 0);
                mma_commit_single(smem_u32(&bars.empty[s]));
            }
            __syncwarp();
            if (++s == (uint32_t)p.stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        if (ok && elected) mma_commit_single(smem_u32(&bars.acc_full[acc & 1u]));
        ++acc;
    }
    if (!ok) {                                           // let the matrix unit finish
        Watch ignore = {};
        if (elect_one()) mma_commit_single(smem_u32(&bars.drained));
        tensor_wait(smem_u32(&bars.drained), 0, &ignore);
    }
}

// ---- the last four warps: outputs.  A lane has a row of weights, a register a column.

template <typename T, bool GATED>
__device__ void few_finish_up(const FewParams &p, const Plan &plan, FewBarriers &bars, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, r = quarter * 32 + lane;
    if (quarter * 32 >= p.rows) return;
    const bool upper = GATED && (r & 8);                 // 8 rows of the gate, 8 of the up half
    const int in = GATED ? (r >> 4) * 8 + (r & 7) : r;
    uint32_t acc = 0;
    for (Walk<false> at(p, plan); at.more(); at.next(), ++acc) {
        const int e = plan.list[at.i], f = at.m * Walk<false>::per_tile(p) + in;
        const bool live = f < p.M && r < p.rows;
        const unsigned long long mask = plan.mask[e];
        float bias = 0.f;
        if (p.bias && live) bias = f32(static_cast<const T *>(p.bias)[(int64_t)e * (GATED ? 2 * p.M : p.M) + (upper ? p.M : 0) + f]);
        if (!warp_wait(smem_u32(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, &bars.watch)) return;
        tcgen_after_sync();
        const uint32_t d = tmem + (acc & 1u) * p.columns + ((uint32_t)(quarter * 32) << 16);
        const int n = columns_of<false>(p, at);
        T *h = static_cast<T *>(p.h) + (int64_t)plan.first[e] * p.M + f;
        for (int c0 = 0; c0 < n; c0 += 16) {
            uint32_t raw[16];
            tmem_load16(d + c0, raw);
            tmem_wait16(raw);
            if (c0 + 16 >= n) {                          // the accumulator may be filled again
                tcgen_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[acc & 1u]));
            }
            const uint32_t chosen = (uint32_t)(mask >> c0) & 0xffffu;
            float v[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(raw[c]) + bias;
            if constexpr (!GATED) {
                activate8(p.act, v);
                activate8(p.act, v + 8);
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                if (!(chosen >> c & 1u)) continue;       // the same for the warp
                float y = v[c];
                if constexpr (GATED) y = y * sigmoidf(y) * __shfl_xor_sync(0xffffffffu, y, 8);
                const T hi = rounded<T>(y);
                const float left = y - f32(hi);
                if (live && !upper) {
                    h[0] = hi;
                    h[p.h_half] = rounded<T>(left == left ? left : 0.f);       // 0 where y is not finite
                }
                h += p.M;
            }
        }
    }
}

// Reads a float of another CTA's shared memory.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__device__ void few_finish_down(const FewParams &p, const Plan &plan, FewBarriers &bars, float *sums, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, r = quarter * 32 + lane;
    if (quarter * 32 >= p.rows) return;
    const int rank = blockIdx.x % p.split;
    float *mine = sums + r;                              // [T][rows], a column for each thread
    for (int t = 0; t < p.T; ++t) mine[t * p.rows] = 0.f;
    // A meeting of these warps of all CTAs that share the tile.
    uint32_t phase = 0;
    auto meet = [&]() -> bool {
        if (p.split == 1) return true;
        __syncwarp();
        if (lane < p.split) cluster_arrive(in_cta(smem_u32(&bars.joined), lane));
        const bool ok = __all_sync(0xffffffffu, tensor_wait<true>(smem_u32(&bars.joined), phase, &bars.watch));
        phase ^= 1u;
        return ok;
    };
    // The tile's outputs; with other CTAs every split-th token of them, the
    // parts added in order of rank.
    auto write = [&](int m) -> bool {
        if (!meet()) return false;
        if (m < p.M) {
            const T *res = static_cast<const T *>(p.residual.ptr);
            T *out = static_cast<T *>(p.out.ptr) + m;
#pragma unroll 4
            for (int t = rank; t < p.T; t += p.split) {
                float v;
                if (p.split == 1) {
                    v = mine[t * p.rows];
                } else {
                    v = 0.f;
                    for (int q = 0; q < p.split; ++q) v += ld_cluster(in_cta(smem_u32(mine + t * p.rows), q));
                }
                if (res) v += f32(res[t * p.residual.row_stride + m]);
                out[t * p.out.row_stride] = rounded<T>(v);
            }
        }
        if (!meet()) return false;                       // the others have read
        for (int t = 0; t < p.T; ++t) mine[t * p.rows] = 0.f;
        return true;
    };
    if (plan.present == 0) {
        for (int u = blockIdx.x / p.split; u * p.rows < p.M; u += gridDim.x / p.split)
            if (!write(u * p.rows + r)) return;
        return;
    }
    uint32_t acc = 0;
    for (Walk<true> at(p, plan); at.more(); at.next(), ++acc) {
        const int e = at.expert(), m = at.m * p.rows + r;
        const int rows = at.rows(), n = columns_of<true>(p, at);
        float bias = 0.f;
        if (p.bias && m < p.M && rank == 0) bias = f32(static_cast<const T *>(p.bias)[(int64_t)e * p.M + m]);
        if (!warp_wait(smem_u32(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, &bars.watch)) return;
        tcgen_after_sync();
        const uint32_t d = tmem + (acc & 1u) * p.columns + ((uint32_t)(quarter * 32) << 16);
        const float *weight = plan.weight + plan.first[e] + at.row;
        const uint8_t *token = plan.token + plan.first[e] + at.row;
        for (int c0 = 0; c0 < n; c0 += 16) {
            uint32_t raw[16];
            tmem_load16(d + c0, raw);
            tmem_wait16(raw);
            if (c0 + 16 >= n) {
                tcgen_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[acc & 1u]));
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int j = c0 / 2 + c;
                if (j >= rows) break;
                const float v = __uint_as_float(raw[c]) + __uint_as_float(raw[c + 8]) + bias;
                mine[token[j] * p.rows] += weight[j] * v;
            }
        }
        if (at.last_of_tile() && !write(m)) return;
    }
}

template <typename T, bool DOWN, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewWork w) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ FewBarriers bars;
    const FewParams &p = w.p;
    const int warp = threadIdx.x >> 5;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (ring - smem_u32(smem_raw));

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], (p.rows + 31) / 32);
        }
        mbar_init(&bars.joined, DOWN ? p.split * ((p.rows + 31) / 32) : 1);
        mbar_init(&bars.drained, 1);
        bars.watch.gave_up = 0;
        bars.watch.loaded = 0;
        mbar_init_fence();
        tma_prefetch_map(&w.a);
        tma_prefetch_map(&w.b);
    }
    __syncwarp();
    if (DOWN && p.split > 1) cluster_sync();             // the barriers stand before another CTA signals
    if (warp == kLoaders) tmem_alloc_single(smem_u32(&bars.tmem), tmem_columns(p.columns));
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    const uint32_t tmem = bars.tmem;
    // Up waits for the kernel before it here.  Down's indices and weights are up's
    // too: they were there before up began, and up lets down begin only after its own
    // wait; down waits where it needs h.
    if (!DOWN) {
        grid_dependency_wait();
        grid_dependents_may_launch();
    }
    Plan plan;
    make_plan<DOWN>(p, smem, &bars.present, &plan);
    if (warp < kLoaders) {
        FewLoader<DOWN, GATED>{w, plan, bars, ring}.run(warp);
    } else {
        if (DOWN) grid_dependency_wait();
        if (warp == kLoaders) few_multiply<T, DOWN>(p, plan, bars, ring, tmem);
        else if constexpr (DOWN) few_finish_down<T>(p, plan, bars, reinterpret_cast<float *>(smem + p.off_acc), tmem);
        else few_finish_up<T, GATED>(p, plan, bars, tmem);
    }
    if (DOWN) grid_dependents_may_launch();
    __syncwarp();
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    if (DOWN && p.split > 1) cluster_sync();             // nobody reads or signals here any more
    if (warp == kLoaders) tmem_free_single(tmem, tmem_columns(p.columns));
    if (threadIdx.x == 0 && bars.watch.gave_up && p.error) atomicOr(p.error, EP_DEVERR_TIMEOUT);
}

// -------------------------------------------------------------- host side

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

// h in two halves, a row for every choice.
int64_t h_rows(const ep_few_desc_t &d) { return (int64_t)d.tokens * d.topk; }
size_t workspace(const ep_few_desc_t &d) { return (size_t)h_rows(d) * d.inner * 4; }

// The ring takes what the rest leaves.  Behind it stand the sums and the plan,
// 16 KB at least: instructions read 128 rows of weights whatever a tile has.
bool lay_out(FewParams *p, bool down, size_t *bytes) {
    const int rows_most = p->T * p->k;
    const int most = p->T < kMostRows ? p->T : kMostRows;
    p->stage_bytes = p->rows * 256 + (down ? (most + 7) / 8 * 16 : p->box) * 256;
    int at = 0;
    auto take = [&](int size) {
        const int was = at;
        at = (at + size + 15) & ~15;
        return was;
    };
    const int acc = take(down ? p->T * p->rows * 4 : 0), mask = take(p->E * 8), weight = take(down ? rows_most * 4 : 0);
    const int first = take(p->E * 2), list = take(p->E * 2), token = take(down ? rows_most : 0);
    if (at < 16384) at = 16384;
    p->stages = (kSmemMost - 1024 - at) / p->stage_bytes;
    if (p->stages > kMaxStages) p->stages = kMaxStages;
    if (p->stages < kLoaders) return false;      // see FewLoader: a warp counts on slices a ring behind its last one
    const int ring = p->stages * p->stage_bytes;
    p->off_acc = ring + acc;
    p->off_mask = ring + mask;
    p->off_weight = ring + weight;
    p->off_first = ring + first;
    p->off_list = ring + list;
    p->off_token = ring + token;
    *bytes = 1024 + ring + at;
    return true;
}

template <typename T, bool DOWN, bool GATED> ep_status_t launch_few(FewWork &w, int64_t tiles, cudaStream_t st) {
    static std::atomic<bool> configured[kMaxDevices];
    int dev;
    size_t bytes;
    if (!lay_out(&w.p, DOWN, &bytes)) return EP_ERR_INVALID_ARGS;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return EP_ERR_GPU_OP;
    const int sms = sm_count(dev);
    if (sms < 1) return EP_ERR_GPU_OP;
    if (!configured[dev].load(std::memory_order_acquire)) {          // the attribute is per device
        if (cudaFuncSetAttribute(few_kernel<T, DOWN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess)
            return EP_ERR_GPU_OP;
        configured[dev].store(true, std::memory_order_release);
    }
    const int64_t clusters = sms / w.p.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < clusters ? tiles : clusters) * w.p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = w.p.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_kernel<T, DOWN, GATED>, w) == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

template <typename T>
ep_status_t launch(const ep_few_desc_t &d, FewWork &up, FewWork &down, int64_t up_tiles, int64_t down_tiles, cudaStream_t st) {
    const ep_status_t s = d.activation == EP_ACT_SWIGLU ? launch_few<T, false, true>(up, up_tiles, st)
                                                        : launch_few<T, false, false>(up, up_tiles, st);
    return s == EP_SUCCESS ? launch_few<T, true, false>(down, down_tiles, st) : s;
}

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
    const bool gated = d->activation == EP_ACT_SWIGLU;
    const int T = d->tokens, H = d->hidden, F = d->inner, E = d->experts;
    const int64_t wide = wide_of(*d), rows = h_rows(*d);
    const int64_t most = E < rows ? E : rows;            // experts that can be chosen

    FewWork up = {}, down = {};
    up.p.T = down.p.T = T;
    up.p.E = down.p.E = E;
    up.p.k = down.p.k = d->topk;
    up.p.act = d->activation;
    up.p.w = down.p.w = d_w;
    up.p.idx = down.p.idx = d_idx;
    up.p.h = down.p.h = d_workspace;
    up.p.h_half = rows * F;
    up.p.error = down.p.error = d_error;
    up.p.M = F;
    up.p.K = H;
    up.p.bias = d->up_bias;
    up.p.box = (T + 7) & ~7;
    up.p.columns = (T + 15) & ~15;
    down.p.M = H;
    down.p.K = F;
    down.p.bias = d->down_bias;
    down.p.box = 16;
    down.p.columns = ((T < kMostRows ? T : kMostRows) + 7) / 8 * 16;
    down.p.residual = *residual;
    down.p.out = *out;

    // narrower tiles while there are too few of them for the SMs
    up.p.rows = 128;
    while (up.p.rows > 32 && most * ((wide + up.p.rows - 1) / up.p.rows) < 300) up.p.rows /= 2;
    down.p.rows = 128;
    const int slices = (F + kSlice - 1) / kSlice, tiles = (H + 127) / 128;
    up.p.split = down.p.split = 1;
    while (down.p.split < 8 && 2 * down.p.split <= slices && tiles * down.p.split * 2 <= 144) down.p.split *= 2;
    const int64_t up_tiles = most * ((wide + up.p.rows - 1) / up.p.rows), down_tiles = (H + down.p.rows - 1) / down.p.rows;

    const ep_rows_t tokens = {x->ptr, 0, x->row_stride};
    const uint64_t dims[3] = {(uint64_t)F, (uint64_t)rows, 2};
    const int64_t strides[3] = {1, F, rows * F};
    const uint32_t box[3] = {64, 8, 2};
    if (!(gated ? encode_gated(&up.a, d->dtype, d->up, H, F, E, up.p.rows / 16)
                : encode_rows(&up.a, d->dtype, d->up, H, F, E, up.p.rows)) ||
        !encode_rows(&up.b, d->dtype, tokens, H, T, 1, up.p.box) ||
        !encode_rows(&down.a, d->dtype, d->down, F, H, E, down.p.rows) ||
        !encode(&down.b, d->dtype, d_workspace, 3, dims, strides, box))
        return EP_ERR_GPU_OP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->dtype == EP_DT_BF16 ? launch<__nv_bfloat16>(*d, up, down, up_tiles, down_tiles, st)
                                  : launch<__half>(*d, up, down, up_tiles, down_tiles, st);
}

}  // extern "C"
