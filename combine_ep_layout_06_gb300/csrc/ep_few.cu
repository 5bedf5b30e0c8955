// The experts of a few tokens: both products and the weighted sum, in two
// kernels; a pair for little work (further down), where latency is all, and this one:
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
// gather.  Down's slices (tiles of outputs, in each all experts, in each the depth) are
// one sequence, of which every CTA takes an equal part; it sums the experts of a tile
// in shared memory.  Where a tile falls to several CTAs, the warp that finishes its
// rows last adds their parts, in the sequence's order: who is last does not show.
// h stands grouped by expert, in two 16-bit halves (a value and what its rounding
// left, see Halves) that are columns of their own, because 16 columns cost what 8 do.
//
// Down is launched programmatically: its CTAs start as up's end, and fill their
// rings with weights before they wait for h.
#include <cuda.h>

#include "ep_rows.cuh"
#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kTile = 128;                   // rows of weights: the instructions' other size costs as much
constexpr int kSlice = 128;                  // k of a slice: two halves of 64, 128 bytes each
constexpr int kMaxStages = 12;
constexpr int kLoaders = 2, kFinishers = 4;    // warps
constexpr int kMostRows = 32;                // of h in an accumulator of down
constexpr int kMostCtas = 160;
// Down gives every tile to equally many CTAs where that uses this many tenths of the
// SMs (one token 102.5 us, 7168 outputs on 112 CTAs; in equal parts of all 152 104.8).
constexpr int kEvenTenths = 7;
constexpr int kLeastSlices = 4;              // of a CTA of down, while there are more CTAs than one
constexpr int kThreads = (kLoaders + 1 + kFinishers) * 32;
constexpr int kSmemMost = 227 * 1024 - 1024; // of a CTA, less what is static

struct FewParams {
    int T, E, k, M, K;           // M: outputs of this product (gated: of a half); K: its depth
    int act;
    int box;                     // up: token rows a copy brings
    int ring_bytes, columns;
    int off_acc, off_mask, off_weight, off_first, off_list, off_token;    // in shared memory, after the ring
    const float *w;
    const int32_t *idx;
    const void *bias;            // [E][features]
    void *h;                     // [2][T * k][F]
    int64_t h_half;
    float *parts;                // down: [CTAs][2][T][kTile] sums of tiles that are shared
    uint32_t *tickets;           // [kMostCtas][kFinishers] parts that are there; up sets them to 0
    ep_rows_t residual, out;
    uint32_t *error;
};
struct FewWork {
    CUtensorMap a, b;
    FewParams p;
};

struct __align__(8) FewBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int present, most;
    Watch watch;
};

// Which tokens chose which expert.  Experts that were chosen stand in `list`, in
// ascending order (for down an expert with more than kMostRows rows stands there
// once for every kMostRows of them); the rows of expert e are first[e] and on, its
// tokens in order.
struct Plan {
    unsigned long long *mask;    // [E] tokens
    float *weight;               // [rows], down only
    uint16_t *first, *list;      // [E], [entries]; an entry is an expert, from bit kChunkBit on the number of its kMostRows rows
    uint8_t *token;              // [rows], down only
    int present;                 // entries of list
    int stages, stage_bytes;     // of the ring: down's stages hold the rows that its entries have at most
};
constexpr int kChunkBit = 12;
static_assert(EP_MAX_ROUTE_EXPERTS <= 1 << kChunkBit, "an entry holds an expert and its chunk");

__device__ __forceinline__ int bits_below(unsigned long long mask, int t) { return __popcll(mask & ((1ull << t) - 1)); }

template <bool DOWN> __device__ void make_plan(const FewParams &p, unsigned char *smem, FewBarriers *bars, Plan *plan) {
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
        int rows = 0, n = 0, most = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int mine = e0 + lane < p.E ? __popcll(plan->mask[e0 + lane]) : 0;
            const int chunks = DOWN ? (mine + kMostRows - 1) / kMostRows : mine > 0;
            most = max(most, min(mine, kMostRows));
            int upto = mine << 16 | chunks;              // both running sums at once
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (mine) plan->first[e0 + lane] = (uint16_t)(rows + (upto >> 16) - mine);
            for (int c = 0; c < chunks; ++c)
                plan->list[n + (upto & 0xffff) - chunks + c] = (uint16_t)(e0 + lane | c << kChunkBit);
            upto = __shfl_sync(0xffffffffu, upto, 31);
            rows += upto >> 16;
            n += upto & 0xffff;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            bars->present = n;
            bars->most = most;
        }
        if (DOWN)
            for (int r = lane; r < rows; r += 32) plan->weight[r] = 0.f;
    }
    __syncthreads();
    plan->present = bars->present;
    plan->stage_bytes = kTile * 256 + (DOWN ? max(1, (bars->most + 7) / 8) * 16 : p.box) * 256;
    plan->stages = min(p.ring_bytes / plan->stage_bytes, kMaxStages);
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

// The accumulators that a CTA fills, one after the other: n slices from ks on of
// the depth of tile m of the i-th entry of the plan's list.  Up: a whole tile of one
// expert.  Down: a part of the sequence of all slices.
template <bool DOWN> struct Walk;
template <> struct Walk<false> {
    const Plan &plan;
    int tiles, u, i, m, n;
    static constexpr int ks = 0;
    static __device__ int per_tile(const FewParams &p) { return p.act == EP_ACT_SWIGLU ? kTile / 2 : kTile; }
    __device__ Walk(const FewParams &p, const Plan &pl)
        : plan(pl), tiles((p.M + per_tile(p) - 1) / per_tile(p)), u(blockIdx.x), n((p.K + kSlice - 1) / kSlice) { place(); }
    __device__ void place() {
        i = u / tiles;
        m = u - i * tiles;
    }
    __device__ bool more() const { return u < tiles * plan.present; }
    __device__ int expert() const { return plan.list[i]; }
    __device__ void next() {
        u += gridDim.x;
        place();
    }
};
template <> struct Walk<true> {
    const Plan &plan;
    int64_t total;               // slices
    int per, ctas;               // slices of a depth; CTAs that take part
    int64_t left;
    int m, i, ks, n;
    __device__ Walk(const FewParams &p, const Plan &pl) : plan(pl), per((p.K + kSlice - 1) / kSlice) {
        total = (int64_t)((p.M + kTile - 1) / kTile) * plan.present * per;
        // A CTA's slices cost 0.4 us each where weights come fast, a part T / 100 us to the
        // one that joins a tile's: both are least at the root of their product (64 tokens of
        // 64 experts, 512 x 256: 30 us, with 4 slices at least 46).
        const int tile_slices = plan.present * per;
        const int least = max(kLeastSlices, (int)sqrtf((float)tile_slices * p.T * (1.0f / 40)));
        const int64_t most = total / least;
        ctas = most < 1 ? 1 : most < gridDim.x ? (int)most : (int)gridDim.x;
        const int c = blockIdx.x;
        const int64_t lo = start(c);
        left = c < ctas ? start(c + 1) - lo : 0;
        const int64_t tile = (int64_t)plan.present * per;
        m = tile ? (int)(lo / tile) : 0;
        const int64_t in = lo - m * tile;
        i = (int)(in / per);
        ks = (int)(in - (int64_t)i * per);
        n = (int)min((int64_t)(per - ks), left);
    }
    __device__ int64_t start(int c) const { return c * total / ctas; }
    // The CTA that has a slice.
    __device__ int owner(int64_t slice) const { return (int)(((slice + 1) * ctas - 1) / total); }
    // The first and the last CTA of this tile.
    __device__ int first_cta() const { return owner((int64_t)m * plan.present * per); }
    __device__ int last_cta() const { return owner((int64_t)(m + 1) * plan.present * per - 1); }
    __device__ bool more() const { return left > 0; }
    __device__ int expert() const { return plan.list[i] & ((1 << kChunkBit) - 1); }
    __device__ int row() const { return (plan.list[i] >> kChunkBit) * kMostRows; }
    __device__ int rows() const { return min(__popcll(plan.mask[expert()]) - row(), kMostRows); }
    // Whether this CTA has no more of this tile after this accumulator.
    __device__ bool last_of_tile() const { return n == left || (i + 1 == plan.present && ks + n == per); }
    __device__ void next() {
        left -= n;
        ks = 0;
        if (++i == plan.present) {
            i = 0;
            ++m;
        }
        n = (int)min((int64_t)per, left);
    }
};

// Columns of an accumulator.  Up: all tokens.  Down: for every 8 rows of h 8 of
// upper and 8 of lower halves.
template <bool DOWN> __device__ __forceinline__ int columns_of(const FewParams &p, const Walk<DOWN> &at) {
    if constexpr (DOWN) return (at.rows() + 7) / 8 * 16;
    else return (p.T + 15) & ~15;
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

    __device__ uint32_t stage(uint32_t s) const { return ring + s * plan.stage_bytes; }
    __device__ void weights(uint32_t s, const Walk<DOWN> &at, int k) const {
        const FewParams &p = w.p;
        const uint32_t bar = smem_u32(&bars.full[s]), half = kTile * 128;
        const int e = at.expert();
        for (int h = 0; h < (p.K - k > 64 ? 2 : 1); ++h) {
            if constexpr (GATED) tma_load5<false>(stage(s) + h * half, &w.a, bar, k + h * 64, 0, 0, at.m * (kTile / 16), e);
            else tma_load3<false>(stage(s) + h * half, &w.a, bar, k + h * 64, at.m * kTile, e);
        }
    }
    // Boxes of tokens in a half slice, and where the halves start.
    __device__ int boxes(const Walk<DOWN> &at) const {
        if constexpr (DOWN) return (at.rows() + 7) / 8;
        else return 1;
    }
    __device__ void tokens(uint32_t s, const Walk<DOWN> &at, int k, int n) const {
        const FewParams &p = w.p;
        const uint32_t bar = smem_u32(&bars.full[s]), to = stage(s) + kTile * 256;
        int first = 0;
        if constexpr (DOWN) first = plan.first[at.expert()] + at.row();
        for (int h = 0; h < (p.K - k > 64 ? 2 : 1); ++h)
            for (int j = 0; j < n; ++j)
                tma_load3<false>(to + (h * n + j) * p.box * 128, &w.b, bar, k + h * 64, first + j * 8, 0);
    }
    __device__ void expect(uint32_t s, int k, int n) const {
        const FewParams &p = w.p;
        mbar_expect(smem_u32(&bars.full[s]), (p.K - k > 64 ? 2 : 1) * (kTile + n * p.box) * 128);
    }

    // This warp's slices: every kLoaders-th one, from its own number on.
    struct Slices {
        Walk<DOWN> at;
        int n, ks;                                       // slice, its place in the accumulator
        __device__ Slices(const FewParams &p, const Plan &plan, int mine) : at(p, plan), n(mine), ks(mine) { settle(); }
        __device__ void settle() {
            for (; at.more() && ks >= at.n; at.next()) ks -= at.n;
        }
        __device__ bool more() const { return at.more(); }
        __device__ int k() const { return (at.ks + ks) * kSlice; }
        __device__ void next() {
            n += kLoaders;
            ks += kLoaders;
            settle();
        }
    };

    __device__ void run(int mine) {
        const FewParams &p = w.p;
        const bool elected = elect_one();
        const int S = plan.stages;
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
        // (Weights that went ahead of h have their tokens by then: a stage's first slice
        // waits for nothing, so that a wait runs out after the first ring only.)
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
    for (Walk<DOWN> at(p, plan); ok && at.more(); at.next()) {
        const int n = columns_of<DOWN>(p, at), boxes = DOWN ? n / 16 : 1;
        const uint32_t idesc = kIdesc | idesc_n(n), d = tmem + (acc & 1u) * p.columns;
        ok = warp_wait(smem_u32(&bars.acc_empty[acc & 1u]), ((acc >> 1) & 1u) ^ 1u, &bars.watch);
        tcgen_after_sync();
        for (int ks = 0; ks < at.n; ++ks) {
            const int k = (at.ks + ks) * kSlice;
            ok = ok && warp_wait(smem_u32(&bars.full[s]), phase, &bars.watch);
            if (!ok) break;
            if (elected) {
                // columns past the tokens that were loaded are whatever follows in
                // shared memory: they are not read
                const uint32_t base = ring + s * plan.stage_bytes;
                const uint64_t a0 = smem_desc(base, 16, 1024), a1 = smem_desc(base + kTile * 128, 16, 1024);
                const uint64_t b0 = smem_desc(base + kTile * 256, 16, 1024);
                const uint64_t b1 = smem_desc(base + kTile * 256 + boxes * p.box * 128, 16, 1024);
#pragma unroll
                for (int j = 0; j < kSlice / 16; ++j)
                    if (j == 0 || k + j * 16 < p.K)
                        mma_f16_single(d, (j < 4 ? a0 : a1) + j % 4 * 2, (j < 4 ? b0 : b1) + j % 4 * 2, idesc, ks > 0 || j > 0);
                mma_commit_single(smem_u32(&bars.empty[s]));
            }
            __syncwarp();
            if (++s == (uint32_t)plan.stages) {
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

__device__ __forceinline__ float activated(int act, float v) {
    return act == EP_ACT_GELU ? gelu2(both(v)).x : act == EP_ACT_SILU ? silu2(both(v)).x : act == EP_ACT_RELU && v <= 0.f ? 0.f : v;
}

// A value in two halves: value = (upper + lower * kLower) * kUnit.  bf16 has fp32's range
// and needs no factors; 8 + 8 bits keep the value within 2^-17.  fp16 is taken in units of
// 16, and its lower half, the rest of at most 2^-11 of the value, 2^11 times as large: so values
// from 2^-16 on are within 2^-16, smaller ones within 2^-32 (without the factors 2^-25), and
// those from 2^20 on (without, 131008) are infinite.  A larger unit would move both ends up.
template <typename T> struct Halves {
    static constexpr float kUnit = 1.f, kLower = 1.f, kLargest = 0x1.fep127f;
};
template <> struct Halves<__half> {
    static constexpr float kUnit = 16.f, kLower = 0x1p-11f, kLargest = 65504.f;
};
template <typename T> __device__ __forceinline__ void store_halves(T *upper, T *lower, float y) {
    using H = Halves<T>;
    y *= 1.f / H::kUnit;
    const bool finite = fabsf(y) <= 0x1.fffffep127f;
    float hi = f32(rounded<T>(y));
    if (finite && fabsf(hi) > H::kLargest) hi = copysignf(H::kLargest, y);       // the lower half has the rest
    *upper = rounded<T>(hi);
    *lower = rounded<T>(finite ? (y - hi) * (1.f / H::kLower) : 0.f);
}
// The sums over both.  Where an infinite weight made the upper one infinite the lower one,
// of rests that are 0 or of another sign, is NaN or infinite the other way: it counts no more.
template <typename T> __device__ __forceinline__ float joined_halves(float upper, float lower) {
    const float rest = fabsf(upper) <= 0x1.fffffep127f ? lower * Halves<T>::kLower : 0.f;
    return (upper + rest) * Halves<T>::kUnit;
}

// ---- the last four warps: outputs.  A lane has a row of weights, a register a column.

template <typename T, bool GATED>
__device__ void few_finish_up(const FewParams &p, const Plan &plan, FewBarriers &bars, float *turn, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, r = quarter * 32 + lane;
    const bool upper = GATED && (r & 8);                 // 8 rows of the gate, 8 of the up half
    const int in = GATED ? (r >> 4) * 8 + (r & 7) : r;
    float *mine = turn + r;                              // [16][kTile], a column for each thread
    uint32_t acc = 0;
    for (Walk<false> at(p, plan); at.more(); at.next(), ++acc) {
        const int e = plan.list[at.i], f = at.m * Walk<false>::per_tile(p) + in;
        const bool live = f < p.M;
        const unsigned long long mask = plan.mask[e];
        float bias = 0.f;
        if (p.bias && live) bias = f32(static_cast<const T *>(p.bias)[(int64_t)e * (GATED ? 2 * p.M : p.M) + (upper ? p.M : 0) + f]);
        if (!warp_wait(smem_u32(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, &bars.watch)) return;
        tcgen_after_sync();
        const uint32_t d = tmem + (acc & 1u) * p.columns + ((uint32_t)(quarter * 32) << 16);
        const int n = columns_of<false>(p, at);
        T *h = static_cast<T *>(p.h) + (int64_t)plan.first[e] * p.M + f;
        for (int c0 = 0; c0 < n; c0 += 16) {
            const uint32_t chosen = (uint32_t)(mask >> c0) & 0xffffu;
            if (!chosen) continue;                       // of most columns few are the expert's
            uint32_t raw[16];
            tmem_load16(d + c0, raw);
            tmem_wait16(raw);
            // by way of shared memory, so that one piece of code serves every column: most
            // of a short kernel's time is its first way through its code
#pragma unroll
            for (int c = 0; c < 16; ++c) mine[c * kTile] = __uint_as_float(raw[c]);
#pragma unroll 1
            for (uint32_t left = chosen; left; left &= left - 1) {
                float y = mine[(__ffs(left) - 1) * kTile] + bias;
                if constexpr (GATED) y = silu2(both(y)).x * __shfl_xor_sync(0xffffffffu, y, 8);
                else y = activated(p.act, y);
                if (live && !upper) store_halves<T>(h, h + p.h_half, y);
                h += p.M;
            }
        }
        tcgen_before_sync();                             // the accumulator may be filled again
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[acc & 1u]));
    }
}

template <typename T>
__device__ void few_finish_down(const FewParams &p, const Plan &plan, FewBarriers &bars, float *sums, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, r = quarter * 32 + lane;
    float *mine = sums + r;                              // [T][kTile], a column for each thread
    for (int t = 0; t < p.T; ++t) mine[t * kTile] = 0.f;
    // What goes to memory: each warp its own 32 rows, a lane 4 neighbouring
    // outputs of every fourth token.
    const int col = quarter * 32 + lane % 8 * 4, t0 = lane / 8;
    auto output = [&](int m) {
        __syncwarp();
        if (m < p.M)
#pragma unroll 2
            for (int t = t0; t < p.T; t += 4) {
                float4 v = *reinterpret_cast<const float4 *>(sums + t * kTile + col);
                if (p.residual.ptr) {
                    const T *res = static_cast<const T *>(p.residual.ptr) + t * p.residual.row_stride + m;
                    const uint2 q = *reinterpret_cast<const uint2 *>(res);
                    const float2 x = unpack2<T>(q.x), y = unpack2<T>(q.y);
                    v = make_float4(v.x + x.x, v.y + x.y, v.z + y.x, v.w + y.y);
                }
                *reinterpret_cast<uint2 *>(static_cast<T *>(p.out.ptr) + t * p.out.row_stride + m) =
                    make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
            }
    };
    // A tile's outputs, or this CTA's part of them.
    auto write = [&](const Walk<true> &at) {
        const int a = at.first_cta(), z = at.last_cta();
        const int64_t part = (int64_t)p.T * kTile;
        bool last = true;
        __syncwarp();
        if (a != z) {
            // a CTA has at most one part that is not a tile's first, and one that is
            float *to = p.parts + (blockIdx.x * 2 + (blockIdx.x == a)) * part + col;
#pragma unroll 2
            for (int t = t0; t < p.T; t += 4)
                __stcg(reinterpret_cast<float4 *>(to + t * kTile), *reinterpret_cast<const float4 *>(sums + t * kTile + col));
            __threadfence();
            __syncwarp();
            uint32_t there = 0;
            if (lane == 0) there = atom_add_acq_rel_gpu(p.tickets + a * kFinishers + quarter, 1u);
            last = __shfl_sync(0xffffffffu, there, 0) == (uint32_t)(z - a);
            if (last) {
                __threadfence();
                constexpr int kAhead = 4;                // tokens, and parts, on their way at a time
#pragma unroll 1
                for (int t = t0; t < p.T; t += 4 * kAhead) {
                    float4 v[kAhead];
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                    for (int c = a; c <= z; c += kAhead) {
                        float4 w[kAhead][kAhead];
#pragma unroll
                        for (int q = 0; q < kAhead; ++q)
#pragma unroll
                            for (int j = 0; j < kAhead; ++j)
                                w[q][j] = c + q <= z && t + 4 * j < p.T
                                              ? __ldcg(reinterpret_cast<const float4 *>(
                                                    p.parts + ((c + q) * 2 + (c + q == a)) * part + (t + 4 * j) * kTile + col))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int q = 0; q < kAhead; ++q)
#pragma unroll
                            for (int j = 0; j < kAhead; ++j) {
                                v[j].x += w[q][j].x;
                                v[j].y += w[q][j].y;
                                v[j].z += w[q][j].z;
                                v[j].w += w[q][j].w;
                            }
                    }
#pragma unroll
                    for (int j = 0; j < kAhead; ++j)
                        if (t + 4 * j < p.T) *reinterpret_cast<float4 *>(sums + (t + 4 * j) * kTile + col) = v[j];
                }
            }
        }
        if (last) output(at.m * kTile + col);
        __syncwarp();
        if (at.n < at.left)                              // more tiles to come
            for (int t = 0; t < p.T; ++t) mine[t * kTile] = 0.f;
    };
    if (plan.present == 0) {
        for (int u = blockIdx.x; u * kTile < p.M; u += gridDim.x) output(u * kTile + col);
        return;
    }
    uint32_t acc = 0;
    for (Walk<true> at(p, plan); at.more(); at.next(), ++acc) {
        const int e = at.expert(), m = at.m * kTile + r, row = at.row();
        const int rows = at.rows(), n = columns_of<true>(p, at);
        float bias = 0.f;                                // with the depth's first part
        if (p.bias && m < p.M && at.ks == 0) bias = f32(static_cast<const T *>(p.bias)[(int64_t)e * p.M + m]);
        if (!warp_wait(smem_u32(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, &bars.watch)) return;
        tcgen_after_sync();
        const uint32_t d = tmem + (acc & 1u) * p.columns + ((uint32_t)(quarter * 32) << 16);
        const float *weight = plan.weight + plan.first[e] + row;
        const uint8_t *token = plan.token + plan.first[e] + row;
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
                const float v = joined_halves<T>(__uint_as_float(raw[c]), __uint_as_float(raw[c + 8])) + bias;
                mine[token[j] * kTile] += weight[j] * v;
            }
        }
        if (at.last_of_tile()) write(at);
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
            mbar_init(&bars.acc_empty[i], kFinishers);
        }
        mbar_init(&bars.drained, 1);
        bars.watch.gave_up = 0;
        bars.watch.loaded = 0;
        mbar_init_fence();
        tma_prefetch_map(&w.a);
        tma_prefetch_map(&w.b);
    }
    __syncwarp();
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
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < kMostCtas * kFinishers; i += kThreads) p.tickets[i] = 0;
    }
    Plan plan;
    make_plan<DOWN>(p, smem, &bars, &plan);
    if (warp < kLoaders) {
        FewLoader<DOWN, GATED>{w, plan, bars, ring}.run(warp);
    } else {
        if (DOWN) grid_dependency_wait();
        if (warp == kLoaders) few_multiply<T, DOWN>(p, plan, bars, ring, tmem);
        else if constexpr (DOWN) few_finish_down<T>(p, plan, bars, reinterpret_cast<float *>(smem + p.off_acc), tmem);
        else few_finish_up<T, GATED>(p, plan, bars, reinterpret_cast<float *>(smem + p.off_acc), tmem);
    }
    if (DOWN) grid_dependents_may_launch();
    __syncwarp();
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    if (warp == kLoaders) tmem_free_single(tmem, tmem_columns(p.columns));
    if (threadIdx.x == 0 && bars.watch.gave_up && p.error) atomicOr(p.error, EP_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------- little work
// A warp (or a part of it) for each choice and feature, then for each output and
// choice: every choice reads its expert's weights anew (from L2 after the first),
// but nothing stands between a launch and its loads.

struct SmallParams {
    int T, E, k, H, F, wide, act;
    ep_rows_t up, down, x, residual, out;
    const void *up_bias, *down_bias;
    const float *w;
    const int32_t *idx;
    float *h;                        // [T * k][F]
    uint32_t *error;
};
constexpr int kSmallWarps = 8, kAtOnce = 2;        // 16-byte loads of a row ahead; 4 cost more in warps (8.9 against 10.8 us at 12.6 MB)

template <typename T> __device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b) {
    float x[8], y[8], s = 0.f;
    unpack8<T>(x, a);
    unpack8<T>(y, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * y[i];
    return s;
}
// Lanes of a warp that share a product of depth K, 8 values each at a time: the others
// have products of their own (64 tokens, 2 of 8 experts 512 x 64: 24 us with a warp a
// product, so 8.5; 128 x 128, 60 tokens, 4 of 20: 20.6 and 10.1).
inline int small_lanes(int K) { return K <= 64 ? 8 : K <= 128 ? 16 : 32; }
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, bool GATED, int LANES>
__global__ void __launch_bounds__(kSmallWarps * 32) small_up_kernel(const SmallParams p) {
    const int lane = threadIdx.x % LANES, f = (blockIdx.x * kSmallWarps * 32 + threadIdx.x) / LANES, pair = blockIdx.y;
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int e = p.idx[pair];
    if ((unsigned)e >= (unsigned)p.E) {
        if (e >= p.E && f == 0 && lane == 0 && p.error) atomicOr(p.error, EP_DEVERR_BAD_INDEX);
        return;
    }
    const bool live = f < p.F;
    const T *x = static_cast<const T *>(p.x.ptr) + (pair / p.k) * p.x.row_stride;
    const T *w = static_cast<const T *>(p.up.ptr) + e * p.up.rank_stride + f * p.up.row_stride;
    const int64_t half = p.F * p.up.row_stride;
    constexpr int step = LANES * 8;
    float v = 0.f, u = 0.f;
    for (int c0 = lane * 8; live && c0 < p.H; c0 += step * kAtOnce) {
        uint4 a[kAtOnce], b[kAtOnce], d[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = c0 + i * step;
            const bool in = c < p.H;
            b[i] = in ? ld_stream16(w + c) : make_uint4(0, 0, 0, 0);
            if (GATED) d[i] = in ? ld_stream16(w + half + c) : make_uint4(0, 0, 0, 0);
            a[i] = in ? *reinterpret_cast<const uint4 *>(x + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            v += dot8<T>(a[i], b[i]);
            if (GATED) u += dot8<T>(a[i], d[i]);
        }
    }
    v = lanes_sum<LANES>(v);
    if (GATED) u = lanes_sum<LANES>(u);
    if (!live) return;
    const T *bias = p.up_bias ? static_cast<const T *>(p.up_bias) + (int64_t)e * p.wide + f : nullptr;
    if (bias) v += f32(bias[0]);
    if constexpr (GATED) {
        if (bias) u += f32(bias[p.F]);
        v = v * sigmoidf(v) * u;
    } else {
        v = activated(p.act, v);
    }
    if (lane == 0) p.h[(int64_t)pair * p.F + f] = v;
}

// Outputs of a block: its warps share an output's choices, up to 8 of them (one token,
// 8 choices of 512 x 512: 12.4 -> 8.1 us), unless there are outputs enough (64 tokens of
// 256: 18.1 us, shared 20.0).
__host__ __device__ inline int small_outputs(int k, int tokens, int outputs) {
    return tokens * outputs >= 8192 ? 8 : k >= 8 ? 1 : k >= 4 ? 2 : k >= 2 ? 4 : 8;
}

template <typename T, int LANES> __global__ void __launch_bounds__(kSmallWarps * 32) small_down_kernel(const SmallParams p) {
    __shared__ float parts[kSmallWarps][4];
    const int outputs = small_outputs(p.k, p.T, p.H), share = kSmallWarps / outputs;
    constexpr int each = 32 / LANES, step = LANES * 8;            // outputs of a warp
    const int lane = threadIdx.x % LANES, which = (threadIdx.x & 31) / LANES, warp = threadIdx.x >> 5, t = blockIdx.y;
    const int m = (blockIdx.x * outputs + warp / share) * each + which, j0 = warp % share;
    // Indices and weights were there before the first kernel began: the weights'
    // lines are on their way while it ends.
    if (m < p.H)
        for (int j = j0; j < p.k; j += share) {
            const int e = p.idx[t * p.k + j];
            if ((unsigned)e >= (unsigned)p.E) continue;
            const T *w = static_cast<const T *>(p.down.ptr) + e * p.down.rank_stride + m * p.down.row_stride;
            for (int c = lane * 64; c < p.F; c += LANES * 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(w + c));
        }
    grid_dependency_wait();
    grid_dependents_may_launch();
    float sum = 0.f;
    for (int j = j0; j < p.k; j += share) {
        const int pair = t * p.k + j, e = p.idx[pair];
        if ((unsigned)e >= (unsigned)p.E) continue;
        const T *w = static_cast<const T *>(p.down.ptr) + e * p.down.rank_stride + m * p.down.row_stride;
        const float *h = p.h + (int64_t)pair * p.F;
        float v = 0.f;
        for (int c0 = lane * 8; m < p.H && c0 < p.F; c0 += step * kAtOnce) {
            uint4 b[kAtOnce];
            float4 a[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int c = c0 + i * step;
                const bool in = c < p.F;
                b[i] = in ? ld_stream16(w + c) : make_uint4(0, 0, 0, 0);
                a[i][0] = in ? __ldcg(reinterpret_cast<const float4 *>(h + c)) : make_float4(0, 0, 0, 0);
                a[i][1] = in ? __ldcg(reinterpret_cast<const float4 *>(h + c + 4)) : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                float f[8];
                unpack8<T>(f, b[i]);
                v += f[0] * a[i][0].x + f[1] * a[i][0].y + f[2] * a[i][0].z + f[3] * a[i][0].w;
                v += f[4] * a[i][1].x + f[5] * a[i][1].y + f[6] * a[i][1].z + f[7] * a[i][1].w;
            }
        }
        v = lanes_sum<LANES>(v);
        if (p.down_bias && m < p.H) v += f32(static_cast<const T *>(p.down_bias)[(int64_t)e * p.H + m]);
        sum += p.w[pair] * v;
    }
    if (lane == 0) parts[warp][which] = sum;
    __syncthreads();
    if (lane == 0 && j0 == 0 && m < p.H) {
        for (int q = 1; q < share; ++q) sum += parts[warp + q][which];
        if (p.residual.ptr) sum += f32(static_cast<const T *>(p.residual.ptr)[t * p.residual.row_stride + m]);
        static_cast<T *>(p.out.ptr)[t * p.out.row_stride + m] = rounded<T>(sum);
    }
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

// h in two halves, a row for every choice; the parts of shared tiles; tickets.
int64_t h_rows(const ep_few_desc_t &d) { return (int64_t)d.tokens * d.topk; }
size_t h_bytes(const ep_few_desc_t &d) { return ((size_t)h_rows(d) * d.inner * 4 + 255) & ~(size_t)255; }
size_t part_bytes(const ep_few_desc_t &d) { return (size_t)kMostCtas * 2 * d.tokens * kTile * 4; }
size_t workspace(const ep_few_desc_t &d) { return h_bytes(d) + part_bytes(d) + kMostCtas * kFinishers * 4; }

// The ring takes what the rest leaves.  Behind it stand the sums (or what turns a
// column) and the plan, 2 KB at least: instructions read 16 columns where 8 tokens were
// loaded.
bool lay_out(FewParams *p, bool down, size_t *bytes) {
    const int rows_most = p->T * p->k;
    int at = 0;
    auto take = [&](int size) {
        const int was = at;
        at = (at + size + 15) & ~15;
        return was;
    };
    const int acc = take((down ? p->T : 16) * kTile * 4), mask = take(p->E * 8), weight = take(down ? rows_most * 4 : 0);
    const int first = take(p->E * 2), list = take(p->E * 2 * (down ? (p->T + kMostRows - 1) / kMostRows : 1));
    const int token = take(down ? rows_most : 0);
    if (at < 2048) at = 2048;
    const int rows = p->T < kMostRows ? p->T : kMostRows;
    const int stage = kTile * 256 + (down ? (rows + 7) / 8 * 16 : p->box) * 256;       // at most
    const int ring = (kSmemMost - 1024 - at) / 1024 * 1024;
    if (ring < kLoaders * stage) return false;           // see FewLoader: a warp counts on slices a ring behind its last one
    p->ring_bytes = ring;
    p->off_acc = ring + acc;
    p->off_mask = ring + mask;
    p->off_weight = ring + weight;
    p->off_first = ring + first;
    p->off_list = ring + list;
    p->off_token = ring + token;
    *bytes = 1024 + ring + at;
    return true;
}

template <typename T, bool DOWN, bool GATED> ep_status_t launch_few(FewWork &w, int64_t ctas, cudaStream_t st) {
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
    const int most = sms < kMostCtas ? sms : kMostCtas;
    if (DOWN && ctas > most) {                           // whole tiles for equally many CTAs each, where that leaves few SMs out
        const int tiles = (w.p.M + kTile - 1) / kTile, even = tiles <= most ? most / tiles * tiles : 0;
        ctas = even * 10 >= most * kEvenTenths ? even : most;
    }
    return launch_after_previous(few_kernel<T, DOWN, GATED>, (unsigned)(ctas < most ? ctas : most), kThreads, bytes, st, w) ==
                   cudaSuccess
               ? EP_SUCCESS : EP_ERR_GPU_OP;
}

template <typename T>
ep_status_t launch(const ep_few_desc_t &d, FewWork &up, FewWork &down, int64_t up_ctas, int64_t down_ctas, cudaStream_t st) {
    const ep_status_t s = d.activation == EP_ACT_SWIGLU ? launch_few<T, false, true>(up, up_ctas, st)
                                                        : launch_few<T, false, false>(up, up_ctas, st);
    return s == EP_SUCCESS ? launch_few<T, true, false>(down, down_ctas, st) : s;
}

template <typename F> void with_lanes(int K, F f) {
    const int n = small_lanes(K);
    if (n == 8) f(std::integral_constant<int, 8>());
    else if (n == 16) f(std::integral_constant<int, 16>());
    else f(std::integral_constant<int, 32>());
}

template <typename T> ep_status_t launch_small(const SmallParams &p, cudaStream_t st) {
    const int outputs = small_outputs(p.k, p.T, p.H);           // warps' worth
    const int features = kSmallWarps * 32 / small_lanes(p.H), block = outputs * 32 / small_lanes(p.F);
    const dim3 up((p.F + features - 1) / features, p.T * p.k), down((p.H + block - 1) / block, p.T);
    cudaError_t e = cudaSuccess;
    with_lanes(p.H, [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        e = launch_after_previous(p.act == EP_ACT_SWIGLU ? small_up_kernel<T, true, L> : small_up_kernel<T, false, L>, up,
                                  kSmallWarps * 32, 0, st, p);
    });
    if (e == cudaSuccess)
        with_lanes(p.F, [&](auto lanes) {
            e = launch_after_previous(small_down_kernel<T, decltype(lanes)::value>, down, kSmallWarps * 32, 0, st, p);
        });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

// Bytes of weights that the choices read, each its own, up to which the kernels for
// little work are faster: 1.8 MB 3.7 against 11.1 us, 12.6 MB 7.1 against 12.7,
// 25 MB 10.1 against 16.1 (with 128 choices 8.5 to 18 against 19 to 20), 50 MB 16.7
// against 19.3 (with 16 choices of 8 experts 14.7 against 13.7); 63 MB 23.8
// against 19.3, 100 MB 25 to 34 against 15 to 29.
constexpr int64_t kSmallBytes = 48 << 20;

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

    if (rows * H * (wide + F) * 2 <= kSmallBytes) {
        const SmallParams p = {T, E, d->topk, H, F, (int)wide, d->activation, d->up, d->down, *x, *residual, *out,
                               d->up_bias, d->down_bias, d_w, d_idx, static_cast<float *>(d_workspace), d_error};
        return d->dtype == EP_DT_BF16 ? launch_small<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream))
                                      : launch_small<__half>(p, static_cast<cudaStream_t>(stream));
    }
    FewWork up = {}, down = {};
    up.p.T = down.p.T = T;
    up.p.E = down.p.E = E;
    up.p.k = down.p.k = d->topk;
    up.p.act = d->activation;
    up.p.w = down.p.w = d_w;
    up.p.idx = down.p.idx = d_idx;
    up.p.h = down.p.h = d_workspace;
    up.p.h_half = rows * F;
    down.p.parts = reinterpret_cast<float *>(static_cast<char *>(d_workspace) + h_bytes(*d));
    up.p.tickets = down.p.tickets =
        reinterpret_cast<uint32_t *>(static_cast<char *>(d_workspace) + h_bytes(*d) + part_bytes(*d));
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

    const int64_t up_tiles = most * ((wide + kTile - 1) / kTile);
    const int64_t down_slices = most * ((H + kTile - 1) / kTile) * ((F + kSlice - 1) / kSlice);
    const int64_t down_ctas = (down_slices + kLeastSlices - 1) / kLeastSlices;

    const ep_rows_t tokens = {x->ptr, 0, x->row_stride};
    const uint64_t dims[3] = {(uint64_t)F, (uint64_t)rows, 2};
    const int64_t strides[3] = {1, F, rows * F};
    const uint32_t box[3] = {64, 8, 2};
    if (!(gated ? encode_gated(&up.a, d->dtype, d->up, H, F, E, kTile / 16)
                : encode_rows(&up.a, d->dtype, d->up, H, F, E, kTile)) ||
        !encode_rows(&up.b, d->dtype, tokens, H, T, 1, up.p.box) ||
        !encode_rows(&down.a, d->dtype, d->down, F, H, E, kTile) ||
        !encode(&down.b, d->dtype, d_workspace, 3, dims, strides, box))
        return EP_ERR_GPU_OP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->dtype == EP_DT_BF16 ? launch<__nv_bfloat16>(*d, up, down, up_tiles, down_ctas, st)
                                  : launch<__half>(*d, up, down, up_tiles, down_ctas, st);
}

}  // extern "C"
