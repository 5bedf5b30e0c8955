// Expert products: one matrix product per group of rows, with bias,
// activation and residual in its epilogue, and its gradient.
//
// Every product here is  out[n][m] = sum_k A[m][k] * B[n][k]  over one group:
//   forward   m = feature, n = row,   k = input    A = weight,    B = x
//   grad_x    m = input,   n = row,   k = feature  A = weight^T,  B = d
//   grad_w    m = input,   n = feature, k = row    A = x^T,       B = d^T
// The output's contiguous dimension is always m.
//
// Pairs of CTAs, one CTA per SM, walk the tiles of all groups (their row
// counts are on the device): 256 m by up to 256 n, accumulated in tensor
// memory, 128 m in each CTA.  Weights or inputs are the 256-wide operand and
// rows (or features) the other, so that a group with few rows costs a narrow
// instruction (n in steps of 32) and not a padded tile.  A CTA loads its own
// 128 m and half of n, so every byte of n serves both.  In each CTA warp 0
// loads 128-deep slices by TMA into a ring in shared memory; warp 1 of the
// first CTA issues the pair's matrix instructions; warps 2..9 turn a finished
// accumulator into outputs while the next one fills: two accumulators of 256
// columns take all of the SM's tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kTileM = 128, kTileN = 256;          // m of one CTA, n of the pair
// A slice is 128 deep (k): two 16 KB halves of each operand.  K-major (x, a
// weight's rows): 128 rows of 64 k each.  MN-major (the gradients' transposed
// operands): 64 m or n each, 128 rows of k.  A copy brings the 128 bytes that
// the swizzle spans by up to 128 rows, and costs the loading thread about as
// much whatever its size: 64-deep slices of 8 KB copies held grad_w of 16384
// rows at 311 us, these take 250.
constexpr int kSliceK = 128, kStages = 3;
constexpr int kHalfBytes = 128 * 128;
constexpr int kBytesA = 2 * kHalfBytes, kStageBytes = 4 * kHalfBytes;
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kTurnBytes = 32 * 32 * 4;            // a warp's transposing buffer
constexpr size_t kSmemBytes = (size_t)kRingBytes + kEpilogueWarps * kTurnBytes + 1024;
constexpr int kThreads = 64 + kEpilogueWarps * 32;

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

enum Mode { kForward, kGated, kGradX, kGradW, kNone };

struct ProductParams {
    Groups gr;
    int M, N, K;           // N or K < 0: the group's number of rows
    int tile_n;            // columns of a tile: kTileN, 128 or 64
    int act;
    const void *bias;      // [G][M], or [G][2M] (gated)
    ep_rows_t residual, out, pre;
    uint32_t *error;
};

template <typename T> __device__ __forceinline__ float f32(T v);
template <> __device__ __forceinline__ float f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ __nv_bfloat16 rounded(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rounded(float v) { return __float2half_rn(v); }

// Within a few units of the last place of fp32 (more of 2^-24 |v|): far below
// the 16-bit rounding of every result it goes into.
__device__ __forceinline__ float sigmoidf(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

template <typename T> struct IsBf16 { static constexpr bool value = false; };
template <> struct IsBf16<__nv_bfloat16> { static constexpr bool value = true; };

// Walks the tiles of all groups in order, 32 groups at a time: a lane holds
// one group's range and the running number of tiles.  Every lane of the warp
// gets the same answer.
struct Tile {
    int g, seg, first, rows, m;
    int n0, n;             // columns: first and number
};
struct Walker {
    int lane, g0;
    int64_t before, upto;      // tiles before this block of 32 groups; up to this lane's group
    int first, rows, tiles;    // this lane's group

    __device__ void load(const ProductParams &p, int mt) {
        const int g = g0 + lane;
        first = rows = tiles = 0;
        if (g < p.gr.R * p.gr.per) {
            group_range(p.gr, g, &first, &rows);
            tiles = mt * (((p.N < 0 ? rows : p.N) + p.tile_n - 1) / p.tile_n);
        }
        upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
    }
    __device__ void start(const ProductParams &p, int mt) {
        lane = threadIdx.x & 31;
        g0 = 0;
        before = 0;
        load(p, mt);
    }
    __device__ bool find(const ProductParams &p, int mt, int64_t index, Tile *t) {
        for (;;) {
            const int64_t here = __shfl_sync(0xffffffffu, upto, 31);
            if (index < before + here) break;
            before += here;
            g0 += 32;
            if (g0 >= p.gr.R * p.gr.per) return false;
            load(p, mt);
        }
        const int64_t rel = index - before;
        const int l = __ffs(__ballot_sync(0xffffffffu, upto > rel)) - 1;
        const int in = (int)(rel - __shfl_sync(0xffffffffu, upto - tiles, l));
        t->g = g0 + l;
        t->seg = t->g / p.gr.per;
        t->first = __shfl_sync(0xffffffffu, first, l);
        t->rows = __shfl_sync(0xffffffffu, rows, l);
        // bands of at most 16 m-tiles: what runs at a time, some 76 tiles, spans
        // about as much of n as of m (8192 x 8192 x 8192: 712 -> 680 us)
        const int bands = (mt + 15) / 16, band = (mt + bands - 1) / bands;
        // equal parts of N instead of full tiles and a rest: a narrow rest would
        // load as much of the other operand for less work
        const int N = p.N < 0 ? t->rows : p.N;
        const int parts = (N + p.tile_n - 1) / p.tile_n;
        const int width = ((N + parts - 1) / parts + 31) & ~31;
        const int b = in / (band * parts), in_band = in - b * band * parts;
        const int wide = min(band, mt - b * band);
        t->m = b * band + in_band % wide;
        t->n0 = in_band / wide * width;
        t->n = min(width, N - t->n0);
        return true;
    }
};

// The last slice of a group's rows (k): the instructions that it needs take
// 16 rows each, so rows from `live` to the next multiple of 16 are set to zero,
// whatever they held, in all `chunks` chunks.  (The 128-byte swizzle moves
// data within a k row only.)  By a whole warp; the matrix unit sees it
// afterwards.
__device__ __forceinline__ void clear_rows(uint32_t slice, int chunks, int live) {
    const int lane = threadIdx.x & 31, end = (live + 15) & ~15;
    for (int r = live + lane / 8; r < end; r += 4)
        for (int c = 0; c < chunks; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                         :: "r"(slice + c * kHalfBytes + r * 128 + lane % 8 * 16), "r"(0) : "memory");
    fence_async_smem();
    __syncwarp();
}

struct __align__(8) Barriers {
    uint64_t full[kStages], empty[kStages], tail[kStages], peer_tail[kStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    Watch watch;
};

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
template <typename T> __device__ __forceinline__ void add8(float *v, const uint4 &r) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += f32(e[i]);
}
// A warp's transposing buffer: row c (a column of the accumulator) of 32
// floats, its 16-byte blocks in the order block ^ (c & 7), so that neither the
// writes along a row nor the reads of blocks down the rows meet in a bank.
__device__ __forceinline__ float *turn_at(float *turn, int c, int i) {
    return turn + c * 32 + (((i >> 2) ^ (c & 7)) << 2) + (i & 3);
}
__device__ __forceinline__ void read8(float *v, float *turn, int c, int i) {
    const float4 a = *reinterpret_cast<const float4 *>(turn_at(turn, c, i));
    const float4 b = *reinterpret_cast<const float4 *>(turn_at(turn, c, i + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
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

// A quarter of the accumulator's lanes belongs to two warps, which take turns
// of 32 columns.
constexpr int kColumnStep = 32 * (kEpilogueWarps / 4);

// A warp's part of the epilogue.  The accumulator comes with one m per lane
// and one n per register; a turn through shared memory gives each lane 8
// neighbouring m of one n, so that residual, pre and out move 16 bytes at a
// time: kTasks pairs (n, 8 m) per lane and 32 columns, lane l starting at
// column l / kPer and block l % kPer.
template <typename T, Mode MODE> struct Epilogue {
    static constexpr int kPer = MODE == kGated ? 2 : 4;      // 8-blocks of outputs per column
    static constexpr int kTasks = kPer;                      // 32 columns * kPer / 32 lanes
    static constexpr bool kActs = MODE == kForward || MODE == kGated;
    T *out, *pre;
    const T *res;
    int64_t out_stride, pre_stride, res_stride;
    int n, M, lane;
    bool live;                   // this lane's block of outputs is inside
    bool pre_live;
    uint4 next[kTasks];          // residual of the columns to come

    __device__ void start(const ProductParams &p, const Tile &t, int quarter, uint32_t rank, int c0) {
        lane = threadIdx.x & 31;
        n = t.n;
        M = p.M;
        const int64_t own = MODE == kGradW ? t.g : t.seg;
        const int64_t row0 = (MODE == kGradW ? 0 : t.first) + (int64_t)t.n0;
        // outputs of the quarter: 32 m, or 16 features (gated)
        const int m0 = (t.m * 2 + (int)rank) * (MODE == kGated ? 64 : 128) + quarter * kPer * 8;
        const int m = m0 + (lane % kPer) * 8;
        live = m < M;
        out_stride = p.out.row_stride;
        out = static_cast<T *>(p.out.ptr) + own * p.out.rank_stride + (row0 + lane / kPer) * out_stride + m;
        if constexpr (kActs) {
            res_stride = p.residual.row_stride;
            res = p.residual.ptr ? static_cast<const T *>(p.residual.ptr) + own * p.residual.rank_stride +
                                       (row0 + lane / kPer) * res_stride + m
                                 : nullptr;
            // pre: four 8-blocks of accumulator lanes per column; gated: gate, up, gate, up
            const int block = lane & 3;
            const int64_t pm = MODE == kGated ? m0 + (block >> 1) * 8 + (block & 1) * (int64_t)M : m;
            pre_live = MODE == kGated ? m0 + (block >> 1) * 8 < M : live;
            pre_stride = p.pre.row_stride;
            pre = p.pre.ptr ? static_cast<T *>(p.pre.ptr) + own * p.pre.rank_stride +
                                  (row0 + lane / 4) * pre_stride + pm
                            : nullptr;
            fetch(c0);
        }
    }
    __device__ void fetch(int c0) {
        if (!kActs || !res) return;
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            const int c = c0 + i * (32 / kPer);
            next[i] = live && c + lane / kPer < n ? *reinterpret_cast<const uint4 *>(res + c * res_stride)
                                                  : make_uint4(0, 0, 0, 0);
        }
    }
    // v: 32 columns from c0 on of this lane's m, bias added.
    __device__ void columns(const ProductParams &p, float *turn, const float *v, int c0) {
        uint4 r[kTasks];
#pragma unroll
        for (int i = 0; i < kTasks; ++i) r[i] = next[i];
        if (c0 + kColumnStep < n) fetch(c0 + kColumnStep);
#pragma unroll
        for (int c = 0; c < 32; ++c) *turn_at(turn, c, lane) = v[c];
        __syncwarp();
        if (kActs && MODE == kGated && pre) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = i * 8 + lane / 4;
                float f[8];
                read8(f, turn, c, (lane & 3) * 8);
                if (pre_live && c0 + c < n) store8<T>(pre + (c0 + i * 8) * pre_stride, f);
            }
        }
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            const int c = i * (32 / kPer) + lane / kPer;
            const bool in = live && c0 + c < n;
            float f[8];
            if constexpr (MODE == kGated) {
                float up[8];
                read8(f, turn, c, (lane & 1) * 16);
                read8(up, turn, c, (lane & 1) * 16 + 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = f[j] * sigmoidf(f[j]) * up[j];
            } else {
                read8(f, turn, c, (lane & 3) * 8);
                if constexpr (MODE == kForward) {
                    if (pre && in) store8<T>(pre + (c0 + i * 8) * pre_stride, f);
                    activate8(p.act, f);
                }
            }
            if (kActs && res) add8<T>(f, r[i]);
            if (in) store8<T>(out + (c0 + i * (32 / kPer)) * out_stride, f);
        }
        __syncwarp();
    }
};

// One product's inputs and outputs.
struct Work {
    CUtensorMap a, b, b32;   // b32: rows of a K-major B, 32 at a time
    ProductParams p;
};

// What the roles share.  A role works through one product's tiles after the
// other's and carries its place in the ring and in the accumulators along;
// `next` is this pair's next tile, counted from the product's first.
struct Cta {
    Barriers *bars;
    uint32_t ring, tmem, rank;
    float *turns;
    int64_t pairs;
    volatile Watch *watch;

    static __device__ uint32_t bar(uint64_t *b) { return smem_u32(b); }
    static __device__ uint32_t first_cta(uint64_t *b) { return in_cta(smem_u32(b), 0); }
};

template <Mode MODE> struct Shape {
    static constexpr bool kAmn = MODE == kGradX || MODE == kGradW, kBmn = MODE == kGradW;
    static constexpr int kFeat = MODE == kGated ? kTileM : 2 * kTileM;     // outputs along m per tile
    static __device__ int m_tiles(const ProductParams &p) { return (p.M + kFeat - 1) / kFeat; }
};

__device__ __forceinline__ void advance(uint32_t &s, uint32_t &phase) {
    if (++s == kStages) {
        s = 0;
        phase ^= 1u;
    }
}

// ---- warp 0 of each CTA: copies

struct Loader {
    uint32_t issued = 0, s = 0, phase = 0;    // slices; the next one's stage and its round's parity
    uint32_t tails = 0, landed = 0;           // by stage: a tail was loaded, its barrier's phase
    int64_t next;

    template <Mode MODE> __device__ bool run(const Cta &c, const Work &w) {
        constexpr bool kAmn = Shape<MODE>::kAmn, kBmn = Shape<MODE>::kBmn;
        Barriers &bars = *c.bars;
        const ProductParams &p = w.p;
        const bool elected = elect_one();
        const uint32_t full0 = c.first_cta(&bars.full[0]);
        const int mt = Shape<MODE>::m_tiles(p);
        bool ok = true;
        Walker walk;
        Tile t;
        walk.start(p, mt);
        for (; ok && walk.find(p, mt, next, &t); next += c.pairs) {
            const int K = p.K < 0 ? t.rows : p.K;
            const int half = ((t.n + 31) & ~31) / 2;      // this CTA's n
            // rows of B: one copy of 128, or up to three of 32
            const bool narrow = !kBmn && half <= 96;
            const int boxes = kBmn ? (half + 63) / 64 : narrow ? (half + 31) / 32 : 1;
            const uint32_t box = narrow ? kHalfBytes / 4 : kHalfBytes;
            const CUtensorMap *mb = narrow ? &w.b32 : &w.b;
            const int m0 = (t.m * 2 + (int)c.rank) * kTileM, n0 = t.n0 + (int)c.rank * half;
            for (int k = 0; k < K; k += kSliceK) {
                if (!tensor_wait(c.bar(&bars.empty[s]), phase ^ 1u, c.watch)) {
                    ok = false;
                    break;
                }
                if (elected) {
                    const int halves = K - k > 64 ? 2 : 1;        // of a K-major operand
                    const uint32_t bytes = (kAmn ? 2 : halves) * kHalfBytes + (kBmn ? 1 : halves) * boxes * box;
                    // the second CTA clears the rows past a group's end before
                    // it tells the first: that slice lands on its own barrier
                    const bool last = MODE == kGradW && K - k < kSliceK, tail = last && c.rank == 1;
                    const uint32_t full = tail ? in_cta(c.bar(&bars.tail[s]), 1) : full0 + s * 8;
                    const uint32_t a = c.ring + s * kStageBytes, b = a + kBytesA;
                    if (c.rank == 0) mbar_expect(c.bar(&bars.full[s]), last ? bytes : 2 * bytes);
                    if (tail) mbar_expect(c.bar(&bars.tail[s]), bytes);
                    if constexpr (kAmn) {
                        const int row = MODE == kGradW ? t.first + k : k;
                        const int own = MODE == kGradW ? t.seg : t.g;
                        tma_load3(a, &w.a, full, m0, row, own);
                        tma_load3(a + kHalfBytes, &w.a, full, m0 + 64, row, own);
                    }
                    if constexpr (kBmn) {
                        for (int j = 0; j < boxes; ++j)
                            tma_load3(b + j * kHalfBytes, mb, full, n0 + j * 64, t.first + k, t.seg);
                    }
                    for (int h = 0; h < halves; ++h) {
                        if constexpr (MODE == kGated)
                            tma_load5(a + h * kHalfBytes, &w.a, full, k + h * 64, 0, 0, m0 / 16, t.g);
                        else if constexpr (!kAmn)
                            tma_load3(a + h * kHalfBytes, &w.a, full, k + h * 64, m0, t.g);
                        if constexpr (!kBmn)
                            for (int j = 0; j < boxes; ++j)
                                tma_load3(b + h * kHalfBytes + j * box, mb, full, k + h * 64, t.first + n0 + j * 32,
                                          t.seg);
                    }
                }
                if (MODE == kGradW && c.rank == 1 && K - k < kSliceK) {
                    if (tails >> s & 1u) landed ^= 1u << s;
                    tails |= 1u << s;
                }
                ++issued;
                if (elected) c.watch->loaded = issued;
                advance(s, phase);
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        next -= walk.before;
        return ok;
    }

    // The pair ends together, and not before its copies have landed and the
    // stages' last signals have come; after a wait that ran out, as far as they
    // come within another wait each.
    __device__ void finish(const Cta &c, bool ok) {
        if ((threadIdx.x & 31) == 0) {
            Barriers &bars = *c.bars;
            Watch ignore = {};
            volatile Watch *watch = ok ? c.watch : &ignore;
            for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j) {
                const uint32_t q = j % kStages, round = (j / kStages) & 1u;
                if (!ok && c.rank == 0) tensor_wait(c.bar(&bars.full[q]), round, watch);
                if (!ok && c.rank == 1 && (tails >> q & 1u))
                    tensor_wait(c.bar(&bars.tail[q]), landed >> q & 1u, watch);
                tensor_wait(c.bar(&bars.empty[q]), round, watch);
            }
        }
        __syncwarp();
    }
};

// ---- warp 1 of the first CTA: matrix instructions

struct Multiplier {
    uint32_t s = 0, phase = 0, acc = 0, tails = 0;
    int64_t next;

    template <typename T, Mode MODE> __device__ bool run(const Cta &c, const Work &w) {
        constexpr bool kAmn = Shape<MODE>::kAmn, kBmn = Shape<MODE>::kBmn;
        constexpr uint32_t kIdesc = f16_idesc(IsBf16<T>::value, kAmn, kBmn, 2 * kTileM);
        Barriers &bars = *c.bars;
        const ProductParams &p = w.p;
        const bool elected = elect_one();
        // descriptors; step j is 16 k on: 32 bytes of a row and the other half
        // after four (K-major), or 16 rows (MN-major)
        const uint64_t a0 = smem_desc(c.ring, kAmn ? kHalfBytes : 16, 1024);
        const uint64_t b0 = smem_desc(c.ring + kBytesA, kBmn ? kHalfBytes : 16, 1024);
        auto step = [](bool mn, int j) -> uint64_t {
            return (mn ? j * 2048 : j / 4 * kHalfBytes + j % 4 * 32) >> 4;
        };
        const int mt = Shape<MODE>::m_tiles(p);
        bool ok = true;
        Walker walk;
        Tile t;
        walk.start(p, mt);
        for (; ok && walk.find(p, mt, next, &t); next += c.pairs) {
            const int K = p.K < 0 ? t.rows : p.K;
            const int n = (t.n + 31) & ~31;
            if (K == 0) continue;
            const uint32_t idesc = kIdesc | idesc_n(n);
            const uint32_t d = c.tmem + (acc & 1u) * 256;
            ok = warp_wait<true>(c.bar(&bars.acc_empty[acc & 1u]), ((acc >> 1) & 1u) ^ 1u, c.watch);
            tcgen_after_sync();
            // One thread issues everything, and has to queue the next slice's
            // instructions before the last one's end: the loop is kept short.
            const int end = !ok ? 0 : MODE == kGradW ? K / kSliceK * kSliceK : K;
            for (int k = 0; k < end; k += kSliceK) {
                if (!tensor_wait(c.bar(&bars.full[s]), phase, c.watch)) {
                    ok = false;
                    break;
                }
                if (elected) {
                    const uint64_t da = a0 + s * (kStageBytes >> 4), db = b0 + s * (kStageBytes >> 4);
#pragma unroll
                    for (int j = 0; j < kSliceK / 16; ++j)
                        if (j == 0 || k + j * 16 < K)
                            mma_f16(d, da + step(kAmn, j), db + step(kBmn, j), idesc, k > 0 || j > 0);
                    mma_commit_pair(c.bar(&bars.empty[s]));
                }
                advance(s, phase);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (MODE == kGradW && ok && K % kSliceK) {
                ok = warp_wait(c.bar(&bars.full[s]), phase, c.watch);
                if (ok) {
                    clear_rows(c.ring + s * kStageBytes, 2 + (n / 2 + 63) / 64, K % kSliceK);
                    ok = warp_wait<true>(c.bar(&bars.peer_tail[s]), tails >> s & 1u, c.watch);
                    tails ^= 1u << s;
                }
                if (ok && elected) {
                    const uint64_t da = a0 + s * (kStageBytes >> 4), db = b0 + s * (kStageBytes >> 4);
#pragma unroll
                    for (int j = 0; j < kSliceK / 16; ++j)
                        if (j * 16 < K % kSliceK)
                            mma_f16(d, da + step(kAmn, j), db + step(kBmn, j), idesc, K > kSliceK || j > 0);
                    mma_commit_pair(c.bar(&bars.empty[s]));
                }
                advance(s, phase);
            }
            if (ok && elected) mma_commit_pair(c.bar(&bars.acc_full[acc & 1u]));
            ++acc;
        }
        next -= walk.before;
        return ok;
    }
    __device__ void finish(const Cta &c, bool ok) {
        if (ok) return;                                  // else let the matrix unit finish
        Watch ignore = {};
        if (elect_one()) mma_commit(c.bar(&c.bars->drained));
        tensor_wait(c.bar(&c.bars->drained), 0, &ignore);
    }
};

// ---- warp 1 of the second CTA: clears its part of a group's last rows

struct Clearer {
    uint32_t slice = 0, tails = 0;
    int64_t next;

    template <Mode MODE> __device__ bool run(const Cta &c, const Work &w) {
        Barriers &bars = *c.bars;
        const ProductParams &p = w.p;
        const int mt = Shape<MODE>::m_tiles(p);
        bool ok = true;
        Walker walk;
        Tile t;
        walk.start(p, mt);
        for (; ok && walk.find(p, mt, next, &t); next += c.pairs) {
            const int K = p.K < 0 ? t.rows : p.K, live = K % kSliceK;
            slice += (K + kSliceK - 1) / kSliceK;
            if (MODE != kGradW || live == 0) continue;
            const int n = (t.n + 31) & ~31;
            const uint32_t s = (slice - 1) % kStages;
            ok = warp_wait(c.bar(&bars.tail[s]), tails >> s & 1u, c.watch);
            if (!ok) break;
            tails ^= 1u << s;
            clear_rows(c.ring + s * kStageBytes, 2 + (n / 2 + 63) / 64, live);
            if ((threadIdx.x & 31) == 0) cluster_arrive(c.first_cta(&bars.peer_tail[s]));
        }
        next -= walk.before;
        return ok;
    }
};

// ---- warps 2..9: outputs

struct Finisher {
    uint32_t acc = 0;
    int64_t next;

    template <typename T, Mode MODE> __device__ bool run(const Cta &c, const Work &w) {
        Barriers &bars = *c.bars;
        const ProductParams &p = w.p;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int quarter = warp & 3;                    // the TMEM lanes this warp may read
        const int c0 = (warp - 2) / 4 * 32;              // its first columns
        float *turn = c.turns + (warp - 2) * (kTurnBytes / 4);
        const int mt = Shape<MODE>::m_tiles(p);
        bool ok = true;
        Epilogue<T, MODE> ep;
        Walker walk;
        Tile t;
        walk.start(p, mt);
        for (; ok && walk.find(p, mt, next, &t); next += c.pairs) {
            const int K = p.K < 0 ? t.rows : p.K, n = t.n;
            ep.start(p, t, quarter, c.rank, c0);
            float bias = 0.f;
            if ((MODE == kForward || MODE == kGated) && p.bias) {
                const int in = quarter * 32 + lane;      // this lane's row of the accumulator
                const int m = (t.m * 2 + (int)c.rank) * (MODE == kGated ? 64 : 128) +
                              (MODE == kGated ? (in >> 4) * 8 + (in & 7) : in);
                const T *b = static_cast<const T *>(p.bias) + (int64_t)t.g * (MODE == kGated ? 2 * p.M : p.M);
                if (m < p.M) bias = f32(b[MODE == kGated && (in & 8) ? p.M + m : m]);
            }
            if (K > 0) {
                ok = warp_wait(c.bar(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, c.watch);
                if (!ok) break;
                tcgen_after_sync();
            }
            const uint32_t d = c.tmem + (acc & 1u) * 256 + ((uint32_t)(quarter * 32) << 16);
            const uint32_t free = c.first_cta(&bars.acc_empty[acc & 1u]);
            if (K > 0 && c0 >= n) {                      // no columns for this warp
                tcgen_before_sync();
                __syncwarp();
                if (lane == 0) cluster_arrive(free);
            }
            for (int col = c0; col < n; col += kColumnStep) {
                uint32_t r[32];
                float v[32];
                if (K > 0) {
                    tmem_load32(d + col, r);
                    tmem_wait(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                if (K > 0 && col + kColumnStep >= n) {   // the accumulator may be filled again
                    tcgen_before_sync();
                    __syncwarp();
                    if (lane == 0) cluster_arrive(free);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) + bias;
                ep.columns(p, turn, v, col);
            }
            if (K > 0) ++acc;
        }
        next -= walk.before;
        return ok;
    }
};

// One product (FIRST), or two in a row (then SECOND), either of which may be
// left out (null).
template <typename T, Mode FIRST, Mode SECOND>
__device__ __forceinline__ void run_products(const Work *first, const Work *second, uint32_t *error) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bars;
    const int warp = threadIdx.x >> 5;
    Cta c;
    c.bars = &bars;
    c.ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    c.turns = reinterpret_cast<float *>(smem_raw + (c.ring - smem_u32(smem_raw)) + kRingBytes);
    c.rank = cluster_rank();
    c.pairs = gridDim.x >> 1;
    c.watch = &bars.watch;
    const int64_t pair = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1);                 // the first CTA's hears of both CTAs' loads
            mbar_init(&bars.empty[i], 1);
            mbar_init(&bars.tail[i], 1);
            mbar_init(&bars.peer_tail[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 2 * kEpilogueWarps);   // both CTAs' epilogue warps
        }
        mbar_init(&bars.drained, 1);
        bars.watch.gave_up = 0;
        bars.watch.loaded = 0;
        mbar_init_fence();
        const Work *w = first ? first : second;
        tma_prefetch_map(&w->a);
        tma_prefetch_map(&w->b);
    }
    __syncwarp();
    cluster_sync();
    if (warp == 1) tmem_alloc(smem_u32(&bars.tmem), 512);
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    c.tmem = bars.tmem;
    // This far while the kernel before ends.  Only then may the next one start
    // to get ready: it may count on all that came before this kernel.
    grid_dependency_wait();
    grid_dependents_may_launch();

    bool ok = true;
    if (warp == 0) {
        Loader r;
        r.next = pair;
        if (first) ok = r.run<FIRST>(c, *first);
        if constexpr (SECOND != kNone)
            if (ok && second) ok = r.run<SECOND>(c, *second);
        r.finish(c, ok);
    } else if (warp == 1 && c.rank == 0) {
        Multiplier r;
        r.next = pair;
        if (first) ok = r.run<T, FIRST>(c, *first);
        if constexpr (SECOND != kNone)
            if (ok && second) ok = r.run<T, SECOND>(c, *second);
        r.finish(c, ok);
    } else if (warp == 1) {
        if constexpr (SECOND != kNone) {
            Clearer r;
            r.next = pair;
            if (first) ok = r.run<FIRST>(c, *first);
            if (ok && second) ok = r.run<SECOND>(c, *second);
        }
    } else {
        Finisher r;
        r.next = pair;
        if (first) ok = r.run<T, FIRST>(c, *first);
        if constexpr (SECOND != kNone)
            if (ok && second) ok = r.run<T, SECOND>(c, *second);
    }
    __syncwarp();
    tcgen_before_sync();
    cluster_sync();              // neither CTA's memory is read or signalled any more
    tcgen_after_sync();
    if (warp == 1) tmem_free(c.tmem, 512);
    if (threadIdx.x == 0 && bars.watch.gave_up && error) atomicOr(error, EP_DEVERR_TIMEOUT);
}

template <typename T, Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Work w) {
    run_products<T, MODE, kNone>(&w, nullptr, w.p.error);
}

// Both gradients in one launch: the pairs that finish grad_x's tiles go on
// with grad_w's.
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gradient_kernel(const __grid_constant__ Work x, const __grid_constant__ Work w, bool has_x, bool has_w) {
    run_products<T, kGradX, kGradW>(has_x ? &x : nullptr, has_w ? &w : nullptr, w.p.error);
}

// d = grad * act'(pre) over every group's rows, and its column sums before it
// is rounded.  d is rounded once to the tensors' 16-bit type, as the operand of
// both products: the matrix instructions take both operands in one type, and a
// 32-bit d would halve their rate and double its traffic.  Next to the inputs'
// own rounding it makes the gradients' error 1.4 times as large.  Bound by memory: grad
// and pre are read once, d is written once.  A block takes 256 features and
// one of `splits` parts of a group's rows; a lane holds 8 features (16 bytes),
// the 8 warps take rows in turn.  Column sums are joined in a fixed order:
// warps in shared memory, parts by sum_parts_kernel.
struct ActGradParams {
    Groups gr;
    int N, act, splits;
    ep_rows_t grad, pre, d;
    float *part;            // [splits][G][wide] column sums, or null
    void *grad_bias;        // [G][wide], with one part a group
    bool write;
};

constexpr int kActWarps = 8, kActCols = 256, kActRows = 4;

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

template <typename T> __device__ __forceinline__ void unpack8(float *v, const uint4 &r) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f32(e[i]);
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kActWarps * 32) act_grad_kernel(const ActGradParams p) {
    __shared__ float sums[kActWarps][GATED ? 2 : 1][kActCols + 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.y, seg = g / p.gr.per, split = blockIdx.z;
    const int c = blockIdx.x * kActCols + lane * 8;
    const bool live = c < p.N;
    int first, rows;
    group_range(p.gr, g, &first, &rows);
    const int per = (rows + p.splits - 1) / p.splits;
    const int r1 = first + min(rows, (split + 1) * per);
    grid_dependents_may_launch();
    const T *grad = static_cast<const T *>(p.grad.ptr) + seg * p.grad.rank_stride + c;
    const T *pre = static_cast<const T *>(p.pre.ptr) + seg * p.pre.rank_stride + c;
    T *d = static_cast<T *>(p.d.ptr) + seg * p.d.rank_stride + c;
    float s0[8] = {}, s1[8] = {};
    const bool reads_pre = p.act != EP_ACT_NONE;
    for (int64_t r = first + split * per + warp; live && r < r1; r += kActWarps * kActRows) {
        uint4 gv[kActRows], v0[kActRows], v1[kActRows];
#pragma unroll
        for (int u = 0; u < kActRows; ++u) {
            const int64_t i = r + u * kActWarps;
            if (i >= r1) continue;
            gv[u] = ld_stream16(grad + i * p.grad.row_stride);
            if (reads_pre) v0[u] = ld_stream16(pre + i * p.pre.row_stride);
            if (GATED) v1[u] = ld_stream16(pre + i * p.pre.row_stride + p.N);
        }
#pragma unroll
        for (int u = 0; u < kActRows; ++u) {
            const int64_t i = r + u * kActWarps;
            if (i >= r1) continue;
            float y[8], v[8], d0[8], d1[8];
            unpack8<T>(y, gv[u]);
            if (GATED) {
                float up[8];
                unpack8<T>(v, v0[u]);
                unpack8<T>(up, v1[u]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = sigmoidf(v[j]);
                    d0[j] = y[j] * up[j] * (s * (1.0f + v[j] * (1.0f - s)));
                    d1[j] = y[j] * v[j] * s;
                    s1[j] += d1[j];
                }
            } else if (reads_pre) {
                unpack8<T>(v, v0[u]);
#pragma unroll
                for (int j = 0; j < 8; ++j) d0[j] = act_grad(p.act, y[j], v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d0[j] = y[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s0[j] += d0[j];
            if (p.write) {
                store8<T>(d + i * p.d.row_stride, d0);
                if (GATED) store8<T>(d + i * p.d.row_stride + p.N, d1);
            }
        }
    }
    if (!p.part && !p.grad_bias) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sums[warp][0][lane * 8 + j] = s0[j];
        if (GATED) sums[warp][GATED ? 1 : 0][lane * 8 + j] = s1[j];
    }
    __syncthreads();
    const int64_t G = (int64_t)p.gr.R * p.gr.per, wide = GATED ? 2 * (int64_t)p.N : p.N;
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const int col = blockIdx.x * kActCols + threadIdx.x;
        float s = 0.f;
        for (int w = 0; w < kActWarps; ++w) s += sums[w][h][threadIdx.x];
        if (col >= p.N) continue;
        if (p.part) p.part[(split * G + g) * wide + h * (int64_t)p.N + col] = s;
        else static_cast<T *>(p.grad_bias)[g * wide + h * (int64_t)p.N + col] = rounded<T>(s);
    }
}

// grad_bias = the parts' sums, in order.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float *part, int splits, int64_t n, T *out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += part[k * n + i];
    out[i] = rounded<T>(s);
}

// Parts of a group's rows in act_grad_kernel: about 64 rows each, going by
// the average group, at most 32.
int act_splits(const ep_product_desc_t &d) {
    const int64_t average = d.rows / d.groups;
    const int64_t parts = (average + 63) / 64;
    return (int)(parts < 1 ? 1 : parts > 32 ? 32 : parts);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of `width` elements: 16-byte aligned, dense rows that do not overlap.
bool valid_rows(const ep_rows_t &r, int64_t width, bool many) {
    return r.ptr && aligned(r.ptr, 16) && r.row_stride >= width && r.row_stride % 8 == 0 &&
           (!many || (r.rank_stride > 0 && r.rank_stride % 8 == 0));
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

// ---- tensor maps

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::atomic<EncodeFn> cached{nullptr};
    EncodeFn f = cached.load(std::memory_order_acquire);
    if (!f) {
        void *sym = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeFn>(sym);
        cached.store(f, std::memory_order_release);
    }
    return f;
}

bool encode(CUtensorMap *map, int dtype, void *ptr, int rank, const uint64_t *dims, const int64_t *strides,
            const uint32_t *box) {
    EncodeFn f = encode_fn();
    if (!f) return false;
    cuuint64_t d[5], s[5];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i) s[i - 1] = (cuuint64_t)strides[i] * 2;
    }
    return f(map, dtype == EP_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             (cuuint32_t)rank, ptr, d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [outer][rows][width] with boxes of 64 elements by `box_rows` rows.  Reads
// past an edge give zeros.
bool encode_rows(CUtensorMap *map, int dtype, const ep_rows_t &r, int64_t width, int64_t rows, int64_t outer,
                 uint32_t box_rows) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)rows, (uint64_t)outer};
    const int64_t strides[3] = {1, r.row_stride, outer > 1 ? r.rank_stride : r.row_stride};
    const uint32_t box[3] = {64, box_rows, 1};
    return encode(map, dtype, r.ptr, 3, dims, strides, box);
}

// Gated weights [G][2][N][K]: one box is 8 features of the gate, the same 8
// of the up half, and so on for 64 features.
bool encode_gated(CUtensorMap *map, int dtype, const ep_rows_t &w, int64_t K, int64_t N, int64_t G) {
    const uint64_t dims[5] = {(uint64_t)K, 8, 2, (uint64_t)(N / 8), (uint64_t)G};
    const int64_t strides[5] = {1, w.row_stride, N * w.row_stride, 8 * w.row_stride,
                                G > 1 ? w.rank_stride : w.row_stride};
    const uint32_t box[5] = {64, 8, 2, 8, 1};
    return encode(map, dtype, w.ptr, 5, dims, strides, box);
}

// ---- launch

constexpr int kMaxDevices = 64;

int sm_count(int dev) {
    static std::atomic<int> cached[kMaxDevices];
    int n = cached[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Tiles of `columns` columns at most: every group's last tile may be a part.
template <Mode MODE> int64_t most_tiles(const ProductParams &p, int columns) {
    const int64_t mt = (p.M + Shape<MODE>::kFeat - 1) / Shape<MODE>::kFeat;
    const int64_t G = (int64_t)p.gr.R * p.gr.per;
    return mt * (p.N < 0 ? (int64_t)p.gr.R * p.gr.rows / columns + G : G * ((p.N + columns - 1) / columns));
}

// Full tiles, or narrower ones while those still find a pair of SMs each: they
// load more for the same work, but outputs (most of a short tile's time) are
// finished by more SMs.  2670 rows of 4 groups x 1688 -> 96 with gelu and
// residual: 12 tiles 21.7 us, 43 tiles 12.6 us; past one tile a pair it turns
// (9448 rows of 24 groups x 120 -> 64 gated: 8.9 us, in two rounds 10.8).
template <Mode MODE> int64_t choose_tile(ProductParams &p, int64_t pairs) {
    p.tile_n = kTileN;
    while (p.tile_n > 64 && most_tiles<MODE>(p, p.tile_n / 2) <= pairs) p.tile_n /= 2;
    return most_tiles<MODE>(p, p.tile_n);
}

// One CTA per SM, in pairs, as a programmatic dependent of the kernel before.
template <typename... Params, typename... Args>
ep_status_t launch_pairs(int dev, std::atomic<bool> *configured, void (*kernel)(Params...), int64_t grid,
                         cudaStream_t st, Args &&...args) {
    if (!configured[dev].load(std::memory_order_acquire)) {        // the attribute is per device
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) != cudaSuccess)
            return EP_ERR_GPU_OP;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_after_previous(kernel, 2 * (unsigned)grid, kThreads, kSmemBytes, st, static_cast<Args &&>(args)...) ==
                   cudaSuccess
               ? EP_SUCCESS : EP_ERR_GPU_OP;
}

// The current device and its pairs of SMs; 0 when there is none.
int device_pairs(int *dev) {
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return 0;
    return sm_count(*dev) / 2;
}

template <typename T, Mode MODE> ep_status_t launch_product(Work &w, cudaStream_t st) {
    static std::atomic<bool> configured[kMaxDevices];
    int dev;
    const int pairs = device_pairs(&dev);
    if (pairs < 1) return EP_ERR_GPU_OP;
    const int64_t tiles = choose_tile<MODE>(w.p, pairs);
    return launch_pairs(dev, configured, product_kernel<T, MODE>, tiles < pairs ? tiles : pairs, st, w);
}
template <typename T>
ep_status_t launch_gradients(Work &x, Work &w, bool has_x, bool has_w, cudaStream_t st) {
    static std::atomic<bool> configured[kMaxDevices];
    int dev;
    const int pairs = device_pairs(&dev);
    if (pairs < 1) return EP_ERR_GPU_OP;
    int64_t tiles = has_x ? choose_tile<kGradX>(x.p, has_w ? pairs / 2 : pairs) : 0;
    if (has_w) tiles += choose_tile<kGradW>(w.p, pairs - tiles);
    return launch_pairs(dev, configured, gradient_kernel<T>, tiles < pairs ? tiles : pairs, st, x, w, has_x, has_w);
}

// The gradient's workspace: d in the tensors' type (not needed where act' is
// 1), then the parts of the bias gradient.
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t rounded_d_bytes(const ep_product_desc_t &d) {
    return d.activation == EP_ACT_NONE ? 0 : align256((size_t)d.ranks * d.rows * (size_t)wide_of(d) * 2);
}
size_t part_bytes(const ep_product_desc_t &d) {
    return align256((size_t)act_splits(d) * d.ranks * d.groups * (size_t)wide_of(d) * 4);
}

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
    Work w = {};
    ProductParams &p = w.p;
    p.gr = groups_of(*d);
    p.M = d->out_features;
    p.N = -1;
    p.K = d->in_features;
    p.act = d->activation;
    p.bias = d_bias;
    p.residual = *residual;
    p.out = *y;
    p.pre = *pre;
    p.error = d_error;
    const bool gated = d->activation == EP_ACT_SWIGLU, bf16 = d->dtype == EP_DT_BF16;
    const int64_t G = (int64_t)d->ranks * d->groups;
    if (!(gated ? encode_gated(&w.a, d->dtype, d->weight, p.K, p.M, G)
                : encode_rows(&w.a, d->dtype, d->weight, p.K, p.M, G, kTileM)) ||
        !encode_rows(&w.b, d->dtype, d->x, p.K, d->rows, d->ranks, kTileN / 2) ||
        !encode_rows(&w.b32, d->dtype, d->x, p.K, d->rows, d->ranks, 32))
        return EP_ERR_GPU_OP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (gated) return bf16 ? launch_product<__nv_bfloat16, kGated>(w, st) : launch_product<__half, kGated>(w, st);
    return bf16 ? launch_product<__nv_bfloat16, kForward>(w, st) : launch_product<__half, kForward>(w, st);
}

ep_status_t ep_expert_product_workspace(const ep_product_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = rounded_d_bytes(*d) + part_bytes(*d);
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
    const int splits = act_splits(*d);
    const int64_t G = (int64_t)d->ranks * d->groups;
    float *part = d_grad_bias && splits > 1
                      ? reinterpret_cast<float *>(static_cast<char *>(d_workspace) + rounded_d_bytes(*d)) : nullptr;
    if (act || d_grad_bias) {
        const ActGradParams q = {gr, d->out_features, d->activation, splits, *grad, *pre, dd, part,
                                 part ? nullptr : d_grad_bias, act};
        const dim3 grid((d->out_features + kActCols - 1) / kActCols, (unsigned)G, splits);
        with_type(d->dtype, [&](auto type) {
            using T = decltype(type);
            if (d->activation == EP_ACT_SWIGLU) act_grad_kernel<T, true><<<grid, kActWarps * 32, 0, st>>>(q);
            else act_grad_kernel<T, false><<<grid, kActWarps * 32, 0, st>>>(q);
        });
    }
    const bool has_x = grad_x->ptr && d->rows > 0, has_w = d_grad_w && d->rows > 0;
    if (has_x || has_w) {
        Work x = {}, w = {};
        x.p.gr = gr;
        x.p.M = d->in_features;
        x.p.N = -1;
        x.p.K = (int)wide;
        x.p.out = *grad_x;
        w.p.gr = gr;
        w.p.M = d->in_features;
        w.p.N = (int)wide;
        w.p.K = -1;
        w.p.out = ep_rows_t{d_grad_w, wide * d->in_features, d->in_features};
        x.p.error = w.p.error = d_error;
        if ((has_x && (!encode_rows(&x.a, d->dtype, d->weight, d->in_features, wide, G, kSliceK) ||
                       !encode_rows(&x.b, d->dtype, dd, wide, d->rows, d->ranks, kTileN / 2) ||
                       !encode_rows(&x.b32, d->dtype, dd, wide, d->rows, d->ranks, 32))) ||
            (has_w && (!encode_rows(&w.a, d->dtype, d->x, d->in_features, d->rows, d->ranks, kSliceK) ||
                       !encode_rows(&w.b, d->dtype, dd, wide, d->rows, d->ranks, kSliceK))))
            return EP_ERR_GPU_OP;
        const ep_status_t s = d->dtype == EP_DT_BF16 ? launch_gradients<__nv_bfloat16>(x, w, has_x, has_w, st)
                                                     : launch_gradients<__half>(x, w, has_x, has_w, st);
        if (s != EP_SUCCESS) return s;
    } else if (d_grad_w) {
        if (cudaMemsetAsync(d_grad_w, 0, (size_t)G * wide * d->in_features * 2, st) != cudaSuccess)
            return EP_ERR_GPU_OP;
    }
    if (part)
        with_type(d->dtype, [&](auto type) {
            using T = decltype(type);
            const int64_t n = G * wide;
            sum_parts_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(part, splits, n,
                                                                             static_cast<T *>(d_grad_bias));
        });
    return launched();
}

}  // extern "C"
