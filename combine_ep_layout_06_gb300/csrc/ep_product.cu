// Expert products: one matrix product per group of rows, with bias,
// activation and residual in its epilogue, and its gradient.
//
// Every product here is  out[n][m] = sum_k A[m][k] * B[n][k]  over one group:
//   forward   m = feature, n = row,   k = input    A = weight,    B = x
//   grad_x    m = input,   n = row,   k = feature  A = weight^T,  B = d
//   grad_w    m = input,   n = feature, k = row    A = x^T,       B = d^T
// The output's contiguous dimension is always m.
//
// One CTA per SM walks the tiles of all groups (their row counts are on the
// device): 128 m by up to 256 n, accumulated in tensor memory.  Weights or
// inputs are the 128-wide operand and rows (or features) the other, so that a
// group with few rows costs a narrow instruction (n in steps of 16) and not a
// padded tile of 128 rows.  Warp 0 loads 64-deep slices by TMA into a ring in
// shared memory, warp 1 issues the matrix instructions, warps 2..5 turn a
// finished accumulator into outputs while the next one fills: two
// accumulators of 256 columns take all of the SM's tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kTileM = 128, kTileN = 256, kSliceK = 64;
constexpr int kStages = 4;
constexpr int kBytesA = kTileM * kSliceK * 2, kBytesB = kTileN * kSliceK * 2;
constexpr int kStageBytes = kBytesA + kBytesB;
constexpr int kChunkBytes = 64 * kSliceK * 2;      // 64 rows (or 64 columns) of one slice
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + 1024;
constexpr int kThreads = 192;

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

enum Mode { kForward, kGated, kGradX, kGradW };

struct ProductParams {
    Groups gr;
    int M, N, K;           // N or K < 0: the group's number of rows
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

__device__ __forceinline__ float sigmoidf(float v) { return 1.0f / (1.0f + expf(-v)); }

template <typename T> struct IsBf16 { static constexpr bool value = false; };
template <> struct IsBf16<__nv_bfloat16> { static constexpr bool value = true; };

// Walks the tiles of all groups in order, 32 groups at a time: a lane holds
// one group's range and the running number of tiles.  Every lane of the warp
// gets the same answer.
struct Tile {
    int g, seg, first, rows, m, n;
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
            tiles = mt * (((p.N < 0 ? rows : p.N) + kTileN - 1) / kTileN);
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
        t->m = in % mt;
        t->n = in / mt;
        return true;
    }
};

struct __align__(8) Barriers {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int gave_up;
};

// The epilogue of 32 columns (rows, or features of grad_w) of one lane's m.
template <typename T, Mode MODE>
__device__ __forceinline__ void store_columns(const ProductParams &p, const Tile &t, float *v, int c0,
                                              int columns, int m, bool live, float b0, float b1) {
    const int64_t own = MODE == kGradW ? t.g : t.seg;
    const int64_t row0 = (MODE == kGradW ? 0 : t.first) + t.n * (int64_t)kTileN + c0;
    T *out = static_cast<T *>(p.out.ptr) + own * p.out.rank_stride + row0 * p.out.row_stride + m;
    if constexpr (MODE == kGradX || MODE == kGradW) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (live && c < columns) out[c * p.out.row_stride] = rounded<T>(v[c]);
    } else {
        const T *res = static_cast<const T *>(p.residual.ptr) + own * p.residual.rank_stride +
                       row0 * p.residual.row_stride + m;
        T *pre = static_cast<T *>(p.pre.ptr) + own * p.pre.rank_stride + row0 * p.pre.row_stride + m;
        if constexpr (MODE == kForward) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] += b0;
            if (p.pre.ptr) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (live && c < columns) pre[c * p.pre.row_stride] = rounded<T>(v[c]);
            }
            switch (p.act) {
            case EP_ACT_RELU:
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = fmaxf(v[c], 0.f);
                break;
            case EP_ACT_GELU:
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = 0.5f * v[c] * (1.0f + erff(v[c] * 0.70710678118654752f));
                break;
            case EP_ACT_SILU:
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] *= sigmoidf(v[c]);
                break;
            default: break;
            }
            if (p.residual.ptr) {
                float r[32];
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    r[c] = live && c < columns ? f32(res[c * p.residual.row_stride]) : 0.f;
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] += r[c];
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (live && c < columns) out[c * p.out.row_stride] = rounded<T>(v[c]);
        } else {
            // Lanes 0-7 and 16-23 hold the gate of 8 features, lanes 8-15 and
            // 24-31 their up half.  Of two rows, the gate's lane finishes the
            // first and the up half's lane the second: one exchange for both.
            const bool up = (threadIdx.x & 8) != 0;
            const int64_t half = up ? p.M : 0;
            const float bias = up ? b1 : b0;
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] += bias;
            if (p.pre.ptr) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (live && c < columns) pre[c * p.pre.row_stride + half] = rounded<T>(v[c]);
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                const float other = __shfl_xor_sync(0xffffffffu, up ? v[c] : v[c + 1], 8);
                const float gate = up ? other : v[c], lin = up ? v[c + 1] : other;
                float y = gate * sigmoidf(gate) * lin;
                const int mine = up ? c + 1 : c;
                if (live && mine < columns) {
                    if (p.residual.ptr) y += f32(res[mine * p.residual.row_stride]);
                    out[mine * p.out.row_stride] = rounded<T>(y);
                }
            }
        }
    }
}

template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_b16, const ProductParams p) {
    constexpr bool kAmn = MODE == kGradX || MODE == kGradW, kBmn = MODE == kGradW;
    constexpr int kFeat = MODE == kGated ? kTileM / 2 : kTileM;     // outputs along m per tile
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bars;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *gave_up = &bars.gave_up;
    auto bar = [](uint64_t *b) { return smem_u32(b); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 4);
        }
        mbar_init(&bars.drained, 1);
        bars.gave_up = 0;
        mbar_init_fence();
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 1) tmem_alloc(smem_u32(&bars.tmem), 512);
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    const uint32_t tmem = bars.tmem;

    const int mt = (p.M + kFeat - 1) / kFeat;
    Walker walk;
    Tile t;
    walk.start(p, mt);
    bool ok = true;

    if (warp == 0) {
        uint32_t issued = 0;
        for (int64_t i = blockIdx.x; ok && walk.find(p, mt, i, &t); i += gridDim.x) {
            const int N = p.N < 0 ? t.rows : p.N, K = p.K < 0 ? t.rows : p.K;
            const int n = min(kTileN, N - t.n * kTileN);
            const bool narrow = !kBmn && n <= 48;         // 16-row boxes: at most 3 loads either way
            const int boxes = narrow ? (n + 15) / 16 : (n + 63) / 64;
            const uint32_t box = narrow ? kChunkBytes / 4 : kChunkBytes;
            if (lane == 0) {
                for (int k = 0; k < K; k += kSliceK) {
                    const uint32_t s = issued % kStages, round = issued / kStages;
                    if (!tensor_wait(bar(&bars.empty[s]), (round & 1u) ^ 1u, gave_up)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = bar(&bars.full[s]);
                    const uint32_t a = ring + s * kStageBytes, b = a + kBytesA;
                    mbar_expect(full, kBytesA + boxes * box);
                    if constexpr (MODE == kGated) {
                        tma_load5(a, &map_a, full, k, 0, 0, t.m * (kFeat / 8), t.g);
                    } else if constexpr (!kAmn) {
                        tma_load3(a, &map_a, full, k, t.m * kTileM, t.g);
                    } else {
                        const int row = MODE == kGradW ? t.first + k : k;
                        const int own = MODE == kGradW ? t.seg : t.g;
                        tma_load3(a, &map_a, full, t.m * kTileM, row, own);
                        tma_load3(a + kChunkBytes, &map_a, full, t.m * kTileM + 64, row, own);
                    }
                    for (int j = 0; j < boxes; ++j) {
                        if constexpr (kBmn)
                            tma_load3(b + j * kChunkBytes, &map_b, full, t.n * kTileN + j * 64, t.first + k, t.seg);
                        else
                            tma_load3(b + j * box, narrow ? &map_b16 : &map_b, full, k,
                                      t.first + t.n * kTileN + j * (narrow ? 16 : 64), t.seg);
                    }
                    ++issued;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // after a wait that ran out: no copy may outlive the CTA
        if (!ok && lane == 0)
            for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j) {
                int ignore = 0;
                tensor_wait(bar(&bars.full[j % kStages]), (j / kStages) & 1u, &ignore);
            }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t kIdesc = f16_idesc(sizeof(T) == 2 && IsBf16<T>::value, kAmn, kBmn, kTileM);
        uint32_t slice = 0, acc = 0;
        for (int64_t i = blockIdx.x; ok && walk.find(p, mt, i, &t); i += gridDim.x) {
            const int N = p.N < 0 ? t.rows : p.N, K = p.K < 0 ? t.rows : p.K;
            const int n = min(kTileN, N - t.n * kTileN);
            if (K == 0) continue;
            const uint32_t idesc = kIdesc | idesc_n((n + 15) & ~15);
            const uint32_t d = tmem + (acc & 1u) * 256;
            ok = warp_wait(bar(&bars.acc_empty[acc & 1u]), ((acc >> 1) & 1u) ^ 1u, gave_up);
            tcgen_after_sync();
            for (int k = 0; ok && k < K; k += kSliceK, ++slice) {
                const uint32_t s = slice % kStages;
                ok = warp_wait(bar(&bars.full[s]), (slice / kStages) & 1u, gave_up);
                if (!ok) break;
                tcgen_after_sync();
                const uint32_t a = ring + s * kStageBytes, b = a + kBytesA;
                if (MODE == kGradW && K - k < kSliceK) {
                    // rows past the group's end: zero, whatever they held (the
                    // 128-byte swizzle moves data within a k row only)
                    const int live = K - k, chunks = 2 + (n + 63) / 64;
                    for (int q = lane; q < chunks * (kSliceK - live) * 8; q += 32) {
                        const int chunk = q / ((kSliceK - live) * 8), r = q % ((kSliceK - live) * 8);
                        const uint32_t at = (chunk < 2 ? a + chunk * kChunkBytes : b + (chunk - 2) * kChunkBytes) +
                                            live * 128 + r * 16;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" :: "r"(at), "r"(0) : "memory");
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < kSliceK / 16; ++j) {
                        const uint64_t da = kAmn ? smem_desc(a + j * 2048, kChunkBytes, 1024)
                                                 : smem_desc(a + j * 32, 16, 1024);
                        const uint64_t db = kBmn ? smem_desc(b + j * 2048, kChunkBytes, 1024)
                                                 : smem_desc(b + j * 32, 16, 1024);
                        mma_f16(d, da, db, idesc, k > 0 || j > 0);
                    }
                    mma_commit(bar(&bars.empty[s]));
                    if (k + kSliceK >= K) mma_commit(bar(&bars.acc_full[acc & 1u]));
                }
                __syncwarp();
            }
            ++acc;
        }
        if (!ok) {                                       // let the matrix unit finish
            int ignore = 0;
            if (lane == 0) mma_commit(bar(&bars.drained));
            tensor_wait(bar(&bars.drained), 0, &ignore);
        }
    } else {
        const int quarter = warp & 3;                    // the TMEM lanes this warp may read
        uint32_t acc = 0;
        for (int64_t i = blockIdx.x; ok && walk.find(p, mt, i, &t); i += gridDim.x) {
            const int N = p.N < 0 ? t.rows : p.N, K = p.K < 0 ? t.rows : p.K;
            const int n = min(kTileN, N - t.n * kTileN);
            // this lane's output index along m
            const int in = quarter * 32 + lane;
            const int m = t.m * kFeat + (MODE == kGated ? (in >> 4) * 8 + (in & 7) : in);
            const bool live = m < p.M;
            float b0 = 0.f, b1 = 0.f;
            if ((MODE == kForward || MODE == kGated) && p.bias && live) {
                const T *bias = static_cast<const T *>(p.bias) + (int64_t)t.g * (MODE == kGated ? 2 * p.M : p.M);
                b0 = f32(bias[m]);
                if (MODE == kGated) b1 = f32(bias[p.M + m]);
            }
            if (K > 0) {
                ok = warp_wait(bar(&bars.acc_full[acc & 1u]), (acc >> 1) & 1u, gave_up);
                if (!ok) break;
                tcgen_after_sync();
            }
            const uint32_t d = tmem + (acc & 1u) * 256 + ((uint32_t)(quarter * 32) << 16);
            for (int c = 0; c < n; c += 32) {
                float v[32];
                if (K > 0) {
                    __syncwarp();
                    tmem_load32(d + c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                }
                if (K > 0 && c + 32 >= n) {              // the accumulator may be filled again
                    tcgen_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(&bars.acc_empty[acc & 1u]));
                }
                store_columns<T, MODE>(p, t, v, c, n - c, m, live, b0, b1);
            }
            if (K > 0) ++acc;
        }
    }
    tcgen_before_sync();
    __syncthreads();
    tcgen_after_sync();
    if (warp == 1) tmem_free(tmem, 512);
    if (threadIdx.x == 0 && bars.gave_up && p.error) atomicOr(p.error, EP_DEVERR_TIMEOUT);
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
    const uint32_t box[3] = {kSliceK, box_rows, 1};
    return encode(map, dtype, r.ptr, 3, dims, strides, box);
}

// Gated weights [G][2][N][K]: one box is 8 features of the gate, the same 8
// of the up half, and so on for 64 features.
bool encode_gated(CUtensorMap *map, int dtype, const ep_rows_t &w, int64_t K, int64_t N, int64_t G) {
    const uint64_t dims[5] = {(uint64_t)K, 8, 2, (uint64_t)(N / 8), (uint64_t)G};
    const int64_t strides[5] = {1, w.row_stride, N * w.row_stride, 8 * w.row_stride,
                                G > 1 ? w.rank_stride : w.row_stride};
    const uint32_t box[5] = {kSliceK, 8, 2, 8, 1};
    return encode(map, dtype, w.ptr, 5, dims, strides, box);
}

// ---- launch

int sm_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    n = cached[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <typename T, Mode MODE>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &b16, const ProductParams &p,
                   cudaStream_t st) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> configured[kMaxDevices];       // the attribute is per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(product_kernel<T, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    // tiles at most: every group's last tile may be a part
    const int64_t mt = (p.M + (MODE == kGated ? 63 : 127)) / (MODE == kGated ? 64 : 128);
    const int64_t G = (int64_t)p.gr.R * p.gr.per;
    const int64_t nt = p.N < 0 ? (int64_t)p.gr.R * p.gr.rows / kTileN + G : G * ((p.N + kTileN - 1) / kTileN);
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t grid = mt * nt < sms ? mt * nt : sms;
    product_kernel<T, MODE><<<(unsigned)grid, kThreads, kSmemBytes, st>>>(a, b, b16, p);
    return cudaGetLastError();
}

template <Mode MODE>
ep_status_t launch_product(int dtype, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &b16,
                           const ProductParams &p, cudaStream_t st) {
    const cudaError_t e = dtype == EP_DT_BF16 ? launch<__nv_bfloat16, MODE>(a, b, b16, p, st)
                                              : launch<__half, MODE>(a, b, b16, p, st);
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
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
    p.M = d->out_features;
    p.N = -1;
    p.K = d->in_features;
    p.act = d->activation;
    p.bias = d_bias;
    p.residual = *residual;
    p.out = *y;
    p.pre = *pre;
    p.error = d_error;
    const bool gated = d->activation == EP_ACT_SWIGLU;
    const int64_t G = (int64_t)d->ranks * d->groups;
    CUtensorMap a, b, b16;
    if (!(gated ? encode_gated(&a, d->dtype, d->weight, p.K, p.M, G)
                : encode_rows(&a, d->dtype, d->weight, p.K, p.M, G, kTileM)) ||
        !encode_rows(&b, d->dtype, d->x, p.K, d->rows, d->ranks, 64) ||
        !encode_rows(&b16, d->dtype, d->x, p.K, d->rows, d->ranks, 16))
        return EP_ERR_GPU_OP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return gated ? launch_product<kGated>(d->dtype, a, b, b16, p, st)
                 : launch_product<kForward>(d->dtype, a, b, b16, p, st);
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
    const int64_t G = (int64_t)d->ranks * d->groups;
    CUtensorMap a, b, b16;
    if (grad_x->ptr && d->rows > 0) {
        ProductParams p = {};
        p.gr = gr;
        p.M = d->in_features;
        p.N = -1;
        p.K = (int)wide;
        p.out = *grad_x;
        p.error = d_error;
        if (!encode_rows(&a, d->dtype, d->weight, d->in_features, wide, G, 64) ||
            !encode_rows(&b, d->dtype, dd, wide, d->rows, d->ranks, 64) ||
            !encode_rows(&b16, d->dtype, dd, wide, d->rows, d->ranks, 16))
            return EP_ERR_GPU_OP;
        const ep_status_t s = launch_product<kGradX>(d->dtype, a, b, b16, p, st);
        if (s != EP_SUCCESS) return s;
    }
    if (d_grad_w && d->rows == 0)
        return cudaMemsetAsync(d_grad_w, 0, (size_t)G * wide * d->in_features * 2, st) == cudaSuccess
                   ? EP_SUCCESS : EP_ERR_GPU_OP;
    if (d_grad_w) {
        ProductParams p = {};
        p.gr = gr;
        p.M = d->in_features;
        p.N = (int)wide;
        p.K = -1;
        p.out = ep_rows_t{d_grad_w, wide * d->in_features, d->in_features};
        p.error = d_error;
        if (!encode_rows(&a, d->dtype, d->x, d->in_features, d->rows, d->ranks, 64) ||
            !encode_rows(&b, d->dtype, dd, wide, d->rows, d->ranks, 64))
            return EP_ERR_GPU_OP;
        const ep_status_t s = launch_product<kGradW>(d->dtype, a, b, b, p, st);
        if (s != EP_SUCCESS) return s;
    }
    return launched();
}

}  // extern "C"
