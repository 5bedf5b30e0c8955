// Root-mean-square norm with the residual's addition, in the rows' type or in
// block-scaled 8 bits, and its gradient.
//
// A row stays in registers from its one read to its one write: a thread holds
// up to 4 chunks of 8 neighbouring values, the row's sums meet by shuffles and,
// where more than a warp shares the row, in shared memory.  Bound by memory:
// 32768 x 7168 bf16 with a residual 264 us (7.1 TB/s), to 8 bits 259 (6.35 TB/s; 64 %
// issue, with arithmetic one value at a time 413 us).
#include "ep_fp8.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kMaxChunks = 4, kMaxThreads = EP_MAX_NORM_WIDTH / (kMaxChunks * 8);

// ------------------------------------------------------------ rows' chunks
// How a thread's chunk of 8 values stands in its row.  kVector: neighbours, one or
// two 16-byte accesses.  Rows that these do not reach go value by value:
// kStrided, every tpr-th value, so that a warp's accesses are next to each other
// (2332 x 4333 fp16: neighbours 56 us, so 27, bound by instructions: its 40 MB
// are 6 us of memory); kNeighbours where a block's codes need 16 lanes to hold 128
// neighbours.
enum Access { kStrided, kNeighbours, kVector };

struct Span {
    int c, step, n;              // first value, distance, how many there are
};
template <Access A> __device__ __forceinline__ Span span_of(int i, int t, int tpr, int H) {
    if constexpr (A == kStrided) {
        const int c = i * tpr * 8 + t;
        return Span{c, tpr, c < H ? (H - 1 - c) / tpr + 1 : 0};
    } else {
        const int c = (t + i * tpr) * 8;
        return Span{c, 1, H - c};
    }
}

template <typename T> struct Raw { uint4 q[sizeof(T) / 2]; };

template <typename T, Access A> __device__ __forceinline__ Raw<T> load_chunk(const T *row, const Span &s) {
    Raw<T> r;
    if constexpr (A == kVector) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = ld_stream16(reinterpret_cast<const uint4 *>(row + s.c) + i);
    } else {
        T *e = reinterpret_cast<T *>(r.q);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < s.n ? row[s.c + i * s.step] : rounded<T>(0.f);
    }
    return r;
}
// As pairs: sums and scalings are two-wide instructions.
template <typename T> __device__ __forceinline__ void values(float2 *f, const Raw<T> &r) {
    if constexpr (sizeof(T) == 2) {
        f[0] = unpack2<T>(r.q[0].x);
        f[1] = unpack2<T>(r.q[0].y);
        f[2] = unpack2<T>(r.q[0].z);
        f[3] = unpack2<T>(r.q[0].w);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[2 * i] = make_float2(__uint_as_float(r.q[i].x), __uint_as_float(r.q[i].y));
            f[2 * i + 1] = make_float2(__uint_as_float(r.q[i].z), __uint_as_float(r.q[i].w));
        }
    }
}
template <typename T> __device__ __forceinline__ Raw<T> packed(const float2 *f) {
    Raw<T> r;
    if constexpr (sizeof(T) == 2) {
        r.q[0] = make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.q[i] = make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y), __float_as_uint(f[2 * i + 1].x),
                                __float_as_uint(f[2 * i + 1].y));
    }
    return r;
}
template <typename T, Access A> __device__ __forceinline__ void store_chunk(T *row, const Raw<T> &r, const Span &s) {
    if constexpr (A == kVector) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(row + s.c)[i] = r.q[i];
    } else {
        const T *e = reinterpret_cast<const T *>(r.q);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) row[s.c + i * s.step] = e[i];
    }
}
// 8 weights, in the rows' type or fp32.
template <typename T, Access A> __device__ __forceinline__ void load_weights(float2 *f, const void *w, bool w32, const Span &s) {
    if (w32) values<float>(f, load_chunk<float, A>(static_cast<const float *>(w), s));
    else values<T>(f, load_chunk<T, A>(static_cast<const T *>(w), s));
}

// Sums over the threads that share a row: a warp, or the whole block.
template <int N> __device__ __forceinline__ void row_sums(float *v, int tpr, float (*part)[32]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr == 32) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();                             // the last sums were read
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < tpr / 32 ? part[i][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// A row's values are summed times a factor where their squares leave fp32's range.  Where the
// sum passes it (some |v| > 2^56): the largest finite values are then below 2^48, and 2^15
// squares of them below 2^111; r goes down to 2^-128, where fp32 still has 21 bits.
// Where it is below 2^-100, so that squares may have lost bits or vanished, and eps,
// below 2^-75, does not make up for them: the values are then between 2^-49 and 2^50.
constexpr float kShrink = 0x1p-80f, kGrow = 0x1p100f;
constexpr float kLeastSum = 0x1p-100f, kLeastEps = 0x1p-75f;

// The factor, from the sum without one; least: kLeastSum, or 0 where eps suffices.
__device__ __forceinline__ float factor_of(float sum, float least) {
    return sum == __int_as_float(0x7f800000) ? kShrink : sum < least ? kGrow : 1.f;
}
// 1 / sqrt(mean(h^2) + eps) from the sum of (h * factor)^2: without the factor, or with.
__device__ __forceinline__ float root_of(float sum, int H, float eps) { return rsqrtf(sum / H + eps); }
__device__ __forceinline__ float root_of(float sum, int H, float eps, float factor) {
    return rsqrtf(sum / H + eps * factor * factor);      // times factor: that of h
}

struct NormParams {
    int R, rows, H;
    float eps, least;            // least: of factor_of
    bool w32;
    const void *weight;
    ep_rows_t x, residual, total, y, scales;
};

__device__ __forceinline__ int64_t row_at(const ep_rows_t &r, int seg, int row) {
    return seg * r.rank_stride + row * r.row_stride;
}

// 1 / sqrt(mean(h^2) + eps) from the sum of squares.
template <int CH>
__device__ __forceinline__ float inverse_root(const float2 (*h)[4], float sum, const NormParams &p, int tpr, float (*part)[32]) {
    const float factor = factor_of(sum, p.least);        // the same for the whole row
    if (factor == 1.f) return root_of(sum, p.H, p.eps);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = mul2_rn(h[i][j], both(factor));
            s[0] += v.x * v.x + v.y * v.y;
        }
    row_sums<1>(s, tpr, part);
    return root_of(s[0], p.H, p.eps, factor) * factor;
}

// A row's chunks, `t` of `tpr` threads: total = x + residual, written if wanted,
// and its squares' sum so far.
template <typename T, int CH, Access A>
__device__ __forceinline__ float make_total(float2 (*h)[4], const Raw<T> *a, const Raw<T> *b, bool add, T *total, int H, int t, int tpr) {
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const Span at = span_of<A>(i, t, tpr, H);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = both(0.f);
        if (at.n > 0) {
            values<T>(h[i], a[i]);
            Raw<T> sum = a[i];
            if (add) {
                float2 f[4];
                values<T>(f, b[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = add2_rn(h[i][j], f[j]);
                sum = packed<T>(f);
                values<T>(h[i], sum);
            }
            if (total) store_chunk<T, A>(total, sum, at);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma2_rn(h[i][j], h[i][j], s);
    }
    return s.x + s.y;
}

// y, or its codes and scales.
template <typename T, int CH, Access A, bool EIGHT>
__device__ __forceinline__ void write_normed(const NormParams &p, int seg, int row, const float2 (*h)[4], float r, int t, int tpr) {
    if constexpr (EIGHT) {
        uint8_t *y = static_cast<uint8_t *>(p.y.ptr) + row_at(p.y, seg, row);
        float *scales = static_cast<float *>(p.scales.ptr) + row_at(p.scales, seg, row);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Span at = span_of<A>(i, t, tpr, p.H);
            const int c = at.c;
            if (c - t % 32 * 8 >= p.H) continue; // the whole warp: a block's codes need all its lanes
            float2 f[4], w[4] = {};
            if (c < p.H) load_weights<T, A>(w, p.weight, p.w32, at);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = c < p.H ? mul2_rn(mul2_rn(h[i][j], both(r)), w[j]) : both(0.f);
            float scale;
            const uint2 q = block_codes(f, &scale);
            if (c >= p.H) continue;
            if constexpr (A == kVector) {
                *reinterpret_cast<uint2 *>(y + c) = q;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[c + j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
            }
            if (c % 128 == 0) scales[c / 128] = scale;
        }
    } else {
        T *y = static_cast<T *>(p.y.ptr) + row_at(p.y, seg, row);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Span at = span_of<A>(i, t, tpr, p.H);
            if (at.n <= 0) continue;
            float2 w[4];
            load_weights<T, A>(w, p.weight, p.w32, at);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul2_rn(mul2_rn(h[i][j], both(r)), w[j]);
            store_chunk<T, A>(y, packed<T>(w), at);
        }
    }
}

// ---- a row a block (or a warp), straight from memory

template <typename T, int CH, Access A, bool EIGHT, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormParams p, int tpr) {
    __shared__ float part[1][32];
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int t = threadIdx.x % tpr;
    const int64_t index = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (index >= (int64_t)p.R * p.rows) return;  // the whole warp: more warps a block only with a warp a row
    const int seg = (int)(index / p.rows), row = (int)(index - (int64_t)seg * p.rows);
    const T *x = static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row);
    const T *res = p.residual.ptr ? static_cast<const T *>(p.residual.ptr) + row_at(p.residual, seg, row) : nullptr;
    Raw<T> a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const Span at = span_of<A>(i, t, tpr, p.H);
        if (at.n > 0) {
            a[i] = load_chunk<T, A>(x, at);
            if (res) b[i] = load_chunk<T, A>(res, at);
        }
    }
    float2 h[CH][4];
    float s[1] = {make_total<T, CH, A>(h, a, b, res, p.total.ptr ? static_cast<T *>(p.total.ptr) + row_at(p.total, seg, row) : nullptr,
                                         p.H, t, tpr)};
    row_sums<1>(s, tpr, part);
    write_normed<T, CH, A, EIGHT>(p, seg, row, h, inverse_root<CH>(h, s[0], p, tpr, part), t, tpr);
}

// ---------------------------------------------------------------- gradient
// A block takes every gridDim-th row and keeps its sums for grad_weight in
// registers; column_kernel joins the blocks' sums in order.  Bound by memory and, at
// 63 % issue, by instructions: 16384 x 7168 bf16 with grad_total 162 us and 5 for the
// sums, at 83 % of the copy rate.

// The number of SMs is fixed here, not asked for: it sets the order of the sums and the
// size of the workspace, which do not depend on the device then.
constexpr int kSms = 152, kParts = 3 * kSms;     // blocks at most where a block keeps no rows ahead

struct NormGradParams {
    int R, rows, H;
    float eps, least;            // least: of factor_of
    bool w32;
    const void *weight;
    ep_rows_t x, grad, grad_total, grad_x;
    float *part;                                 // [blocks][H]
};

// A row's sums, h^2 and u h, and what its outputs need of them.
struct RowGrad {
    float2 squares = {0.f, 0.f}, inner = {0.f, 0.f};
    float r, mean;               // mean(u n), n = h r the normed row

    __device__ __forceinline__ void add(const float2 *h, const float2 *g, const float2 *w) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            squares = fma2_rn(h[j], h[j], squares);
            inner = fma2_rn(mul2_rn(g[j], w[j]), h[j], inner);
        }
    }
    __device__ __forceinline__ void sums(float *s) const {
        s[0] = squares.x + squares.y;
        s[1] = inner.x + inner.y;
    }
    // From the sums of h * factor.
    __device__ __forceinline__ void set(const float *s, int H, float eps, float factor) {
        r = factor == 1.f ? root_of(s[0], H, eps) : root_of(s[0], H, eps, factor);
        mean = s[1] / H * r;
        r *= factor;
    }
    // 8 values of the row's gradient, added to f; the weight's is added to dw.
    __device__ __forceinline__ void out(float2 *f, float2 *dw, const float2 *h, const float2 *g, const float2 *w) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 n = mul2_rn(h[j], both(r));
            dw[j] = fma2_rn(g[j], n, dw[j]);
            f[j] = fma2_rn(fma2_rn(n, both(-mean), mul2_rn(g[j], w[j])), both(r), f[j]);
        }
    }
};
__device__ __forceinline__ void scale8(float2 *h, float factor) {
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = mul2_rn(h[j], both(factor));
}
template <int CH> __device__ __forceinline__ void write_part(float *to, int H, const float2 (*dw)[4], int t, int tpr) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (t + i * tpr) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < H) to[c + j] = j & 1 ? dw[i][j / 2].y : dw[i][j / 2].x;
    }
}

template <typename T, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && CH < 4 ? 3 : 1) norm_grad_kernel(const NormGradParams p, int tpr) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int t = threadIdx.x % tpr, per = blockDim.x / tpr;
    const int64_t first = (int64_t)blockIdx.x * per + threadIdx.x / tpr, step = (int64_t)gridDim.x * per;
    float2 dw[CH][4] = {};
    for (int64_t index = first; index < (int64_t)p.R * p.rows; index += step) {
        const int seg = (int)(index / p.rows), row = (int)(index - (int64_t)seg * p.rows);
        const T *x = static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row);
        const T *grad = static_cast<const T *>(p.grad.ptr) + row_at(p.grad, seg, row);
        const T *total = p.grad_total.ptr ? static_cast<const T *>(p.grad_total.ptr) + row_at(p.grad_total, seg, row) : nullptr;
        T *out = static_cast<T *>(p.grad_x.ptr) + row_at(p.grad_x, seg, row);
        Raw<T> a[CH], b[CH], more[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Span at = span_of<kVector>(i, t, tpr, p.H);
            if (at.n > 0) {
                a[i] = load_chunk<T, kVector>(x, at);
                b[i] = load_chunk<T, kVector>(grad, at);
                if (total) more[i] = load_chunk<T, kVector>(total, at);      // before grad_x, perhaps the same rows, is written
            }
        }
        float s[2];
        auto sums = [&](float factor) {
            RowGrad sum;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const Span at = span_of<kVector>(i, t, tpr, p.H);
                if (at.n <= 0) continue;
                float2 h[4], g[4], w[4];
                values<T>(h, a[i]);
                values<T>(g, b[i]);
                load_weights<T, kVector>(w, p.weight, p.w32, at);
                if (factor != 1.f) scale8(h, factor);
                sum.add(h, g, w);
            }
            sum.sums(s);
            row_sums<2>(s, tpr, part);
        };
        sums(1.f);
        const float factor = factor_of(s[0], p.least);               // the same for the whole row
        if (factor != 1.f) sums(factor);
        RowGrad rg;
        rg.set(s, p.H, p.eps, factor);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Span at = span_of<kVector>(i, t, tpr, p.H);
            if (at.n <= 0) continue;
            float2 h[4], g[4], w[4], f[4] = {};
            values<T>(h, a[i]);
            values<T>(g, b[i]);
            load_weights<T, kVector>(w, p.weight, p.w32, at);
            if (total) values<T>(f, more[i]);
            rg.out(f, dw[i], h, g, w);
            store_chunk<T, kVector>(out, packed<T>(f), at);
        }
    }
    float *mine = p.part + (int64_t)blockIdx.x * p.H;
    if (tpr > 32) {
        write_part<CH>(mine, p.H, dw, t, tpr);
        return;
    }
    // a warp a row: the block's warps add theirs, in order
    __shared__ float sums[THREADS == 256 ? 8 : 1][CH * 256];
    const int warp = threadIdx.x / 32;
    if constexpr (THREADS == 256) {
        write_part<CH>(sums[warp], p.H, dw, t, tpr);
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += 256) {
            float v = 0.f;
            for (int w = 0; w < 8; ++w) v += sums[w][c];
            mine[c] = v;
        }
    }
}

// Rows that 16-byte accesses do not reach: a thread has every tpr-th value, reads it
// again (from L1) once the row's sums are known, and keeps the weight's sums in
// shared memory, all of it in loops of few registers: 16384 x 5001 bf16 313 us, bound by
// instructions (its bytes are 72 us of memory); in registers, unrolled, 629.
template <typename T>
__global__ void __launch_bounds__(512, 3) norm_grad_strided_kernel(const NormGradParams p, int tpr) {
    extern __shared__ __align__(16) float weight_sums[];
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int t = threadIdx.x % tpr, per = blockDim.x / tpr;
    const int64_t first = (int64_t)blockIdx.x * per + threadIdx.x / tpr, step = (int64_t)gridDim.x * per;
    float *dw = weight_sums + threadIdx.x / tpr * p.H;
    auto weight = [&](int c) {
        return p.w32 ? __ldg(static_cast<const float *>(p.weight) + c) : f32(static_cast<const T *>(p.weight)[c]);
    };
    for (int c = t; c < p.H; c += tpr) dw[c] = 0.f;
    for (int64_t index = first; index < (int64_t)p.R * p.rows; index += step) {
        const int seg = (int)(index / p.rows), row = (int)(index - (int64_t)seg * p.rows);
        const T *x = static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row);
        const T *grad = static_cast<const T *>(p.grad.ptr) + row_at(p.grad, seg, row);
        const T *total = p.grad_total.ptr ? static_cast<const T *>(p.grad_total.ptr) + row_at(p.grad_total, seg, row) : nullptr;
        T *out = static_cast<T *>(p.grad_x.ptr) + row_at(p.grad_x, seg, row);
        float s[2];
        float factor = 1.f;
        for (;;) {
            s[0] = s[1] = 0.f;
#pragma unroll 4
            for (int c = t; c < p.H; c += tpr) {
                const float h = f32(x[c]) * factor;
                s[0] += h * h;
                s[1] += f32(grad[c]) * weight(c) * h;
            }
            row_sums<2>(s, tpr, part);
            if (factor != 1.f) break;
            factor = factor_of(s[0], p.least);                       // the same for the whole row
            if (factor == 1.f) break;
        }
        RowGrad rg;
        rg.set(s, p.H, p.eps, factor);
        if (total) {
#pragma unroll 4
            for (int c = t; c < p.H; c += tpr) {
                const float g = f32(grad[c]), n = f32(x[c]) * rg.r, more = f32(total[c]);     // before grad_x, perhaps the same row
                dw[c] += g * n;
                out[c] = rounded<T>((g * weight(c) - n * rg.mean) * rg.r + more);
            }
        } else {
#pragma unroll 4
            for (int c = t; c < p.H; c += tpr) {
                const float g = f32(grad[c]), n = f32(x[c]) * rg.r;
                dw[c] += g * n;
                out[c] = rounded<T>((g * weight(c) - n * rg.mean) * rg.r);
            }
        }
    }
    float *mine = p.part + (int64_t)blockIdx.x * p.H;
    if (tpr > 32) {
        for (int c = t; c < p.H; c += tpr) mine[c] = dw[c];
        return;
    }
    // a warp a row: the block's warps add theirs, in order
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < per; ++w) v += weight_sums[w * p.H + c];
        mine[c] = v;
    }
}

// ---- many rows: a block goes from row to row and has the next ones brought into
// shared memory by bulk copies meanwhile, so that reads never pause.

constexpr int kMaxRing = 8;
constexpr uint64_t kRingWaitNs = 1000000000ull;

struct Ring {
    uint64_t *full;
    unsigned char *rows;
    int stages, tensors, bytes;                  // bytes of a row
    int *gave_up;

    __device__ unsigned char *at(int s, int tensor) const { return rows + ((size_t)s * tensors + tensor) * bytes; }
    // By one thread: rows of all tensors into stage s.
    __device__ void load(int s, const void *const *from) const {
        mbar_expect_tx(&full[s], tensors * bytes);
        for (int i = 0; i < tensors; ++i) bulk_load<false>(at(s, i), from[i], bytes, &full[s], 0);
    }
    // By one thread, after a wait that gave up: as many of the last loads as come.
    __device__ void drain(int64_t loads) const {
        for (int64_t n = loads > stages ? loads - stages : 0; n < loads; ++n)
            mbar_wait(&full[n % stages], (uint32_t)(n / stages) & 1u, kRingWaitNs);
    }
    // By every thread: a row is there.  After a wait of a second all others end at once.
    __device__ void wait(int s, uint32_t phase) const {
        if (mbar_try_wait(&full[s], phase) || *(volatile int *)gave_up) return;
        if (!mbar_wait(&full[s], phase, kRingWaitNs)) *(volatile int *)gave_up = 1;
    }
};
template <typename T> __device__ __forceinline__ Raw<T> ring_chunk(const unsigned char *row, int c) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = reinterpret_cast<const uint4 *>(row + (size_t)c * sizeof(T))[i];
    return r;
}
// A block's sums with one barrier: `slot` alternates.
template <int N> __device__ __forceinline__ void block_sums(float *v, float (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lane == 0) part[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < warps ? part[i][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

constexpr int kGradRingThreads = 512;
template <typename T, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS, 2) norm_grad_ring_kernel(const NormGradParams p, int stages, uint32_t *error) {
    extern __shared__ __align__(128) unsigned char ring_rows[];
    __shared__ uint64_t full[kMaxRing];
    __shared__ float part[3][2][32];
    __shared__ int gave_up;
    const int t = threadIdx.x, tpr = blockDim.x;
    const Ring ring = {full, ring_rows, stages, p.grad_total.ptr ? 3 : 2, p.H * (int)sizeof(T), &gave_up};
    if (t == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        mbar_init_fence();
        gave_up = 0;
    }
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int all = p.R * p.rows;
    int64_t loads = 0, next = blockIdx.x;        // of thread 0
    int to = 0;
    auto load = [&]() {
        if (t != 0 || next >= all || *(volatile int *)&gave_up) return;
        const int seg = (int)next / p.rows, row = (int)next - seg * p.rows;
        const void *from[3] = {static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row),
                               static_cast<const T *>(p.grad.ptr) + row_at(p.grad, seg, row),
                               static_cast<const T *>(p.grad_total.ptr) + row_at(p.grad_total, seg, row)};
        ring.load(to, from);
        ++loads;
        next += gridDim.x;
        if (++to == stages) to = 0;
    };
    for (int s = 0; s < stages - 1; ++s) load();
    float2 dw[CH][4] = {};
    int s = 0;
    uint32_t phase = 0, turn = 0;
    for (int64_t index = blockIdx.x; index < all; index += gridDim.x) {
        const int seg = (int)index / p.rows, row = (int)index - seg * p.rows;
        T *out = static_cast<T *>(p.grad_x.ptr) + row_at(p.grad_x, seg, row);
        ring.wait(s, phase);
        // The row is read twice, before and after its sums are known, so that
        // registers suffice for two blocks an SM.
        float v[2];
        auto sums = [&](float factor) {
            RowGrad sum;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const Span at = span_of<kVector>(i, t, tpr, p.H);
                if (at.n <= 0) continue;
                float2 h[4], g[4], w[4];
                values<T>(h, ring_chunk<T>(ring.at(s, 0), at.c));
                values<T>(g, ring_chunk<T>(ring.at(s, 1), at.c));
                load_weights<T, kVector>(w, p.weight, p.w32, at);
                if (factor != 1.f) scale8(h, factor);
                sum.add(h, g, w);
            }
            sum.sums(v);
        };
        sums(1.f);
        block_sums<2>(v, part[turn]);            // and every thread is done with the row before
        load();
        const float factor = factor_of(v[0], p.least);               // the same for the whole row
        if (factor != 1.f) {
            sums(factor);
            row_sums<2>(v, tpr, part[2]);
        }
        RowGrad rg;
        rg.set(v, p.H, p.eps, factor);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Span at = span_of<kVector>(i, t, tpr, p.H);
            if (at.n <= 0) continue;
            float2 h[4], g[4], w[4], f[4] = {};
            values<T>(h, ring_chunk<T>(ring.at(s, 0), at.c));
            values<T>(g, ring_chunk<T>(ring.at(s, 1), at.c));
            load_weights<T, kVector>(w, p.weight, p.w32, at);
            if (p.grad_total.ptr) values<T>(f, ring_chunk<T>(ring.at(s, 2), at.c));
            rg.out(f, dw[i], h, g, w);
            store_chunk<T, kVector>(out, packed<T>(f), at);
        }
        turn ^= 1u;
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
    }
    write_part<CH>(p.part + (int64_t)blockIdx.x * p.H, p.H, dw, t, tpr);
    if (t == 0 && *(volatile int *)&gave_up) {
        ring.drain(loads);
        if (error) atomicOr(error, EP_DEVERR_TIMEOUT);
    }
}

// Column sums of part [n][H]: 32 columns a block, 32 rows at a time.
constexpr int kColumnRows = 32;
template <typename T> __global__ void __launch_bounds__(32 * kColumnRows) column_kernel(const float *part, int n, int H, T *out) {
    __shared__ float sums[kColumnRows][32];
    grid_dependency_wait();
    grid_dependents_may_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
#pragma unroll 8
        for (int i = warp; i < n; i += kColumnRows) s += part[(int64_t)i * H + c];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < H) {
        for (int i = 1; i < kColumnRows; ++i) s += sums[i][lane];
        out[c] = rounded<T>(s);
    }
}

// -------------------------------------------------------------- host side

template <typename F> void with_any_type(int dtype, F f) {
    if (dtype == EP_DT_FP32) f(float());
    else with_type(dtype, f);
}
template <typename F> void with_chunks(int n, F f) {
    if (n == 1) f(std::integral_constant<int, 1>());
    else if (n == 2) f(std::integral_constant<int, 2>());
    else f(std::integral_constant<int, 4>());
}

int64_t size_of(int dtype) { return dtype == EP_DT_FP32 ? 4 : 2; }

bool valid_norm_rows(const ep_rows_t &r, const ep_norm_desc_t &d, int64_t width, int64_t size) {
    return r.ptr && aligned(r.ptr, size) && r.row_stride >= width && (d.ranks == 1 || r.rank_stride > 0);
}

bool valid(const ep_norm_desc_t *d) {
    if (!d || d->ranks < 1 || d->ranks > 65535 || d->rows < 0 || (int64_t)d->ranks * d->rows > 1 << 30) return false;
    if (d->width < 1 || d->width > EP_MAX_NORM_WIDTH || !(d->eps >= 0.f) || d->eps > 3.4e38f) return false;
    if (d->dtype != EP_DT_BF16 && d->dtype != EP_DT_FP16 && d->dtype != EP_DT_FP32) return false;
    if (d->weight_dtype != d->dtype && d->weight_dtype != EP_DT_FP32) return false;
    return d->weight && aligned(d->weight, size_of(d->weight_dtype)) &&
           (d->rows == 0 || valid_norm_rows(d->x, *d, d->width, size_of(d->dtype)));
}

float least_sum(const ep_norm_desc_t &d) { return d.eps < kLeastEps ? kLeastSum : 0.f; }

// Whether 16-byte accesses (8-byte ones of codes) reach all of the rows.
bool vectors(const ep_rows_t &r, int ranks, int64_t size, int64_t bytes = 16) {
    return !r.ptr || (aligned(r.ptr, bytes) && r.row_stride * size % bytes == 0 &&
                      (ranks == 1 || r.rank_stride * size % bytes == 0));
}

// Threads a row, chunks a thread, rows a block.  A warp a row where `most`
// chunks a lane hold it, else a block.
struct Shape {
    int chunks, tpr, per;
};
Shape shape_of(int H, int most) {
    const int all = (H + 7) / 8;
    if (all <= 32 * most) return Shape{all <= 32 ? 1 : all <= 64 ? 2 : 4, 32, 8};
    Shape s = {most, 0, 1};
    while ((all + s.chunks - 1) / s.chunks > kMaxThreads) s.chunks *= 2;
    s.tpr = ((all + s.chunks - 1) / s.chunks + 31) / 32 * 32;
    return s;
}

// Stages of rows in `bytes` of shared memory, at most kMaxRing.
int ring_stages(int64_t row_bytes, int tensors, int64_t bytes) {
    const int64_t n = bytes / (row_bytes * tensors);
    return (int)(n < kMaxRing ? n : kMaxRing);
}
constexpr int64_t kRingMost = 220 * 1024;
constexpr int64_t kRingRow = 1024;               // bytes of a row at least

template <typename... Params, typename... Args>
cudaError_t launch_ring(void (*kernel)(Params...), std::atomic<bool> *configured, int blocks, int threads, size_t bytes, cudaStream_t st,
                        Args &&...args) {
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {         // the attribute is per device
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingMost);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_after_previous(kernel, blocks, threads, bytes, st, static_cast<Args &&>(args)...);
}

// How the gradient of many rows goes through the ring; stages 0: it does not.
struct RingShape {
    int stages, threads, blocks;
};
RingShape grad_ring(const ep_norm_desc_t &d, bool vec, bool total) {
    const int64_t row = d.width * size_of(d.dtype), rows = (int64_t)d.ranks * d.rows;
    RingShape r = {0, 0, 0};
    r.threads = ((d.width / 8 + 1) / 2 + 31) / 32 * 32;
    if (!vec || row < kRingRow || r.threads < 64 || r.threads > kGradRingThreads) return r;
    int blocks = 1024 / r.threads;                               // an SM's, by registers
    if (blocks > 8) blocks = 8;
    while (blocks > 1 && ring_stages(row, total ? 3 : 2, kRingMost / blocks) < 3) --blocks;
    if (blocks == 1 && ring_stages(row, total ? 3 : 2, kRingMost / 2) == 2) blocks = 2;
    const int stages = ring_stages(row, total ? 3 : 2, kRingMost / blocks);
    r.blocks = kSms * blocks;
    if (stages >= 2 && rows >= 4 * r.blocks) r.stages = stages < 4 ? stages : 4;
    return r;
}

// Chunks a thread as in the norm: fewer where a row is all that a block has.
Shape grad_shape(const ep_norm_desc_t &d) { return shape_of(d.width, (int64_t)d.ranks * d.rows <= kParts ? 1 : 2); }
// Rows that vectors do not reach: a warp a row, or more threads the longer it is;
// blocks by registers and shared memory.
struct StridedShape {
    int tpr, per, blocks;
};
StridedShape strided_shape(const ep_norm_desc_t &d) {
    const int64_t rows = (int64_t)d.ranks * d.rows;
    StridedShape s = {d.width <= 512 ? 32 : d.width <= 1024 ? 64 : d.width <= 2048 ? 128 : d.width <= 8192 ? 256 : 512, 1, 0};
    if (rows <= kParts) s.tpr = d.width <= 64 ? 32 : d.width <= 256 ? 128 : 512;    // all of a row at once
    else if (s.tpr == 32) s.per = 8;
    int64_t an_sm = kRingMost / ((int64_t)s.per * d.width * 4 + 1024);
    if (an_sm > 1536 / (s.tpr * s.per)) an_sm = 1536 / (s.tpr * s.per);
    if (an_sm > 8) an_sm = 8;
    const int64_t blocks = (rows + s.per - 1) / s.per;
    s.blocks = (int)(blocks < an_sm * kSms ? blocks : an_sm * kSms);
    return s;
}

// Parts of the weight's gradient, one a block.
int64_t grad_parts(const ep_norm_desc_t &d) {
    const Shape s = grad_shape(d);
    const int64_t rows = (int64_t)d.ranks * d.rows, blocks = (rows + s.per - 1) / s.per;
    return blocks < kParts ? blocks : kParts;
}
// Of the kernel with most blocks, as other tensors' alignment may choose any; and never fewer
// than for fewer rows (some shapes have a warp a row only where rows are many), so that
// a workspace for the largest batch does for all.
int64_t most_parts(const ep_norm_desc_t &d) {
    const int64_t rows = (int64_t)d.ranks * d.rows;
    int64_t most = 0;
    for (const int64_t n : {rows < kParts ? rows : (int64_t)kParts, rows}) {
        ep_norm_desc_t e = d;
        e.ranks = 1;
        e.rows = (int32_t)n;
        const RingShape with = grad_ring(e, true, true), without = grad_ring(e, true, false);
        for (const int64_t parts : {grad_parts(e), (int64_t)strided_shape(e).blocks, (int64_t)(with.stages ? with.blocks : 0),
                                    (int64_t)(without.stages ? without.blocks : 0)})
            if (parts > most) most = parts;
    }
    return most;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_rms_norm(const ep_norm_desc_t *d, const ep_rows_t *residual, const ep_rows_t *total,
                        const ep_rows_t *y, const ep_rows_t *scales, void *stream) {
    EP_RANGE("ep_rms_norm");
    if (!valid(d) || !residual || !total || !y || !scales) return EP_ERR_INVALID_ARGS;
    if (d->rows == 0) return EP_SUCCESS;
    const bool eight = scales->ptr != nullptr;
    const int64_t size = size_of(d->dtype);
    if ((eight && d->width % 128) || !valid_norm_rows(*y, *d, d->width, eight ? 1 : size) ||
        (eight && !valid_norm_rows(*scales, *d, d->width / 128, 4)) ||
        (residual->ptr && !valid_norm_rows(*residual, *d, d->width, size)) ||
        (total->ptr && !valid_norm_rows(*total, *d, d->width, size)))
        return EP_ERR_INVALID_ARGS;
    const NormParams p = {d->ranks, d->rows, d->width, d->eps, least_sum(*d), d->weight_dtype == EP_DT_FP32 && d->dtype != EP_DT_FP32,
                          d->weight, d->x, *residual, *total, *y, *scales};
    const bool vec = d->width % 8 == 0 && aligned(d->weight, 16) && vectors(d->x, d->ranks, size) &&
                     vectors(*residual, d->ranks, size) && vectors(*total, d->ranks, size) &&
                     vectors(*y, d->ranks, eight ? 1 : size, eight ? 8 : 16);
    const int64_t rows = (int64_t)d->ranks * d->rows;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    // Chunks a thread: 4 of 16 bits (32768 x 7168 to 8 bits 259 us, with 2 348) or 2 of fp32 (4096 x
    // 16384 168 us, with 4 205); few rows: one, all of a row on its way at once (1.1 us less).
    const Shape s = shape_of(d->width, rows <= 304 ? 1 : d->dtype == EP_DT_FP32 ? 2 : kMaxChunks);
    const unsigned blocks = (unsigned)((rows + s.per - 1) / s.per), threads = s.tpr * s.per;
    with_any_type(d->dtype, [&](auto type) {
        using T = decltype(type);
        with_chunks(s.chunks, [&](auto chunks) {
            constexpr int CH = decltype(chunks)::value;
            auto go = [&](auto most) {
                constexpr int N = decltype(most)::value;
                auto kernel = eight ? (vec ? norm_kernel<T, CH, kVector, true, N> : norm_kernel<T, CH, kNeighbours, true, N>)
                                    : (vec ? norm_kernel<T, CH, kVector, false, N> : norm_kernel<T, CH, kStrided, false, N>);
                e = launch_after_previous(kernel, blocks, threads, 0, st, p, s.tpr);
            };
            if (threads <= 256) go(std::integral_constant<int, 256>());
            else go(std::integral_constant<int, kMaxThreads>());
        });
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

ep_status_t ep_rms_norm_workspace(const ep_norm_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = (size_t)most_parts(*d) * d->width * 4;
    return EP_SUCCESS;
}

ep_status_t ep_rms_norm_backward(const ep_norm_desc_t *d, const ep_rows_t *grad, const ep_rows_t *grad_total,
                                 const ep_rows_t *grad_x, void *d_grad_weight, void *d_workspace,
                                 size_t workspace_bytes, uint32_t *d_error, void *stream) {
    EP_RANGE("ep_rms_norm_backward");
    if (!valid(d) || !aligned(d_error, 4) || !grad || !grad_total || !grad_x || !d_grad_weight || !aligned(d_workspace, 16) ||
        !aligned(d_grad_weight, size_of(d->weight_dtype)))
        return EP_ERR_INVALID_ARGS;
    const int64_t size = size_of(d->dtype);
    size_t need = 0;
    ep_rms_norm_workspace(d, &need);
    if (workspace_bytes < need || (need && !d_workspace)) return EP_ERR_INVALID_ARGS;
    if (d->rows > 0 && (!valid_norm_rows(*grad, *d, d->width, size) || !valid_norm_rows(*grad_x, *d, d->width, size) ||
                        (grad_total->ptr && !valid_norm_rows(*grad_total, *d, d->width, size))))
        return EP_ERR_INVALID_ARGS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool w32 = d->weight_dtype == EP_DT_FP32;
    const Shape s = grad_shape(*d);
    int n = (int)grad_parts(*d);
    float *part = static_cast<float *>(d_workspace);
    cudaError_t e = cudaSuccess;
    if (d->rows > 0) {
        const NormGradParams p = {d->ranks, d->rows, d->width, d->eps, least_sum(*d), w32 && d->dtype != EP_DT_FP32, d->weight,
                                  d->x, *grad, *grad_total, *grad_x, part};
        const bool vec = d->width % 8 == 0 && aligned(d->weight, 16) && vectors(d->x, d->ranks, size) &&
                         vectors(*grad, d->ranks, size) && vectors(*grad_total, d->ranks, size) &&
                         vectors(*grad_x, d->ranks, size);
        const RingShape ring = grad_ring(*d, vec, grad_total->ptr);
        with_any_type(d->dtype, [&](auto type) {
            using T = decltype(type);
            if (ring.stages) {
                static std::atomic<bool> configured[2][kMaxDevices];
                const size_t bytes = (size_t)ring.stages * (grad_total->ptr ? 3 : 2) * d->width * size;
                n = ring.blocks;
                e = ring.threads <= 448      // 72 registers a thread, else 64
                        ? launch_ring(norm_grad_ring_kernel<T, 2, 448>, configured[0], n, ring.threads, bytes, st, p, ring.stages, d_error)
                        : launch_ring(norm_grad_ring_kernel<T, 2, kGradRingThreads>, configured[1], n, ring.threads, bytes, st, p,
                                      ring.stages, d_error);
                return;
            }
            if (!vec) {
                static std::atomic<bool> configured[kMaxDevices];
                const StridedShape q = strided_shape(*d);
                n = q.blocks;
                e = launch_ring(norm_grad_strided_kernel<T>, configured, n, q.tpr * q.per, (size_t)q.per * d->width * 4, st, p, q.tpr);
                return;
            }
            with_chunks(s.chunks, [&](auto chunks) {
                constexpr int CH = decltype(chunks)::value;
                auto go = [&](auto most) {
                    constexpr int N = decltype(most)::value;
                    e = launch_after_previous(norm_grad_kernel<T, CH, N>, n, s.tpr * s.per, 0, st, p, s.tpr);
                };
                if constexpr (CH <= 2) {             // 4 only where 2 would take more threads than there are
                    if (s.tpr * s.per <= 256) return go(std::integral_constant<int, 256>());
                    if (s.tpr * s.per <= 512) return go(std::integral_constant<int, 512>());
                }
                go(std::integral_constant<int, kMaxThreads>());
            });
        });
    }
    if (e != cudaSuccess) return EP_ERR_GPU_OP;
    with_any_type(d->weight_dtype, [&](auto type) {
        using T = decltype(type);
        e = launch_after_previous(column_kernel<T>, (d->width + 31) / 32, 32 * kColumnRows, 0, st, part, n, d->width,
                                  static_cast<T *>(d_grad_weight));
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

}  // extern "C"
