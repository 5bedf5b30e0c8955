// Root-mean-square norm with the residual's addition, in the rows' type or in
// block-scaled 8 bits, and its gradient.
//
// A row stays in registers from its one read to its one write: a thread holds
// up to 4 chunks of 8 neighbouring values, the row's sums meet by shuffles and,
// where more than a warp shares the row, in shared memory.  Bound by memory.
#include "ep_fp8.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kMaxChunks = 4, kMaxThreads = EP_MAX_NORM_WIDTH / (kMaxChunks * 8);

// ------------------------------------------------------------ rows' chunks
// 8 values of a row.  VEC: one or two 16-byte accesses; else value by value,
// `n` of them (a row's end, or rows that are not 16-byte aligned).

template <typename T> struct Raw { uint4 q[sizeof(T) / 2]; };

template <typename T, bool VEC> __device__ __forceinline__ Raw<T> load_chunk(const T *p, int n) {
    Raw<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = ld_stream16(reinterpret_cast<const uint4 *>(p) + i);
    } else {
        T *e = reinterpret_cast<T *>(r.q);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : rounded<T>(0.f);
    }
    return r;
}
template <typename T> __device__ __forceinline__ void values(float *f, const Raw<T> &r) {
    const T *e = reinterpret_cast<const T *>(r.q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f32(e[i]);
}
template <typename T, bool VEC> __device__ __forceinline__ void store_chunk(T *p, const float *f, int n) {
    if constexpr (VEC && sizeof(T) == 2) {
        store8<T>(p, f);
    } else if constexpr (VEC) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = rounded<T>(f[i]);
    }
}
// 8 weights, in the rows' type or fp32.
template <typename T, bool VEC> __device__ __forceinline__ void load_weights(float *f, const void *w, bool w32, int c, int n) {
    if (w32) {
        const float *p = static_cast<const float *>(w) + c;
        if constexpr (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = i < n ? __ldg(p + i) : 0.f;
        }
    } else {
        values<T>(f, load_chunk<T, VEC>(static_cast<const T *>(w) + c, n));
    }
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

// Past this factor's use the squares of a row's largest finite values fit fp32.
// Rows need it where their sum of squares does not (some |v| > 2^56), which makes eps
// vanish next to it.
constexpr float kShrink = 0x1p-70f;

struct NormParams {
    int R, rows, H;
    float eps;
    bool w32;
    const void *weight;
    ep_rows_t x, residual, total, y, scales;
};

__device__ __forceinline__ int64_t row_at(const ep_rows_t &r, int seg, int row) {
    return seg * r.rank_stride + row * r.row_stride;
}

template <typename T, int CH, bool VEC, bool EIGHT>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p, int tpr) {
    __shared__ float part[1][32];
    const int t = threadIdx.x % tpr;
    const int64_t index = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (index >= (int64_t)p.R * p.rows) return;  // the whole warp: more warps a block only with a warp a row
    const int seg = (int)(index / p.rows), row = (int)(index - (int64_t)seg * p.rows);
    const T *x = static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row);
    const T *res = p.residual.ptr ? static_cast<const T *>(p.residual.ptr) + row_at(p.residual, seg, row) : nullptr;
    T *total = p.total.ptr ? static_cast<T *>(p.total.ptr) + row_at(p.total, seg, row) : nullptr;
    float h[CH][8];
    {
        Raw<T> a[CH], b[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
            if (c < p.H) {
                a[i] = load_chunk<T, VEC>(x + c, p.H - c);
                if (res) b[i] = load_chunk<T, VEC>(res + c, p.H - c);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
            if (c < p.H) {
                values<T>(h[i], a[i]);
                if (res) {
                    float f[8];
                    values<T>(f, b[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = f32(rounded<T>(h[i][j] + f[j]));
                }
                if (total) store_chunk<T, VEC>(total + c, h[i], p.H - c);
            }
        }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += h[i][j] * h[i][j];
    row_sums<1>(s, tpr, part);
    float r = rsqrtf(s[0] / p.H + p.eps);
    if (s[0] == __int_as_float(0x7f800000)) {    // the same for the whole row
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += (h[i][j] * kShrink) * (h[i][j] * kShrink);
        row_sums<1>(s, tpr, part);
        r = rsqrtf(s[0] / p.H) * kShrink;
    }
    if constexpr (EIGHT) {
        uint8_t *y = static_cast<uint8_t *>(p.y.ptr) + row_at(p.y, seg, row);
        float *scales = static_cast<float *>(p.scales.ptr) + row_at(p.scales, seg, row);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
            float f[8], w[8] = {};
            if (c < p.H) load_weights<T, VEC>(w, p.weight, p.w32, c, p.H - c);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = c < p.H ? h[i][j] * r * w[j] : 0.f;
            float scale;
            const uint2 q = block_codes(f, &scale);
            if (c >= p.H) continue;
            if constexpr (VEC) {
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
            const int c = (t + i * tpr) * 8;
            if (c >= p.H) continue;
            float w[8];
            load_weights<T, VEC>(w, p.weight, p.w32, c, p.H - c);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * r;
            store_chunk<T, VEC>(y + c, w, p.H - c);
        }
    }
}

// ---------------------------------------------------------------- gradient
// A block takes every gridDim-th row and keeps its sums for grad_weight in
// registers; column_kernel joins the blocks' sums in order.

constexpr int kParts = 304;                      // blocks at most, two for each SM

struct NormGradParams {
    int R, rows, H;
    float eps;
    bool w32;
    const void *weight;
    ep_rows_t x, grad, grad_total, grad_x;
    float *part;                                 // [rows taken at a time][H]
};

template <typename T, int CH, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) norm_grad_kernel(const NormGradParams p, int tpr) {
    __shared__ float part[2][32];
    const int t = threadIdx.x % tpr, per = blockDim.x / tpr;
    const int64_t first = (int64_t)blockIdx.x * per + threadIdx.x / tpr, step = (int64_t)gridDim.x * per;
    float dw[CH][8] = {};
    for (int64_t index = first; index < (int64_t)p.R * p.rows; index += step) {
        const int seg = (int)(index / p.rows), row = (int)(index - (int64_t)seg * p.rows);
        const T *x = static_cast<const T *>(p.x.ptr) + row_at(p.x, seg, row);
        const T *grad = static_cast<const T *>(p.grad.ptr) + row_at(p.grad, seg, row);
        float h[CH][8], u[CH][8];
        float s[2] = {0.f, 0.f};
        Raw<T> a[CH], b[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
            if (c < p.H) {
                a[i] = load_chunk<T, VEC>(x + c, p.H - c);
                b[i] = load_chunk<T, VEC>(grad + c, p.H - c);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = u[i][j] = 0.f;
            if (c < p.H) {
                float w[8];
                values<T>(h[i], a[i]);
                values<T>(u[i], b[i]);
                load_weights<T, VEC>(w, p.weight, p.w32, c, p.H - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[0] += h[i][j] * h[i][j];
                    s[1] += u[i][j] * w[j] * h[i][j];
                }
            }
        }
        row_sums<2>(s, tpr, part);
        float shrink = 1.f;
        float r = rsqrtf(s[0] / p.H + p.eps);
        if (s[0] == __int_as_float(0x7f800000)) {        // the same for the whole row
            shrink = kShrink;
            s[0] = s[1] = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = (t + i * tpr) * 8;
                float w[8] = {};
                if (c < p.H) load_weights<T, VEC>(w, p.weight, p.w32, c, p.H - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = h[i][j] * kShrink;
                    s[0] += v * v;
                    s[1] += u[i][j] * w[j] * v;
                }
            }
            row_sums<2>(s, tpr, part);
            r = rsqrtf(s[0] / p.H);
        }
        const float mean = s[1] / p.H * r;               // mean(u * n), n = total * r the normed row
        T *out = static_cast<T *>(p.grad_x.ptr) + row_at(p.grad_x, seg, row);
        const T *more = p.grad_total.ptr
                            ? static_cast<const T *>(p.grad_total.ptr) + row_at(p.grad_total, seg, row) : nullptr;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (t + i * tpr) * 8;
            if (c >= p.H) continue;
            float w[8], f[8] = {};
            load_weights<T, VEC>(w, p.weight, p.w32, c, p.H - c);
            if (more) {
                // plain loads: grad_x may be the same rows
                if constexpr (VEC) {
                    Raw<T> m;
#pragma unroll
                    for (int k = 0; k < (int)sizeof(T) / 2; ++k) m.q[k] = reinterpret_cast<const uint4 *>(more + c)[k];
                    values<T>(f, m);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = c + j < p.H ? f32(more[c + j]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = h[i][j] * shrink * r;
                dw[i][j] += u[i][j] * n;
                f[j] += (u[i][j] * w[j] - n * mean) * r * shrink;
            }
            store_chunk<T, VEC>(out + c, f, p.H - c);
        }
    }
    float *mine = p.part + first * p.H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (t + i * tpr) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < p.H) mine[c + j] = dw[i][j];
    }
}

// Column sums of part [n][H]: 32 columns a block, 16 rows at a time.
constexpr int kColumnRows = 16;
template <typename T> __global__ void __launch_bounds__(32 * kColumnRows) column_kernel(const float *part, int n, int H, T *out) {
    __shared__ float sums[kColumnRows][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
#pragma unroll 4
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

// Whether 16-byte accesses (8-byte ones of codes) reach all of the rows.
bool vectors(const ep_rows_t &r, int ranks, int64_t size, int64_t bytes = 16) {
    return !r.ptr || (aligned(r.ptr, bytes) && r.row_stride * size % bytes == 0 &&
                      (ranks == 1 || r.rank_stride * size % bytes == 0));
}

// Threads a row, chunks a thread, rows a block.
struct Shape {
    int chunks, tpr, per;
};
Shape shape_of(int H, int most) {
    const int all = (H + 7) / 8;
    Shape s;
    s.chunks = all <= 32 ? 1 : all <= 64 ? 2 : all <= 32 * most ? most : 1;
    if (all <= 32 * most) {
        s.tpr = 32;
        s.per = 8;
        return s;
    }
    while (s.chunks < most || (all + s.chunks - 1) / s.chunks > kMaxThreads) {
        if (s.chunks == kMaxChunks) break;
        s.chunks *= 2;
    }
    s.tpr = ((all + s.chunks - 1) / s.chunks + 31) / 32 * 32;
    s.per = 1;
    return s;
}

Shape grad_shape(const ep_norm_desc_t &d) { return shape_of(d.width, 2); }
// Rows that the gradient's blocks take at a time.
int64_t grad_parts(const ep_norm_desc_t &d) {
    const Shape s = grad_shape(d);
    const int64_t rows = (int64_t)d.ranks * d.rows, blocks = (rows + s.per - 1) / s.per;
    return (blocks < kParts ? blocks : kParts) * s.per;
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
    const NormParams p = {d->ranks, d->rows, d->width, d->eps, d->weight_dtype == EP_DT_FP32 && d->dtype != EP_DT_FP32,
                          d->weight, d->x, *residual, *total, *y, *scales};
    const bool vec = d->width % 8 == 0 && aligned(d->weight, 16) && vectors(d->x, d->ranks, size) &&
                     vectors(*residual, d->ranks, size) && vectors(*total, d->ranks, size) &&
                     vectors(*y, d->ranks, eight ? 1 : size, eight ? 8 : 16);
    const Shape s = shape_of(d->width, kMaxChunks);
    const int64_t rows = (int64_t)d->ranks * d->rows;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned blocks = (unsigned)((rows + s.per - 1) / s.per), threads = s.tpr * s.per;
    with_any_type(d->dtype, [&](auto type) {
        using T = decltype(type);
        with_chunks(s.chunks, [&](auto chunks) {
            constexpr int CH = decltype(chunks)::value;
            if (eight && vec) norm_kernel<T, CH, true, true><<<blocks, threads, 0, st>>>(p, s.tpr);
            else if (eight) norm_kernel<T, CH, false, true><<<blocks, threads, 0, st>>>(p, s.tpr);
            else if (vec) norm_kernel<T, CH, true, false><<<blocks, threads, 0, st>>>(p, s.tpr);
            else norm_kernel<T, CH, false, false><<<blocks, threads, 0, st>>>(p, s.tpr);
        });
    });
    return launched();
}

ep_status_t ep_rms_norm_workspace(const ep_norm_desc_t *d, size_t *bytes) {
    if (!valid(d) || !bytes) return EP_ERR_INVALID_ARGS;
    *bytes = (size_t)grad_parts(*d) * d->width * 4;
    return EP_SUCCESS;
}

ep_status_t ep_rms_norm_backward(const ep_norm_desc_t *d, const ep_rows_t *grad, const ep_rows_t *grad_total,
                                 const ep_rows_t *grad_x, void *d_grad_weight, void *d_workspace,
                                 size_t workspace_bytes, void *stream) {
    EP_RANGE("ep_rms_norm_backward");
    if (!valid(d) || !grad || !grad_total || !grad_x || !d_grad_weight || !aligned(d_workspace, 16) ||
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
    const int n = (int)grad_parts(*d);
    float *part = static_cast<float *>(d_workspace);
    if (d->rows > 0) {
        const NormGradParams p = {d->ranks, d->rows, d->width, d->eps, w32 && d->dtype != EP_DT_FP32, d->weight,
                                  d->x, *grad, *grad_total, *grad_x, part};
        const bool vec = d->width % 8 == 0 && aligned(d->weight, 16) && vectors(d->x, d->ranks, size) &&
                         vectors(*grad, d->ranks, size) && vectors(*grad_total, d->ranks, size) &&
                         vectors(*grad_x, d->ranks, size);
        with_any_type(d->dtype, [&](auto type) {
            using T = decltype(type);
            with_chunks(s.chunks, [&](auto chunks) {
                constexpr int CH = decltype(chunks)::value;
                if (vec) norm_grad_kernel<T, CH, true><<<n / s.per, s.tpr * s.per, 0, st>>>(p, s.tpr);
                else norm_grad_kernel<T, CH, false><<<n / s.per, s.tpr * s.per, 0, st>>>(p, s.tpr);
            });
        });
    }
    with_any_type(d->weight_dtype, [&](auto type) {
        using T = decltype(type);
        column_kernel<T><<<(d->width + 31) / 32, 32 * kColumnRows, 0, st>>>(part, n, d->width,
                                                                           static_cast<T *>(d_grad_weight));
    });
    return launched();
}

}  // extern "C"
