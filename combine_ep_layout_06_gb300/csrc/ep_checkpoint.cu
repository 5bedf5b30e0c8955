// Activations kept in block-scaled 8 bits between forward and backward: saved,
// and restored through the activation.
//
// Element-wise over the rows of every group.  A lane takes 8 (restored) or 16 (saved)
// neighbouring values, a warp 256 or 512 of a row; a block's warps take rows in turn.
#include "ep_fp8.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kCols = 256, kRows = 4;

struct CheckpointParams {
    Groups gr;
    int F, act, splits;
    ep_rows_t x, codes, scales;          // x: what is saved, or what is restored
};

// This block's part of its group's rows.
struct Part {
    int seg, first, end;
};
__device__ __forceinline__ Part part_of(const CheckpointParams &p) {
    const int g = blockIdx.y;
    int first, rows;
    group_range(p.gr, g, &first, &rows);
    const int per = (rows + p.splits - 1) / p.splits;
    const int64_t a = (int64_t)blockIdx.z * per, b = a + per;
    return Part{g / p.gr.per, first + (int)(a < rows ? a : rows), first + (int)(b < rows ? b : rows)};
}

// The larger magnitudes of 16-bit values, pair by pair, NaN above all: the bits
// without their signs stand in that order.
__device__ __forceinline__ uint32_t larger(const uint4 &q) {
    return __vmaxu2(__vmaxu2(q.x & 0x7fff7fffu, q.y & 0x7fff7fffu), __vmaxu2(q.z & 0x7fff7fffu, q.w & 0x7fff7fffu));
}

// A lane takes 16 neighbouring values, so that 8 lanes share a block's scale: the
// kernel is bound by instructions (16 lanes of 8 values: 64 us where this takes
// 54, for 32768 x 3584).
constexpr int kSaveCols = 512, kSaveRows = 2;
template <typename T> __global__ void __launch_bounds__(kWarps * 32, 4) save_kernel(const CheckpointParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * kSaveCols + lane * 16;
    const bool live = c < p.F, second = c + 8 < p.F;
    grid_dependency_wait();
    grid_dependents_may_launch();
    const Part part = part_of(p);
    const int64_t r0 = part.first + warp;
    const T *x = static_cast<const T *>(p.x.ptr) + part.seg * p.x.rank_stride + r0 * p.x.row_stride + c;
    uint8_t *codes = static_cast<uint8_t *>(p.codes.ptr) + part.seg * p.codes.rank_stride + r0 * p.codes.row_stride + c;
    float *scales = static_cast<float *>(p.scales.ptr) + part.seg * p.scales.rank_stride + r0 * p.scales.row_stride + c / 128;
    const int64_t xs = kWarps * p.x.row_stride, cs = kWarps * p.codes.row_stride, ss = kWarps * p.scales.row_stride;
    for (int left = part.end - (int)r0; left > 0; left -= kWarps * kSaveRows) {
        uint4 v[kSaveRows][2];
#pragma unroll
        for (int u = 0; u < kSaveRows; ++u) {
            v[u][0] = live && u * kWarps < left ? ld_stream16(x + u * xs) : make_uint4(0, 0, 0, 0);
            v[u][1] = second && u * kWarps < left ? ld_stream16(x + u * xs + 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kSaveRows; ++u) {
            if (u * kWarps >= left) break;       // the same for the warp
            uint32_t m = __vmaxu2(larger(v[u][0]), larger(v[u][1]));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint16_t top = (uint16_t)max(m >> 16, m & 0xffffu);
            const float2 f[8] = {unpack2<T>(v[u][0].x), unpack2<T>(v[u][0].y), unpack2<T>(v[u][0].z), unpack2<T>(v[u][0].w),
                                 unpack2<T>(v[u][1].x), unpack2<T>(v[u][1].y), unpack2<T>(v[u][1].z), unpack2<T>(v[u][1].w)};
            uint2 q[2];
            const float scale = scaled_codes<2>(f, f32(*reinterpret_cast<const T *>(&top)), q);
            if (live) *reinterpret_cast<uint2 *>(codes + u * cs) = q[0];
            if (second) *reinterpret_cast<uint2 *>(codes + u * cs + 8) = q[1];
            if (live && (lane & 7) == 0) scales[u * ss] = scale;
        }
        x += kSaveRows * xs;
        codes += kSaveRows * cs;
        scales += kSaveRows * ss;
    }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kWarps * 32, 4) restore_kernel(const CheckpointParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int N = GATED ? p.F / 2 : p.F;
    const int c = blockIdx.x * kCols + lane * 8;
    grid_dependency_wait();
    grid_dependents_may_launch();
    if (c >= N) return;
    const Part part = part_of(p);
    const int64_t r0 = part.first + warp;
    T *y = static_cast<T *>(p.x.ptr) + part.seg * p.x.rank_stride + r0 * p.x.row_stride + c;
    const uint8_t *codes = static_cast<const uint8_t *>(p.codes.ptr) + part.seg * p.codes.rank_stride + r0 * p.codes.row_stride + c;
    // 8 neighbours from a multiple of 8 on share a block
    const float *scales = static_cast<const float *>(p.scales.ptr) + part.seg * p.scales.rank_stride + r0 * p.scales.row_stride + c / 128;
    const int up = (c + N) / 128 - c / 128;
    const int64_t ys = kWarps * p.x.row_stride, cs = kWarps * p.codes.row_stride, ss = kWarps * p.scales.row_stride;
    for (int left = part.end - (int)r0; left > 0; left -= kWarps * kRows) {
        uint2 q0[kRows], q1[kRows];
        float s0[kRows], s1[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u * kWarps >= left) break;
            q0[u] = ld_stream8(codes + u * cs);
            s0[u] = __ldg(scales + u * ss);
            if (GATED) {
                q1[u] = ld_stream8(codes + u * cs + N);
                s1[u] = __ldg(scales + u * ss + up);
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u * kWarps >= left) break;
            float2 f[4];
            block_values(f, q0[u], s0[u]);
            if (GATED) {
                float2 w[4];
                block_values(w, q1[u], s1[u]);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul2_rn(silu2(f[j]), w[j]);
            } else if (p.act != EP_ACT_NONE) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = p.act == EP_ACT_GELU   ? gelu2(f[j])
                           : p.act == EP_ACT_SILU ? silu2(f[j])
                                                  : make_float2(f[j].x <= 0.f ? 0.f : f[j].x, f[j].y <= 0.f ? 0.f : f[j].y);
            }
            *reinterpret_cast<uint4 *>(y + u * ys) =
                make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y));
        }
        y += kRows * ys;
        codes += kRows * cs;
        scales += kRows * ss;
    }
}

bool valid(const ep_checkpoint_desc_t *d) {
    if (!d || d->ranks < 1 || d->groups < 1 || (int64_t)d->ranks * d->groups > 65535) return false;
    if (d->rows < 0 || d->rows > 1 << 30) return false;
    if (d->features < 8 || d->features % 8 || d->features > 1 << 24) return false;
    if (d->dtype != EP_DT_BF16 && d->dtype != EP_DT_FP16) return false;
    if (d->activation < EP_ACT_NONE || d->activation > EP_ACT_SWIGLU) return false;
    if ((d->d_count == nullptr) != (d->d_offset == nullptr) || (!d->d_count && d->groups != 1)) return false;
    return aligned(d->d_count, 4) && aligned(d->d_offset, 4);
}

// About 64 rows a block, or 16 where that leaves SMs without a few of them (4346 x 1672 in
// 8 groups, saved: 64 rows 10.6 us, 16 rows 6.2).
CheckpointParams params(const ep_checkpoint_desc_t &d, const ep_rows_t &x, const ep_rows_t &codes,
                        const ep_rows_t &scales, int columns) {
    const int64_t rows = (int64_t)d.rows / d.groups, blocks = (int64_t)columns * d.ranks * d.groups;
    int64_t each = 64;
    while (each > 16 && blocks * ((rows + each - 1) / each) < 1216) each /= 2;
    const int64_t parts = (rows + each - 1) / each;
    return CheckpointParams{Groups{d.d_count, d.d_offset, d.ranks, d.groups, d.rows}, d.features, d.activation,
                            (int)(parts < 1 ? 1 : parts > 256 ? 256 : parts), x, codes, scales};
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_checkpoint_save(const ep_checkpoint_desc_t *d, const ep_rows_t *x, const ep_rows_t *codes,
                               const ep_rows_t *scales, void *stream) {
    EP_RANGE("ep_checkpoint_save");
    if (!valid(d) || !x || !codes || !scales) return EP_ERR_INVALID_ARGS;
    if (d->rows == 0) return EP_SUCCESS;
    if (!valid_rows(*x, d->features, d->ranks > 1) || !valid_codes(*codes, *scales, d->features, d->ranks > 1))
        return EP_ERR_INVALID_ARGS;
    const int columns = (d->features + kSaveCols - 1) / kSaveCols;
    const CheckpointParams p = params(*d, *x, *codes, *scales, columns);
    const dim3 grid(columns, d->ranks * d->groups, p.splits);
    cudaError_t e = cudaSuccess;
    with_type(d->dtype, [&](auto type) {
        e = launch_after_previous(save_kernel<decltype(type)>, grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream), p);
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

ep_status_t ep_checkpoint_restore(const ep_checkpoint_desc_t *d, const ep_rows_t *codes, const ep_rows_t *scales,
                                  const ep_rows_t *y, void *stream) {
    EP_RANGE("ep_checkpoint_restore");
    if (!valid(d) || !codes || !scales || !y) return EP_ERR_INVALID_ARGS;
    const bool gated = d->activation == EP_ACT_SWIGLU;
    const int N = gated ? d->features / 2 : d->features;
    if (N % 8) return EP_ERR_INVALID_ARGS;
    if (d->rows == 0) return EP_SUCCESS;
    if (!valid_rows(*y, N, d->ranks > 1) || !valid_codes(*codes, *scales, d->features, d->ranks > 1))
        return EP_ERR_INVALID_ARGS;
    const int columns = (N + kCols - 1) / kCols;
    const CheckpointParams p = params(*d, *y, *codes, *scales, columns);
    const dim3 grid(columns, d->ranks * d->groups, p.splits);
    cudaError_t e = cudaSuccess;
    with_type(d->dtype, [&](auto type) {
        using T = decltype(type);
        e = launch_after_previous(gated ? restore_kernel<T, true> : restore_kernel<T, false>, grid, kWarps * 32, 0,
                                  static_cast<cudaStream_t>(stream), p);
    });
    return e == cudaSuccess ? EP_SUCCESS : EP_ERR_GPU_OP;
}

}  // extern "C"
