// Activations kept in block-scaled 8 bits between forward and backward: saved,
// and restored through the activation.
//
// Element-wise over the rows of every group and bound by memory.  A lane takes 8
// neighbouring values, so 16 lanes hold a block of 128; a warp takes 256
// values of a row, a block's warps take rows in turn.
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

template <typename T> __global__ void __launch_bounds__(kWarps * 32) save_kernel(const CheckpointParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * kCols + lane * 8;
    const bool live = c < p.F;
    const Part part = part_of(p);
    const T *x = static_cast<const T *>(p.x.ptr) + part.seg * p.x.rank_stride + c;
    uint8_t *codes = static_cast<uint8_t *>(p.codes.ptr) + part.seg * p.codes.rank_stride + c;
    float *scales = static_cast<float *>(p.scales.ptr) + part.seg * p.scales.rank_stride + c / 128;
    for (int64_t r = part.first + warp; r < part.end; r += kWarps * kRows) {
        uint4 v[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t i = r + u * kWarps;
            v[u] = live && i < part.end ? ld_stream16(x + i * p.x.row_stride) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t i = r + u * kWarps;
            const float2 f[4] = {unpack2<T>(v[u].x), unpack2<T>(v[u].y), unpack2<T>(v[u].z), unpack2<T>(v[u].w)};
            float scale;
            const uint2 q = block_codes(f, &scale);
            if (!live || i >= part.end) continue;
            *reinterpret_cast<uint2 *>(codes + i * p.codes.row_stride) = q;
            if ((lane & 15) == 0) scales[i * p.scales.row_stride] = scale;
        }
    }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) restore_kernel(const CheckpointParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int N = GATED ? p.F / 2 : p.F;
    const int c = blockIdx.x * kCols + lane * 8;
    if (c >= N) return;
    const Part part = part_of(p);
    T *y = static_cast<T *>(p.x.ptr) + part.seg * p.x.rank_stride + c;
    const uint8_t *codes = static_cast<const uint8_t *>(p.codes.ptr) + part.seg * p.codes.rank_stride + c;
    const float *scales = static_cast<const float *>(p.scales.ptr) + part.seg * p.scales.rank_stride;
    const int b0 = c / 128, b1 = (c + N) / 128;      // 8 neighbours from a multiple of 8 on share a block
    for (int64_t r = part.first + warp; r < part.end; r += kWarps * kRows) {
        uint2 q0[kRows], q1[kRows];
        float s0[kRows], s1[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t i = r + u * kWarps;
            if (i >= part.end) continue;
            q0[u] = ld_stream8(codes + i * p.codes.row_stride);
            s0[u] = __ldg(scales + i * p.scales.row_stride + b0);
            if (GATED) {
                q1[u] = ld_stream8(codes + i * p.codes.row_stride + N);
                s1[u] = __ldg(scales + i * p.scales.row_stride + b1);
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t i = r + u * kWarps;
            if (i >= part.end) continue;
            float f[8];
            block_values(f, q0[u], s0[u]);
            if (GATED) {
                float up[8];
                block_values(up, q1[u], s1[u]);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = f[j] * sigmoidf(f[j]) * up[j];
            } else {
                activate8(p.act, f);
            }
            store8<T>(y + i * p.x.row_stride, f);
        }
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

CheckpointParams params(const ep_checkpoint_desc_t &d, const ep_rows_t &x, const ep_rows_t &codes,
                        const ep_rows_t &scales) {
    const int64_t parts = ((int64_t)d.rows / d.groups + 63) / 64;      // about 64 rows each
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
    const CheckpointParams p = params(*d, *x, *codes, *scales);
    const dim3 grid((d->features + kCols - 1) / kCols, d->ranks * d->groups, p.splits);
    with_type(d->dtype, [&](auto type) {
        save_kernel<decltype(type)><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return launched();
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
    const CheckpointParams p = params(*d, *y, *codes, *scales);
    const dim3 grid((N + kCols - 1) / kCols, d->ranks * d->groups, p.splits);
    with_type(d->dtype, [&](auto type) {
        using T = decltype(type);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (gated) restore_kernel<T, true><<<grid, kWarps * 32, 0, st>>>(p);
        else restore_kernel<T, false><<<grid, kWarps * 32, 0, st>>>(p);
    });
    return launched();
}

}  // extern "C"
