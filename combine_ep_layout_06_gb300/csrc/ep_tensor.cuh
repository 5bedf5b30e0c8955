// Tensor-core building blocks for sm_103a: TMA tile loads, tcgen05 matrix
// instructions with accumulators in tensor memory, and the descriptors both
// take, following the PTX ISA's chapters on cp.async.bulk.tensor and tcgen05.
#pragma once

#include <cuda.h>

#include "ep_rows.cuh"

namespace ep {

// ------------------------------------------------------------- bounded waits

constexpr uint64_t kTensorWaitNs = 1000000000ull;

// PEER: the barrier is signalled by ordinary instructions of the other CTA
// of the pair (copies and matrix instructions need no cluster-wide order).
template <bool PEER = false>
__device__ __forceinline__ bool tensor_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (PEER)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// What a CTA's waits share, in its shared memory.  `loaded` moves with every
// slice that the CTA loads; `gave_up` is set by a wait that runs out, and seen by
// the others.
struct Watch {
    int gave_up;
    uint32_t loaded;
};
// Waits for `parity` of an mbarrier, until a second has passed without another
// slice loaded.  A limit on the whole wait would end work that goes on: an
// epilogue waits for all of a tile's slices, 2^23 of them in the weight gradient
// of a group of 2^30 rows.
template <bool PEER>
__device__ __noinline__ bool tensor_wait_long(uint32_t bar, uint32_t parity, volatile Watch *watch) {
    uint64_t t0 = 0;
    uint32_t seen = 0;
    for (uint32_t it = 0; it < (1u << 26); ++it) {
        if (tensor_try<PEER>(bar, parity)) return true;
        if ((it & 63) == 63) {
            if (watch->gave_up) return false;
            const uint64_t now = globaltimer_ns();
            const uint32_t loaded = watch->loaded;
            if (t0 == 0 || loaded != seen) {
                t0 = now;
                seen = loaded;
                it = 63;
            } else if (now - t0 > kTensorWaitNs) {
                break;
            }
        }
    }
    watch->gave_up = 1;
    return false;
}
template <bool PEER = false>
__device__ __forceinline__ bool tensor_wait(uint32_t bar, uint32_t parity, volatile Watch *watch) {
    return tensor_try<PEER>(bar, parity) || tensor_wait_long<PEER>(bar, parity, watch);
}
// The same by a whole warp, with one answer for all its lanes.
template <bool PEER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile Watch *watch) {
    return __all_sync(0xffffffffu, tensor_wait<PEER>(bar, parity, watch));
}
// One lane of the warp, the same one each time.  Code that only it runs,
// inside control flow that the whole warp follows, keeps its operands in
// uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// ------------------------------------------------------------ pairs of CTAs
// Two CTAs of a cluster share each matrix instruction.

__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

// ------------------------------------------------------------------ TMA tiles
// For a pair (PAIR) `bar` is in the shared memory of either CTA; for a single
// CTA in its own.

template <bool PAIR = true>
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                          int y, int z) {
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%3, %4, %5}], [%2];"
                     :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%3, %4, %5}], [%2];"
                     :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
template <bool PAIR = true>
__device__ __forceinline__ void tma_load5(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                          int y, int z, int u, int v) {
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
                     :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
                     :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v) : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// -------------------------------------------------------------------- tcgen05

// Shared-memory matrix descriptor of a 128-byte-swizzled tile of 16-bit
// elements.  K-major (rows of 64 k): 8-row groups are `stride` = 1024 bytes
// apart.  MN-major (rows of 64 m or n, one row per k): 8-k groups are 1024
// bytes apart, the next 64 m or n `leading` bytes on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(leading >> 4) << 16) |
           ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16 with fp32 accumulators; both operands
// have the same type.
__host__ __device__ constexpr uint32_t f16_idesc(bool bf16, bool a_mn, bool b_mn, int m) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_n(int n) { return (uint32_t)(n >> 3) << 17; }

// One instruction of the pair, by the first CTA's thread: m = 256, rows
// 0-127 of A and of the accumulator in the first CTA, 128-255 in the second;
// each CTA holds half of B's n rows.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// One instruction of a single CTA: m = 128.
__device__ __forceinline__ void mma_f16_single(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// Arrives on the mbarrier once every matrix instruction issued so far by
// this thread is complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
// The same, at the barrier's place in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
                 "[%0], %1;" :: "r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void mma_commit_single(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
// Taken and freed by one warp of a CTA.
__device__ __forceinline__ void tmem_alloc_single(uint32_t smem_slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_single(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(columns)
                 : "memory");
}
// Taken and freed by one warp of each CTA of the pair together.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(columns)
                 : "memory");
}
__device__ __forceinline__ void tcgen_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 lanes x 32 columns of fp32: r[c] is column c of the thread's lane, there
// after tmem_wait (which the values pass through, so that no use of them can
// come before it).
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
          "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
          "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
          "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :: "memory");
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
          "+r"(r[15])
        :: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------ tensor maps (host)

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
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

inline bool encode(CUtensorMap *map, int dtype, void *ptr, int rank, const uint64_t *dims, const int64_t *strides,
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
inline bool encode_rows(CUtensorMap *map, int dtype, const ep_rows_t &r, int64_t width, int64_t rows, int64_t outer,
                 uint32_t box_rows) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)rows, (uint64_t)outer};
    const int64_t strides[3] = {1, r.row_stride, outer > 1 ? r.rank_stride : r.row_stride};
    const uint32_t box[3] = {64, box_rows, 1};
    return encode(map, dtype, r.ptr, 3, dims, strides, box);
}

// Gated weights [G][2][N][K]: one box is 8 features of the gate, the same 8
// of the up half, and so on for 8 * `eights` features.
inline bool encode_gated(CUtensorMap *map, int dtype, const ep_rows_t &w, int64_t K, int64_t N, int64_t G,
                         uint32_t eights = 8) {
    const uint64_t dims[5] = {(uint64_t)K, 8, 2, (uint64_t)(N / 8), (uint64_t)G};
    const int64_t strides[5] = {1, w.row_stride, N * w.row_stride, 8 * w.row_stride,
                                G > 1 ? w.rank_stride : w.row_stride};
    const uint32_t box[5] = {64, 8, 2, eights, 1};
    return encode(map, dtype, w.ptr, 5, dims, strides, box);
}

}  // namespace ep
