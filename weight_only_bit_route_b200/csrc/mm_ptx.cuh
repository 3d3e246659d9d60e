// PTX wrappers of the 16-bit and 8-bit expert products (grouped_mm.cu, grouped_wgrad.cu) beyond those of
// tc_ptx.cuh: 3D tensor copies, matrix descriptors of operands stored along M or N, CTA pairs.
#pragma once

#include "tc_ptx.cuh"

namespace moe {

// Bounded warp-wide wait (as g_wait_w) that lets the hardware suspend the warp for up to 10 us a try instead of polling:
// the waiting roles then cost no power, which is what bounds long batches.
__device__ __forceinline__ bool g_try_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000u) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool g_wait_long(uint32_t bar, uint32_t parity, volatile GAbort* ab) {
    if (__all_sync(0xffffffffu, g_try_long(bar, parity))) return true;
    const unsigned long long t0 = g_timer();
    while (true) {
        if (__all_sync(0xffffffffu, g_try_long(bar, parity))) return true;
        if (__any_sync(0xffffffffu, ab->flag || g_timer() - t0 > ab->limit_ns)) return false;
    }
}

__device__ __forceinline__ void g_tma3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// The same copies of a CTA pair: the barrier may be the other CTA's.
__device__ __forceinline__ void g_tma3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void g_tma2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void g_tma4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}
__device__ __forceinline__ void g_tma4d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t g_cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of this CTA's shared-memory location in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t g_mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void g_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same without a release, which costs its warp about a thousand cycles: for an arrival that publishes no memory
// (a finished tcgen05.wait::ld says that the accumulator has been read; a barrier's bytes say so themselves)
__device__ __forceinline__ void g_arrive_remote_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void g_expect_remote(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void g_st_cluster4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 16 bytes into another CTA's shared memory, counted there on barrier bar: no fence on either side
__device__ __forceinline__ void g_st_async4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}
__device__ __forceinline__ void g_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ uint32_t g_ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// All threads of the cluster's CTAs (each CTA's threads converged)
__device__ __forceinline__ void g_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without ordering memory (a release would wait for the CTA's global stores): keeps the CTAs alive together
__device__ __forceinline__ void g_cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// Operand stored along M (or N): 64-element rows of 128 bytes, one row per K, 128-byte swizzle.  8-row groups
// of K are 1024 bytes apart (stride offset); the next 64 elements along M (or N) follow at lbo bytes.
__device__ __forceinline__ uint64_t g_desc_mn(uint32_t saddr, uint32_t lbo) {
    return uint64_t((saddr >> 4) & 0x3FFF) | (uint64_t(lbo >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
constexpr uint32_t G_IDESC_A_MN = 1u << 15;     // instruction descriptor: A stored along M
constexpr uint32_t G_IDESC_B_MN = 1u << 16;     // B stored along N
// kind::i8, both operands signed
__device__ __forceinline__ uint32_t g_idesc_s8(int n, int m = 128) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void g_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
template <int CG>
__device__ __forceinline__ void g_mma_s8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Commit to this CTA's barrier, or to the barrier at this offset in both CTAs of the pair
template <int CG>
__device__ __forceinline__ void g_commit_cg(uint32_t bar) {
    if constexpr (CG == 1)
        g_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"(uint16_t(3)) : "memory");
}
// Commit to this CTA's barrier alone
template <int CG>
__device__ __forceinline__ void g_commit_own(uint32_t bar) {
    if constexpr (CG == 1)
        g_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void g_tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void g_tmem_free(uint32_t tmem, uint32_t cols) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

// Tile stores from shared memory (one thread issues, commits and waits); add: += in fp32
__device__ __forceinline__ void g_store3d(const CUtensorMap* map, int x, int y, int z, uint32_t src, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void g_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N committed groups may still be reading shared memory
template <int N>
__device__ __forceinline__ void g_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void g_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Host: 3D tensor map over [z][rows][inner elements] (pitches in bytes).
inline int g_map3(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows, uint64_t z,
                  uint64_t pitch, uint64_t zpitch, uint32_t box_in, uint32_t box_rows) {
    if ((reinterpret_cast<uintptr_t>(base) & 15u) || (pitch & 15u) || (zpitch & 15u)) return MOE_ERR_INVALID_ARG;
    cuuint64_t dims[3] = {inner, rows, z};
    cuuint64_t strides[2] = {pitch, zpitch};
    cuuint32_t box[3] = {box_in, box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = g_encode_fn_ref()(m, type, 3, const_cast<void*>(base), dims, strides, box, es,
                                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

// Host: [z][rows][chunk * chunks] elements seen as [z][chunks][rows][chunk] (chunk: 128 bytes of a row): one box
// holds box_rows rows of each of two neighbouring chunks.
inline int g_map4(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint32_t chunk, uint64_t rows,
                  uint64_t chunks, uint64_t z, uint64_t pitch, uint64_t zpitch, uint32_t box_rows) {
    if ((reinterpret_cast<uintptr_t>(base) & 15u) || (pitch & 15u) || (zpitch & 15u)) return MOE_ERR_INVALID_ARG;
    cuuint64_t dims[4] = {chunk, rows, chunks, z};
    cuuint64_t strides[3] = {pitch, 128, zpitch};
    cuuint32_t box[4] = {chunk, box_rows, 2, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUresult r = g_encode_fn_ref()(m, type, 4, const_cast<void*>(base), dims, strides, box, es,
                                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
