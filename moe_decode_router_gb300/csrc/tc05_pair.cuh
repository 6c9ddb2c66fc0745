// Pairs of CTAs (cta_group::2) on top of tc05.cuh: one MMA over two SMs.  The even CTA
// of the pair (cluster rank 0) issues; each CTA's shared memory holds its 128 rows of A
// and its half of B's rows at the same offsets, and each CTA's tensor memory receives
// its 128 rows of D.  Written from the PTX ISA description.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "tc05_e4m3.cuh"

namespace flint {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

namespace tc05 {

// Shared-cluster address of `addr` (a shared-memory address of this CTA) in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrivals on an mbarrier of either CTA of the pair.  Their release covers this CTA alone,
// which is enough for what they announce here: operands in this SM's own memories, written
// for the tensor cores before (fence.proxy.async, tcgen05.wait::st), or its accumulator read
// (tcgen05.wait::ld).  A release to the cluster waits for every write under way, some 500
// cycles: the integer product of 8191 x 4096 x 4096 took 518 us with it.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void arrive_expect_cluster(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr), "r"(bytes) : "memory");
}
// A cluster barrier that orders execution alone.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Bits of the instruction descriptor: an operand whose M or N dimension is contiguous in memory.
constexpr uint32_t A_ROWS_CONTIGUOUS = 1u << 15, B_ROWS_CONTIGUOUS = 1u << 16;

// Matrix descriptor of a 16-bit operand whose M (or N) dimension is contiguous, 128-byte
// swizzle: pieces of 64 of M x the tile's rows of K, `piece` bytes apart (leading byte
// offset); 8 rows of K are 1024 bytes (stride byte offset).
__device__ __forceinline__ uint64_t sw128_rows_desc(uint32_t smem_addr, uint32_t piece) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | (uint64_t)(piece >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// D (+)= A * B^T over both CTAs of the pair, 256 x N x 64: four instructions whose operands lie
// DA and DB (in descriptor units) apart, of the lane that elect.sync picks of a whole
// converged warp of the even CTA; then the stage's release: an arrival on an mbarrier of
// either CTA (shared-cluster addresses) when all MMAs that the lane issued so far have
// completed.  In one piece, as an election for every instruction made a step 350 cycles long.
template <int DA>
__device__ __forceinline__ void mma_pair_step(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t db,
                                              uint32_t idesc, uint32_t accumulate, uint32_t bar0, uint32_t bar1) {
  asm volatile(
      "{\n .reg .pred p, q, e;\n .reg .b64 a1, a2, a3, b1, b2, b3, db;\n"
      " setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, %4, %4;\n cvt.u64.u32 db, %5;\n"
      " add.s64 a1, %1, %8;\n add.s64 a2, a1, %8;\n add.s64 a3, a2, %8;\n"
      " add.s64 b1, %2, db;\n add.s64 b2, b1, db;\n add.s64 b3, b2, db;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, q;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, q;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, q;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%6];\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%7];\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(db), "r"(bar0), "r"(bar1), "n"(DA)
      : "memory");
}
// One of its instructions (256 x N x 16).
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Four with A in tensor memory, 8 columns each: lanes are its rows, a column holds two neighbours of K.
__device__ __forceinline__ void mma_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q, e;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n"
      " setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, %4, %4;\n"
      " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, q;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, q;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, q;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 TMEM lanes x 16 consecutive 32-bit columns, laid out as by ld_16x256b_x4.
__device__ __forceinline__ void ld_16x256b_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// 16 32-bit columns of the warp's 32 lanes (thread i -> lane i), and the wait for such stores.
__device__ __forceinline__ void st_32x32b_x16(uint32_t taddr, const uint4 (&v)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w),
      "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Arrives (once) on an mbarrier of either CTA, given by its shared-cluster address, when all
// MMAs that the warp issued that way so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t cluster_addr) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(cluster_addr)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Copies of a tile into this CTA's shared memory, counted on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int v,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(v), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_5d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int v, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w), "r"(bar)
      : "memory");
}

}  // namespace tc05
}  // namespace flint
