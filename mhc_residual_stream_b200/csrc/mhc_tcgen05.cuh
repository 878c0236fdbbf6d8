// PTX wrappers of the fifth-generation tensor core (tcgen05) and of the
// tensor-map copies that feed it (sm_100a).
#pragma once

#include "mhc_device.cuh"

namespace mhc {

// One lane of the converged warp, the same one every time. The issuing loops run in
// all lanes and elect at the instruction: their operands then stay in uniform
// registers (a K block issued inside an `if (lane == 0)` took 685 cycles).
__device__ __forceinline__ bool elect_one() {
  unsigned r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- tensor-map copies (this GPU's memory)

__device__ __forceinline__ void tma_load_2d(unsigned dst, const void* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Four rows of a 2-D map (box one row high) at columns x..: the rows land one
// after the other at dst.
__device__ __forceinline__ void tma_gather4(unsigned dst, const void* map, int x, int4 rows, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- tensor memory

__device__ __forceinline__ void tmem_alloc(unsigned* slot, unsigned cols) {  // whole warp; cols a power of two >= 32
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc(unsigned addr, unsigned cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

// 16 consecutive columns of the warp's 32 lanes: thread l gets lane l's values.
__device__ __forceinline__ void tmem_ld16(unsigned addr, float (&v)[16]) {
  unsigned r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------------- MMA (one issuing thread)

// Shared-memory operand descriptor of a K-major tile of 128-byte rows in the
// 128-byte swizzle (8-row groups 1024 bytes apart): the high word is the same for
// every tile, the low word takes the address (1024-byte aligned, plus 32 bytes per
// K step within the row: 2 units).
constexpr unsigned kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ unsigned desc_lo(unsigned addr) { return ((addr & 0x3ffffu) >> 4) | (1u << 16); }
// Descriptor of a 512-byte scale tile (32 rows of 16 bytes, 8-row groups 128
// bytes apart, no swizzle).
__device__ __forceinline__ uint64_t desc_scales(unsigned addr) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (8ull << 32) | (1ull << 46);
}

// D[128 x N] (+)= A[128 x 16] B[N x 16]^T, bf16 operands (low descriptor words),
// fp32 accumulator.
__device__ __forceinline__ void mma_bf16(unsigned d, unsigned a, unsigned b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi)
      : "memory");
}
// D[128 x N] (+)= A[128 x 32] B[N x 32]^T, E4M3 operands with one E8M0 scale per
// row and 32 elements (tensor memory at sa, sb; the byte is in idesc).
__device__ __forceinline__ void mma_mxf8(unsigned d, unsigned a, unsigned b, unsigned idesc, unsigned sa, unsigned sb,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(sa), "r"(sb), "n"(kDescHi)
      : "memory");
}
// A 512-byte scale tile into 4 columns of tensor memory, the 32 lanes repeated in
// every quarter.
__device__ __forceinline__ void tmem_copy_scales(unsigned addr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(addr), "l"(desc) : "memory");
}
// Arrive on bar once every MMA and copy this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// mbar_try_wait on a barrier that other CTAs of the cluster arrive on.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace mhc
