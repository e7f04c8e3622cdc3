// mrs_tc.cuh -- the fifth-generation tensor cores, tensor memory and tensor copies: thin wrappers
// of the PTX instructions, and the descriptors they take.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mrs_device.cuh"

namespace mrs {

// ------------------------------------------------------------------------ tensor memory
// All 32 lanes of one warp; the address lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(where)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 lanes (the warp's quarter of tensor memory) x 32 columns of 32 bits.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// Every load of this thread so far has arrived; named registers are not read before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// -------------------------------------------------------------------------- descriptors
// Shared-memory operand: rows of 128 bytes swizzled by 128, eight rows (1024 bytes) a group.
__device__ __forceinline__ uint64_t desc_rows128(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr & 0x3ffffu) >> 4) | (uint64_t{1} << 16) |
         (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// Scale bytes: 32 rows of 16 bytes, no swizzle, eight rows (128 bytes) a group.
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr & 0x3ffffu) >> 4) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}
// Instruction word of kind::mxf4 with one scale byte (E8M0) per 32 elements: E2M1 operands, fp32
// sums, M x N, scale ids (0 or 2: which half of the 4 scale bytes a row's 64 elements take).
__device__ __forceinline__ constexpr uint32_t mxf4_word(int M, int N, int id) {
  return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) |
         (static_cast<uint32_t>(id) << 29);
}

// ------------------------------------------------------------------- one thread issues
// One lane of a converged warp.  The operands of these instructions are the warp's, not a
// lane's: behind this choice the compiler knows that one lane acts and keeps them in uniform
// registers; behind `lane == 0` it does not, and issuing took longer than the products.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0u;
}
// 512 bytes of scales to tensor memory, repeated in its four lane quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                            uint32_t scale_a, uint32_t scale_b, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(word), "r"(scale_a), "r"(scale_b), "r"(add ? 1u : 0u)
      : "memory");
}
// Arrives on the barrier once everything this thread issued before has completed.
__device__ __forceinline__ void tc_commit(unsigned long long* mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(mbar))
      : "memory");
}

// Wait of one thread for phase `phase` of `mbar`, at most about `limit_ns` (0: report a timeout at
// once without looking, a test hook).  The clock is only asked every 64 looks.
__device__ __forceinline__ bool thread_wait(unsigned long long* mbar, uint32_t phase,
                                            unsigned long long limit_ns) {
  if (limit_ns == 0ull) return false;
  unsigned long long t0 = 0ull;
  for (uint32_t i = 1; !mbar_try_wait(mbar, phase); ++i) {
    if ((i & 63u) != 0u) continue;
    const unsigned long long t = globaltimer_ns();
    if (t0 == 0ull) t0 = t;
    else if (t - t0 > limit_ns) return false;
  }
  return true;
}
// The same for a whole warp: every lane looks (each gets the acquire), the answer is uniform.
__device__ __forceinline__ bool warp_wait(unsigned long long* mbar, uint32_t phase,
                                          unsigned long long limit_ns) {
  return __all_sync(kFull, thread_wait(mbar, phase, limit_ns));
}

// ------------------------------------------------------------------------- thread copies
// 16 bytes from global to shared memory, in the background.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's last kLeft closed groups have landed.
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// 4 bytes, of which the first `bytes` are read and the others are zeros.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// One arrival on the barrier (counted in its expected number) once this thread's copies so far
// have landed.
__device__ __forceinline__ void copy_arrive(unsigned long long* mbar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(mbar)) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ------------------------------------------------------------------------- tensor copies
__device__ __forceinline__ void mbar_arrive(unsigned long long* mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(mbar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(unsigned long long* mbar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, unsigned long long* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(mbar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
}  // namespace mrs
