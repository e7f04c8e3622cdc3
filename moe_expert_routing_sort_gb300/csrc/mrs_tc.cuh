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

// Eight columns of the lane, added as fp32.
__device__ __forceinline__ void tmem_add8(uint32_t addr, uint32_t* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(r[i]));
}

// 16 lanes x 32 columns of 32 bits in fragments: of eight columns (8 k on) a thread t of the warp has
// columns 2 (t % 4) and the next, of lane t / 4 in r[4 k], r[4 k + 1] and of lane t / 4 + 8 in
// r[4 k + 2], r[4 k + 3].
__device__ __forceinline__ void tmem_load_fragments(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// Four 8 x 8 matrices of 16-bit elements, transposed: thread t has row t / 4, columns 2 (t % 4) and
// the next of each; column c of matrix i goes to the 16 bytes at thread 8 i + c's address.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                 uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
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
// 16 bytes, or 16 zeros (bytes == 0: nothing is read).  The rest of their 256 bytes is fetched to L2,
// for rows that are copied 128 bytes a step.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
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

// A tile of shared memory to global memory, as the map says; what lies outside is left out.  One
// thread issues, closes groups and waits.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y,
                                             int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          map),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The groups so far have been read from shared memory; and have been written.
__device__ __forceinline__ void tma_store_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------------ pairs of CTAs
// Two CTAs of a cluster work on one product of 256 rows: each holds its half of both operands and
// of the sums, and the CTA of rank 0 issues for both.
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of both CTAs; what either wrote to shared memory before is visible behind it.
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(where)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
// One arrival on the barrier that lies at this address in the CTA of rank 0.  (Its scope is the
// default one: what it announces is read by this CTA's own tensor core, or was read from its tensor
// memory.  A release to the cluster takes 2000 clocks beside copies in flight: 3900 us and not 1377
// for T = 8192, E = 64, 7168 -> 2048.)
__device__ __forceinline__ void pair_arrive_first(unsigned long long* mbar) {
  asm volatile(
      "{ .reg .b32 at; mapa.shared::cluster.u32 at, %0, 0;\n"
      " mbarrier.arrive.shared::cluster.b64 _, [at]; }" ::"r"(smem_u32(mbar))
      : "memory");
}
// thread_wait for arrivals that may come from the other CTA.
__device__ __forceinline__ bool pair_wait(unsigned long long* mbar, uint32_t phase,
                                          unsigned long long limit_ns) {
  if (limit_ns == 0ull) return false;
  unsigned long long t0 = 0ull;
  for (uint32_t i = 1;; ++i) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(smem_u32(mbar)), "r"(phase)
        : "memory");
    if (done != 0u) return true;
    if ((i & 63u) != 0u) continue;
    const unsigned long long t = globaltimer_ns();
    if (t0 == 0ull) t0 = t;
    else if (t - t0 > limit_ns) return false;
  }
}
// Arrives on the barrier at this address of both CTAs once everything this thread issued before
// has completed.
__device__ __forceinline__ void pair_commit(unsigned long long* mbar) {
  asm volatile(
      "{ .reg .b16 m; mov.b16 m, 3;\n"
      " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], m; }" ::"r"(smem_u32(mbar))
      : "memory");
}
__device__ __forceinline__ void pair_commit_first(unsigned long long* mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(mbar))
      : "memory");
}
// 256 x N products of 32 bytes of each row; 16-bit operands, or e4m3 ones.
template <bool kFp8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                         bool add) {
  if constexpr (kFp8)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(add ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(add ? 1u : 0u)
        : "memory");
}
// Instruction word of these kinds: fp32 sums, M = 256 rows of both CTAs by N; type: 0 fp16 or e4m3,
// 1 bf16 (both operands); an operand is transposed where its rows run along the contraction.
__device__ __forceinline__ uint32_t pair_word(int type, bool transpose_a, bool transpose_b, int N) {
  return (1u << 4) | (static_cast<uint32_t>(type) << 7) | (static_cast<uint32_t>(type) << 10) |
         (transpose_a ? 1u << 15 : 0u) | (transpose_b ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | ((256u >> 4) << 24);
}
// A transposed operand: lines of 64 elements (128 bytes, swizzled by 128) along its rows, one line
// for each of the contraction's `deep` positions, the next 64 elements behind them.
__device__ __forceinline__ uint64_t desc_lines128(uint32_t smem_addr, int deep) {
  return static_cast<uint64_t>((smem_addr & 0x3ffffu) >> 4) |
         (static_cast<uint64_t>(deep * 128 >> 4) << 16) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// The address of a CTA's shared memory in the CTA of rank 0.
__device__ __forceinline__ uint32_t pair_first(const void* p) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(p)));
  return at;
}
// Tensor copies into this CTA whose bytes are counted on a barrier of either CTA of the pair
// (mbar: an address of the cluster).
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                             int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(mbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace mrs
