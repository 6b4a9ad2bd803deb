// The 5th-generation tensor core (tcgen05) as the kernels use it: fp16
// products with the A operand in tensor memory, the B operand in swizzled
// shared memory and float32 sums in tensor memory.
//
// Tensor memory is 128 lanes x 512 columns of 32 bits; an address is lane << 16
// | column.  Warp w of a CTA reads and writes lanes 32 (w % 4) .. + 31.
#pragma once

#include "common.cuh"

namespace epq {

// All 512 columns.  Called by one whole warp; the address goes to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t *address) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(address)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t address) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(address) : "memory");
}

// Order of tcgen05 instructions and what other threads do before / after a barrier.
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared memory that was written by ordinary stores is read by the tensor core.
__device__ __forceinline__ void fence_shared_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// `bar` completes a phase when the thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// fp16 x fp16 -> float32, M = 128; kMnMajorB: B's rows in memory run along n.
template <int N, bool kMnMajorB>
__host__ __device__ constexpr uint32_t mma_f16_shape() {
  return (1u << 4) | (kMnMajorB ? 1u << 16 : 0u) | (static_cast<uint32_t>(N / 8) << 17) | ((128u / 16) << 24);
}

// B in shared memory: rows of 128 bytes in groups of 8 (1024 bytes, aligned)
// whose 16-byte pieces are permuted by the row's index (128-byte swizzle).
// `lead`: bytes between column groups of 64 where B's rows run along n.
__device__ __forceinline__ uint64_t mma_b_descriptor(uint32_t address, uint32_t lead) {
  return static_cast<uint64_t>((address & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// d (+)= a b over 16 of k: a 8 columns of tensor memory.
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 32 columns of the thread's lane.  The wait is part of the instruction's text:
// nothing that uses the values can be moved in front of it.
__device__ __forceinline__ void tmem_load32(uint32_t address, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
        "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]),
        "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]),
        "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
      : "r"(address)
      : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t address, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
        "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
      : "r"(address)
      : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t address, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(x[0]),
      "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
      "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(address)
      : "memory");
}

// 32 columns of 16 lanes, four threads to a lane: of columns 8 n .. 8 n + 7
// thread t has 2 (t % 4) and the next one, x[4 n] and x[4 n + 1] for the lane
// t / 4, x[4 n + 2] and x[4 n + 3] for the lane 8 further on.
__device__ __forceinline__ void tmem_store_quads(uint32_t address, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(x[0]),
      "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
      "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(address)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace epq
