// Inline-PTX helpers for kernels on the fifth-generation tensor cores:
// mbarriers with bounded waits, tcgen05 matrix products, tensor memory.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace kvq {
namespace um {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- mbarriers

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tests the phase of that parity; the thread sleeps in hardware until it is
// done, or about a millisecond.
constexpr uint32_t kTryNs = 1000000;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase of that parity, two seconds at most; *stop is raised
// when the time runs out and ends every other wait of the CTA too.
constexpr uint64_t kWaitLimitNs = 2000000000ull;
// A whole warp calls it, and leaves it converged, as the .aligned instructions
// behind it need.
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  if (!mbar_try(bar, parity)) {
    const uint64_t t0 = now_ns();
    while (!mbar_try(bar, parity) && !*stop)
      if (now_ns() - t0 > kWaitLimitNs) *stop = 1;
  }
  __syncwarp();
}

// ---------------------------------------------------------------- pairs of fp32
// Two fp32 operations an instruction, each rounded as the single one.

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---------------------------------------------------------------- registers
// Sets a warpgroup's registers a thread to N, of FROM at launch: more are taken
// from what others gave back (the instruction waits for them), fewer are given
// back.  Each direction has its own instruction, and the other is illegal.
template <int N, int FROM>
__device__ __forceinline__ void regs_set() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "registers a thread");
  if constexpr (N > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------- fences

// Earlier generic writes to shared memory become visible to the tensor cores'
// reads (followed by an mbarrier arrival).
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------------- tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {   // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {   // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

#define KVQ_R8(A, I) "=f"(A[I]), "=f"(A[I + 1]), "=f"(A[I + 2]), "=f"(A[I + 3]), "=f"(A[I + 4]), "=f"(A[I + 5]), \
                     "=f"(A[I + 6]), "=f"(A[I + 7])
#define KVQ_P8(A, I) "+f"(A[I]), "+f"(A[I + 1]), "+f"(A[I + 2]), "+f"(A[I + 3]), "+f"(A[I + 4]), "+f"(A[I + 5]), \
                     "+f"(A[I + 6]), "+f"(A[I + 7])
#define KVQ_I8(A, I) "r"(A[I]), "r"(A[I + 1]), "r"(A[I + 2]), "r"(A[I + 3]), "r"(A[I + 4]), "r"(A[I + 5]), \
                     "r"(A[I + 6]), "r"(A[I + 7])
#define KVQ_F8(A, I) "f"(A[I]), "f"(A[I + 1]), "f"(A[I + 2]), "f"(A[I + 3]), "f"(A[I + 4]), "f"(A[I + 5]), \
                     "f"(A[I + 6]), "f"(A[I + 7])

// 32 columns of the warp's 32 lanes: lane i gets row i.  The values may be
// used after tmem_ld_wait on the same array.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : KVQ_R8(x, 0), KVQ_R8(x, 8), KVQ_R8(x, 16), KVQ_R8(x, 24)
      : "r"(addr));
}
// Waits for every load of this thread; naming the array keeps its uses behind the wait.
__device__ __forceinline__ void tmem_ld_wait(float (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : KVQ_P8(x, 0), KVQ_P8(x, 8), KVQ_P8(x, 16), KVQ_P8(x, 24)::"memory");
}
// Eight columns there and back.
__device__ __forceinline__ void tmem_ld8_wait(uint32_t addr, float (&x)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : KVQ_R8(x, 0)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::KVQ_F8(x, 0),
               "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::KVQ_I8(x, 0),
      KVQ_I8(x, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- matrix products

// Instruction descriptor of fp16 x fp16 -> fp32, M = 128: D fp32 (bit 4), A and
// B fp16 (0), B along N in memory (bit 16) or along K, N / 8 (bits 17..), M / 16
// (bits 24..).
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_along_n) {
  return (1u << 4) | (b_along_n ? 1u << 16 : 0u) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(128 / 16) << 24);
}
// Shared-memory descriptor of a tile in rows of 128 bytes with the 128-byte
// swizzle (16-byte chunk index XOR row mod 8): groups of eight rows follow one
// another (stride 1024 bytes); the next 128 bytes of a row lie `lead` bytes on
// (used where B runs along N).  Version 1 (bit 46), swizzle mode 2 (bits 61..).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// D (+)= A B, one 16-deep step: A from shared memory, or from tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
// The barrier gets one arrival when every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace um
}  // namespace kvq
