// tcgen05, TMA and mbarrier instructions of the paged attention kernels (mtp_paged_tc.cu,
// mtp_chunk_tc.cu), and the tensor map of a paged cache.
#pragma once

#include <cuda.h>

#include "mtp_paged.cuh"

namespace mtp {
namespace pgt {

__device__ __forceinline__ unsigned sa(const void* p) { return static_cast<unsigned>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool test_wait(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool try_wait(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// Bounded wait; false when this CTA has given up (the word `dead`) or gives up here.
static __device__ __noinline__ bool wait_slow(unsigned bar, unsigned parity, volatile int* dead, long long limit) {
  const long long t0 = clock64();
  while (!try_wait(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > limit) {
      *dead = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(unsigned bar, unsigned parity, volatile int* dead, long long limit) {
  return test_wait(bar, parity) || wait_slow(bar, parity, dead, limit);
}
__device__ __forceinline__ void tma_4d(unsigned dst, const CUtensorMap* map, int x, int t, int h, int page, unsigned bar,
                                       unsigned long long policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(map), "r"(x), "r"(t), "r"(h), "r"(page), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_4d(unsigned dst, const CUtensorMap* map, int x, int t, int h, int page, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(t), "r"(h), "r"(page), "r"(bar)
      : "memory");
}
// Shared-memory descriptors, 128-byte swizzle: 8-row groups are 1024 bytes apart; in the MN-major
// form (rows = K index, 64 MN elements per row) `lead` is the distance of the next 64. The low
// word holds the address, so a step is one 32-bit addition.
__device__ __forceinline__ constexpr unsigned desc_lo(unsigned addr, unsigned lead) {
  return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
constexpr unsigned kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// One elected thread issues (its caller's branch is made by elect.sync, which keeps the operands
// in uniform registers: 36 cycles per instruction instead of 53, measured; any other choice of
// the thread makes the compiler guard every instruction).
__device__ __forceinline__ void mma(unsigned d, unsigned a, unsigned b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ bool elect() {
  unsigned e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void commit(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void ld8(unsigned t, float* v) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void ld4(unsigned t, float* v) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(t));
}
__device__ __forceinline__ void st4(unsigned t, const float* v) {
  const unsigned* r = reinterpret_cast<const unsigned*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A map of a bf16 tensor of four dimensions (the innermost first, strides in bytes from the second
// on), 128-byte swizzle, zeros outside.
int encode_map(CUtensorMap* map, const void* p, const unsigned long long* dims, const unsigned long long* strides,
               const unsigned* box_dims, const char* what);
// A map of the pages from `p` (k or v of the cache): boxes of `rows` tokens x 64 dims of one KV head
// of one page, 128-byte swizzle; rows of no page read as zeros.
int make_map(CUtensorMap* map, const pg::Cache& c, const void* p, int rows);

}  // namespace pgt
}  // namespace mtp
