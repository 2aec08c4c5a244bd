// What the tensor-core kernels share: mbarriers with bounded waits, TMA loads,
// tcgen05 fences and commits, shared-memory descriptors, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace moe {
namespace tc {

constexpr long long kWaitCycles = 2000000000LL;   // ~1 s at the B200's clocks

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// whether the phase has completed, at once (try_wait may suspend the thread for
// a while of the hardware's choosing)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// try_wait with a suspend-time hint: a thread whose phase is not complete
// sleeps until it completes or about `ns` nanoseconds pass, instead of
// spinning and taking issue slots from the warps that do the work
__device__ __forceinline__ bool mbar_try_sleep(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// Bounded wait for the phase of `parity` to complete: at most `limit` SM
// cycles. Returns false when the kernel is aborting (another role timed out;
// ignored when !honor_abort) or this wait ran out. Waits for work use the
// launch's bound (Params::wait_limit); the waits for copies and MMAs still in
// flight before the CTA exits keep the full bound, so that nothing lands in
// shared memory or TMEM after the CTA has released it. A bound below ~50 us
// also drops the sleep hint, so the wait notices its deadline promptly; with
// POLL such a bound never suspends the thread at all, so that a phase which is
// not complete at once runs out for certain (a template argument: the choice at
// every wait cost the grouped kernels 2 %).
template <bool POLL = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* status, bool honor_abort = true,
                                          long long limit = kWaitCycles) {
  const bool poll = POLL && limit < 100000;
  if (poll ? mbar_test(bar, parity) : mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  const bool sleep = limit >= 100000;
  const uint32_t af = smem_u32(const_cast<const int*>(abort_flag));
  for (;;) {
    if (sleep  ? mbar_try_sleep(bar, parity, 20000u)
        : POLL ? mbar_test(bar, parity)
               : mbar_try(bar, parity))
      return true;
    uint32_t aborting;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(aborting) : "r"(af) : "memory");
    if (honor_abort && aborting) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      report_status(status, MOE_ERR_TIMEOUT);
      return false;
    }
  }
}

// Every lane waits; the result is the same in all lanes, so the warp stays
// converged for the .sync.aligned tcgen05 instructions that follow.
template <bool POLL = false>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, int* status,
                                               bool honor_abort = true,
                                               long long limit = kWaitCycles) {
  const bool r = mbar_wait<POLL>(bar, parity, abort_flag, status, honor_abort, limit);
  return __all_sync(0xffffffffu, r);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// address of barrier i of an array of 8-byte mbarriers at shared address base
__device__ __forceinline__ uint32_t bar_at(uint32_t base, uint32_t i) { return base + 8u * i; }

// tcgen05.commit from one elected lane of a converged warp
__device__ __forceinline__ void mma_commit_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}

// K-major operand in shared memory, 128-byte swizzle, rows of 128 bytes,
// 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;              // leading byte offset (unused for swizzled K-major)
  d |= (uint64_t)(1024 >> 4) << 32;    // stride byte offset
  d |= (uint64_t)1 << 46;              // descriptor version for sm_100
  d |= (uint64_t)2 << 61;              // SWIZZLE_128B
  return d;
}

// ------------------------------------------------------------------ host

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 2-D tiled map: inner extent `inner` elements (contiguous), `outer` rows of
// `row_bytes`, box (box_inner, box_outer).
inline bool make_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                     uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                     CUtensorMapSwizzle sw, uint32_t outer_step = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_bytes};
  // with an outer traversal stride of s the box spans box_outer rows and
  // loads every s-th of them (box_outer / s rows)
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, outer_step};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (looked up once per device)
inline int num_sms() {
  static std::atomic<int> sms[64];
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return n;
  const int known = sms[dev].load(std::memory_order_relaxed);
  if (known) return known;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace tc
}  // namespace moe
