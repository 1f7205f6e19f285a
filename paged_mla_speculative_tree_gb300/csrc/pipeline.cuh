// Bounded waits of a block's pipeline roles, and descriptor arithmetic.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla_tree_verify.h"
#include "tc_ptx.cuh"

namespace mtv {

constexpr long long kWaitCycles = 1ll << 31;  // about a second

struct Ctl {
  uint32_t tmem;
  volatile int abort;  // set by a wait that gave up
  uint32_t peer;       // of a pair of CTAs, the other one's abort flag (address from mapa); else 0
  int asked[4];        // of a pair: see head_product.cu
  long long deadline;  // of the waits' test form
};

// By one thread, before the block's first wait.  kTest: from 512 (give_up - 1) cycles
// on, every wait that has to spin gives up.
template <bool kTest> __device__ __forceinline__ void init_ctl(Ctl* ctl, int give_up, uint32_t peer = 0) {
  ctl->abort = 0;
  ctl->peer = peer;
  if constexpr (kTest) ctl->deadline = clock64() + 512ll * (give_up - 1);
}

// Ends the block's other waits, and those of a pair's other CTA.
__device__ __forceinline__ void give_up_waits(Ctl* ctl, uint32_t* err) {
  ctl->abort = 1;
  if (ctl->peer) ptx::st_cluster_u32(ctl->peer, 1);
  if (err) atomicOr(err, MTV_DEVERR_TIMEOUT);
}
// False when the wait gave up or another one of the block has.  kTest: the forms of
// waits for tests, with a deadline and a first look that does not suspend the thread
// (deciding it as the kernel runs took 3 % of long prompts).
template <bool kTest> __device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  const long long t0 = clock64();
  while (kTest ? !ptx::mbar_test_wait(bar, parity) : !ptx::mbar_try_wait(bar, parity)) {
    if (ctl->abort) return false;
    if (clock64() - t0 > kWaitCycles || (kTest && clock64() >= ctl->deadline)) {
      give_up_waits(ctl, err);
      return false;
    }
  }
  return true;
}
template <bool kTest> __device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  if constexpr (!kTest)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow<kTest>(bar, parity, ctl, err);
}
// The same with the slow way as a call: less code, but a call's convention costs a
// kernel without registers to spare its spills (prefill.cu).
template <bool kTest> static __device__ __noinline__ bool wait_slow_call(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  return wait_slow<kTest>(bar, parity, ctl, err);
}
template <bool kTest> __device__ __forceinline__ bool wait_for_call(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  if constexpr (!kTest)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow_call<kTest>(bar, parity, ctl, err);
}
// For a barrier that the other CTA of a cluster arrives on.
template <bool kTest> static __device__ __noinline__ bool wait_for_peer(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait_cluster(bar, parity)) {
    if (ctl->abort) return false;
    if (clock64() - t0 > kWaitCycles || (kTest && clock64() >= ctl->deadline)) {
      give_up_waits(ctl, err);
      return false;
    }
  }
  return true;
}
// For what has to land before the block may end: ignores the flag and the deadline.
// Waits one after another share their limit, counted from `since`.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, long long since, uint32_t* err) {
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - since > kWaitCycles) {
      if (err) atomicOr(err, MTV_DEVERR_TIMEOUT);
      return;
    }
}

// A shared-memory descriptor moved by `off` bytes: shared-memory addresses stay
// below 2^18, so the sum never carries out of the address field.
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t off) {
  return (d & 0xFFFFFFFF00000000ull) | uint64_t(uint32_t(d) + (off >> 4));
}

}  // namespace mtv
