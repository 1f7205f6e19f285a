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
};

// False when the wait gave up or another one of the block has.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ctl->abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      ctl->abort = 1;
      if (err) atomicOr(err, MTV_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  return ptx::mbar_try_wait(bar, parity) || wait_slow(bar, parity, ctl, err);
}
// The same with the slow way as a call: less code, but a call's convention costs a
// kernel without registers to spare its spills (prefill.cu).
static __device__ __noinline__ bool wait_slow_call(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  return wait_slow(bar, parity, ctl, err);
}
__device__ __forceinline__ bool wait_for_call(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  return ptx::mbar_try_wait(bar, parity) || wait_slow_call(bar, parity, ctl, err);
}
// For a barrier that the other CTA of a cluster arrives on.
static __device__ __noinline__ bool wait_for_peer(uint32_t bar, uint32_t parity, Ctl* ctl, uint32_t* err) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait_cluster(bar, parity)) {
    if (ctl->abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      ctl->abort = 1;
      if (err) atomicOr(err, MTV_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// For what has to land before the block may end: ignores the flag.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, uint32_t* err) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitCycles) {
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
