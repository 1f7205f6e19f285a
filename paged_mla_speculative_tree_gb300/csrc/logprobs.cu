// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits: the target's prediction that the acceptance walk follows ("The Glue
// That Connects" -- "What the Edit Actually Does") and what a server returns
// beside it.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "mla_step_ops.h"
#include "mtv_internal.cuh"

namespace mtv {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;

struct LogprobArgs {
  const void* logits;
  const float* inv_temperature;
  const int32_t* tokens;
  const int32_t* token_rows;
  float* logprobs;
  float* stats;
  int32_t* top_tokens;
  float* top_logprobs;
  uint32_t* err;
  int64_t num_rows, row_stride, num_tokens;
  int vocab, top_k;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

__device__ __forceinline__ void set_err(uint32_t* err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

// Larger for a larger logit and, among equal ones (-0 and 0 too), for a lower id.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t id) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (uint64_t((b >> 31) ? ~b : (b | 0x80000000u)) << 32) | uint32_t(~id);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t b = uint32_t(key >> 32);
  return __uint_as_float((b >> 31) ? (b & 0x7fffffffu) : ~b);
}

__device__ __forceinline__ bool usable_temperature(float s) { return s > 0.f && s < INFINITY; }

// One block a row: its maximum, then the sums relative to it, then one search
// a rank for the largest key below the previous one.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_rows_kernel(const LogprobArgs A) {
  __shared__ float fs[2][kLpWarps];
  __shared__ uint64_t ks[kLpWarps];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const T* x = static_cast<const T*>(A.logits) + r * A.row_stride;
  const float scale = A.inv_temperature ? A.inv_temperature[r] : 1.f;
  bool bad = !usable_temperature(scale);
  float m = -INFINITY;
  for (int i = tid; i < A.vocab; i += kLpThreads) {
    const float v = to_float(x[i]);
    bad |= !(v < INFINITY);
    m = fmaxf(m, v);
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) fs[0][w] = m;
  __syncthreads();
  for (int i = 0; i < kLpWarps; ++i) m = fmaxf(m, fs[0][i]);
  __syncthreads();
  // the reference of every exponent is this rounded product, so that one
  // fused multiply-add gives z - zmax to half a step of the difference
  float zmax = m * scale;
  bad |= m > -INFINITY && !(fabsf(zmax) < INFINITY);
  float s = 0.f, u = 0.f;
  if (!bad && m > -INFINITY) {
    for (int i = tid; i < A.vocab; i += kLpThreads) {
      const float d = fmaf(to_float(x[i]), scale, -zmax);
      const float e = expf(d);
      s += e;
      if (e > 0.f) u += e * d;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    u += __shfl_xor_sync(0xffffffffu, u, o);
  }
  if (lane == 0) {
    fs[0][w] = s;
    fs[1][w] = u;
  }
  __syncthreads();
  s = u = 0.f;
  for (int i = 0; i < kLpWarps; ++i) {
    s += fs[0][i];
    u += fs[1][i];
  }
  float log_s, entropy;
  if (bad) log_s = entropy = zmax = NAN;
  else if (m == -INFINITY) {
    log_s = -INFINITY;
    entropy = 0.f;
  } else {
    log_s = logf(s);
    entropy = log_s - u / s;
  }
  if (tid == 0) {
    A.stats[r] = zmax;
    A.stats[A.num_rows + r] = log_s;
    A.stats[2 * A.num_rows + r] = entropy;
    if (bad) set_err(A.err, MTV_DEVERR_LOGITS);
  }
  uint64_t below = ~uint64_t(0);
  for (int k = 0; k < A.top_k; ++k) {
    uint64_t best = 0;
    if (!bad) {
      for (int i = tid; i < A.vocab; i += kLpThreads) {
        const uint64_t key = order_key(to_float(x[i]), uint32_t(i));
        if (key < below && key > best) best = key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    __syncthreads();
    if (lane == 0) ks[w] = best;
    __syncthreads();
    for (int i = 0; i < kLpWarps; ++i) best = ks[i] > best ? ks[i] : best;
    below = best;
    if (tid == 0) {
      const bool none = bad || best == 0 || key_logit(best) == -INFINITY;
      A.top_tokens[k * A.num_rows + r] = none ? -1 : int32_t(~uint32_t(best));
      A.top_logprobs[k * A.num_rows + r] = bad ? NAN : none ? -INFINITY : fmaf(key_logit(best), scale, -zmax) - log_s;
    }
  }
}

// The given tokens, from the stats of their rows.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_tokens_kernel(const LogprobArgs A) {
  const int64_t i = int64_t(blockIdx.x) * kLpThreads + threadIdx.x;
  if (i >= A.num_tokens) return;
  const int64_t r = A.token_rows ? int64_t(A.token_rows[i]) : i;
  const int tok = A.tokens[i];
  float lp = NAN;
  if (r < 0 || r >= A.num_rows || tok < -1 || tok >= A.vocab) {
    set_err(A.err, MTV_DEVERR_TOKEN);
  } else if (tok < 0) {
    lp = 0.f;
  } else {
    const float scale = A.inv_temperature ? A.inv_temperature[r] : 1.f;
    const float x = to_float(static_cast<const T*>(A.logits)[r * A.row_stride + tok]);
    const float log_s = A.stats[A.num_rows + r];
    lp = x == -INFINITY && !isnan(log_s) ? -INFINITY : fmaf(x, scale, -A.stats[r]) - log_s;
  }
  A.logprobs[i] = lp;
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs& A, cudaStream_t st) {
  if (A.num_rows > 0) {
    logprob_rows_kernel<T><<<unsigned(A.num_rows), kLpThreads, 0, st>>>(A);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (A.num_tokens > 0)
    logprob_tokens_kernel<T><<<unsigned((A.num_tokens + kLpThreads - 1) / kLpThreads), kLpThreads, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mtv

extern "C" int mla_token_logprobs(const void* logits, int dtype, int64_t num_rows, int vocab, int64_t row_stride,
                                  const float* inv_temperature, const int32_t* tokens, const int32_t* token_rows,
                                  int64_t num_tokens, float* logprobs, float* stats, int top_k,
                                  int32_t* top_tokens, float* top_logprobs, uint32_t* err, void* stream) {
  using namespace mtv;
  if (num_rows < 0 || num_tokens < 0 || row_stride < 0 || vocab < 1 || vocab > MTV_MAX_VOCAB || top_k < 0 ||
      top_k > MTV_MAX_TOP || dtype < MTV_DTYPE_BF16 || dtype > MTV_DTYPE_FP32 ||
      (!token_rows && num_tokens > num_rows))
    return MTV_E_BAD_ARGUMENT;
  if (num_rows > INT32_MAX || num_tokens > INT32_MAX) return MTV_E_UNSUPPORTED;
  if (num_rows == 0 && num_tokens == 0) return MTV_OK;
  if ((num_rows > 0 && (!logits || !stats)) || (num_tokens > 0 && (!tokens || !logprobs)) ||
      (top_k > 0 && num_rows > 0 && (!top_tokens || !top_logprobs)))
    return MTV_E_NULL_POINTER;
  const LogprobArgs A{logits, inv_temperature, tokens, token_rows, logprobs, stats, top_tokens, top_logprobs,
                      err,    num_rows,        row_stride, num_tokens, vocab,  top_k};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MTV_DTYPE_BF16) e = launch_logprobs<__nv_bfloat16>(A, st);
  else if (dtype == MTV_DTYPE_FP16) e = launch_logprobs<__half>(A, st);
  else e = launch_logprobs<float>(A, st);
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
