// Root-mean-square norms of the latent part and of query heads, the rotary
// positions of both, and the write of the latent rows into the paged pool, in
// one pass over a token's projections.
#include <math.h>
#include <stdint.h>

#include "mla_layer_ops.h"
#include "mtv_internal.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

struct NormArgs {
  const uint64_t* turns;
  const int64_t* positions;
  const int64_t* num_valid;
  const void* q_in;
  const void* q_weight;
  void* q_nope;
  void* q_rope;
  const void* c_in;
  const void* c_weight;
  const void* k_in;
  const int64_t* out_cache_loc;
  __nv_bfloat16* pool;
  uint32_t* err;
  int64_t q_tok, q_head, nope_tok, nope_head, rope_tok, rope_head, c_tok, k_tok, num_slots;
  float amplitude, eps;
  int rope_dim, nope_dim, num_heads;
};

constexpr int kPlainThreads = 256;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of the token's angles, times the amplitude (the angle of pair i
// is position * turns[i] modulo one turn, as in rope.cu).
__device__ __forceinline__ void angles(const NormArgs& A, int64_t t, int tid, int threads, float* cos_s, float* sin_s) {
  const uint64_t pos = uint64_t(A.positions[t]);
  for (int i = tid; i < A.rope_dim / 2; i += threads) {
    float s, c;
    sincospif(float(int32_t((pos * A.turns[i]) >> 32)) * 0x1p-31f, &s, &c);
    cos_s[i] = c * A.amplitude;
    sin_s[i] = s * A.amplitude;
  }
}

// The plain form, for any strides and sizes: a block a token, a warp a head,
// the latent row by the first warp.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kPlainThreads) norm_rope_plain_kernel(const NormArgs A) {
  __shared__ float cos_s[MTV_MAX_ROPE_DIM / 2], sin_s[MTV_MAX_ROPE_DIM / 2];
  const int64_t t = blockIdx.x;
  if (A.num_valid && t >= *A.num_valid) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = A.rope_dim / 2;
  angles(A, t, tid, kPlainThreads, cos_s, sin_s);
  __syncthreads();
  const int second = kHalf ? pairs : 1;
  if (A.q_in) {
    const int dim = A.nope_dim + A.rope_dim;
    const T* weight = static_cast<const T*>(A.q_weight);
    for (int h = warp; h < A.num_heads; h += kPlainThreads / 32) {
      const T* x = static_cast<const T*>(A.q_in) + t * A.q_tok + h * A.q_head;
      T* nope = static_cast<T*>(A.q_nope) + t * A.nope_tok + h * A.nope_head;
      T* rope = static_cast<T*>(A.q_rope) + t * A.rope_tok + h * A.rope_head;
      float r = 1.f;
      if (weight) {
        float sum = 0.f;
        for (int d = lane; d < dim; d += 32) sum = fmaf(to_float(x[d]), to_float(x[d]), sum);
        r = rsqrtf(warp_sum(sum) / float(dim) + A.eps);
        for (int d = lane; d < A.nope_dim; d += 32) nope[d] = from_float<T>(to_float(x[d]) * r * to_float(weight[d]));
      }
      x += A.nope_dim;
      for (int i = lane; i < pairs; i += 32) {
        const int d = kHalf ? i : 2 * i, e = d + second;
        float x1 = to_float(x[d]), x2 = to_float(x[e]);
        if (weight) {
          x1 *= r * to_float(weight[A.nope_dim + d]);
          x2 *= r * to_float(weight[A.nope_dim + e]);
        }
        rope[d] = from_float<T>(x1 * cos_s[i] - x2 * sin_s[i]);
        rope[e] = from_float<T>(x1 * sin_s[i] + x2 * cos_s[i]);
      }
    }
  }
  if (!A.pool || warp != 0) return;
  const int64_t slot = A.out_cache_loc[t];
  if (slot < 0 || slot >= A.num_slots) {
    if (lane == 0 && A.err) atomicOr(A.err, MTV_DEVERR_SLOT_RANGE);
    return;
  }
  __nv_bfloat16* row = A.pool + slot * kDQK;
  const T* c = static_cast<const T*>(A.c_in) + t * A.c_tok;
  const T* weight = static_cast<const T*>(A.c_weight);
  float r = 1.f;
  if (weight) {
    float sum = 0.f;
    for (int d = lane; d < kDLat; d += 32) sum = fmaf(to_float(c[d]), to_float(c[d]), sum);
    r = rsqrtf(warp_sum(sum) / float(kDLat) + A.eps);
  }
  for (int d = lane; d < kDLat; d += 32)
    row[d] = __float2bfloat16_rn(weight ? to_float(c[d]) * r * to_float(weight[d]) : to_float(c[d]));
  const T* k = static_cast<const T*>(A.k_in) + t * A.k_tok;
  for (int i = lane; i < pairs; i += 32) {
    const int d = kHalf ? i : 2 * i, e = d + second;
    const float x1 = to_float(k[d]), x2 = to_float(k[e]);
    row[kDLat + d] = __float2bfloat16_rn(x1 * cos_s[i] - x2 * sin_s[i]);
    row[kDLat + e] = __float2bfloat16_rn(x1 * sin_s[i] + x2 * cos_s[i]);
  }
}

template <typename T> cudaError_t launch_norm(const NormArgs& A, int layout, int64_t tokens, cudaStream_t st) {
  auto kernel = layout == MTV_ROPE_HALF ? norm_rope_plain_kernel<T, true> : norm_rope_plain_kernel<T, false>;
  kernel<<<unsigned(tokens), kPlainThreads, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mtv

extern "C" int mla_norm_rope_write(const uint64_t* turns, int rope_dim, float amplitude, int layout,
                                   const int64_t* positions, int64_t num_tokens, const int64_t* num_valid, int dtype,
                                   float eps, const void* q_in, int64_t q_tok_stride, int64_t q_head_stride,
                                   int num_heads, int nope_dim, const void* q_weight, void* q_nope,
                                   int64_t q_nope_tok_stride, int64_t q_nope_head_stride, void* q_rope,
                                   int64_t q_rope_tok_stride, int64_t q_rope_head_stride, const void* c_in,
                                   int64_t c_tok_stride, const void* c_weight, const void* k_in,
                                   int64_t k_tok_stride, const int64_t* out_cache_loc, void* kv_pool,
                                   int64_t num_slots, uint32_t* err, void* stream) {
  using namespace mtv;
  if (rope_dim < 2 || rope_dim > MTV_MAX_ROPE_DIM || (rope_dim & 1) || !isfinite(amplitude) ||
      (layout != MTV_ROPE_INTERLEAVED && layout != MTV_ROPE_HALF) || !isfinite(eps) || eps < 0 || num_tokens < 0 ||
      num_heads < 0 || num_slots < 0 || nope_dim < 0 || nope_dim > MTV_MAX_NORM_DIM - rope_dim ||
      dtype < MTV_DTYPE_BF16 || dtype > MTV_DTYPE_FP32)
    return MTV_E_BAD_ARGUMENT;
  if (num_tokens > INT32_MAX) return MTV_E_UNSUPPORTED;
  if ((q_in == nullptr) != (q_rope == nullptr)) return MTV_E_NULL_POINTER;
  if (q_in ? (q_nope != nullptr) != (q_weight != nullptr && nope_dim > 0) : (q_nope || q_weight))
    return MTV_E_BAD_ARGUMENT;
  if (kv_pool) {
    if (rope_dim != kDRope) return MTV_E_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(kv_pool) & 15) return MTV_E_BAD_ARGUMENT;
  }
  if (num_tokens == 0 || (!kv_pool && (!q_in || num_heads == 0))) return MTV_OK;
  if (!turns || !positions || (kv_pool && (!k_in || !c_in || !out_cache_loc))) return MTV_E_NULL_POINTER;
  const uintptr_t size = dtype == MTV_DTYPE_FP32 ? 4 : 2;
  uintptr_t bits = 0;
  for (const void* p : {q_in, q_weight, static_cast<const void*>(q_nope), static_cast<const void*>(q_rope), c_in,
                        c_weight, k_in})
    bits |= reinterpret_cast<uintptr_t>(p);
  if (bits & (size - 1)) return MTV_E_BAD_ARGUMENT;
  const NormArgs A{turns, positions, num_valid, q_in, q_weight, q_nope, q_rope, c_in, c_weight, k_in, out_cache_loc,
                   static_cast<__nv_bfloat16*>(kv_pool), err, q_tok_stride, q_head_stride, q_nope_tok_stride,
                   q_nope_head_stride, q_rope_tok_stride, q_rope_head_stride, c_tok_stride, k_tok_stride, num_slots,
                   amplitude, eps, rope_dim, nope_dim, num_heads};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MTV_DTYPE_BF16) e = launch_norm<__nv_bfloat16>(A, layout, num_tokens, st);
  else if (dtype == MTV_DTYPE_FP16) e = launch_norm<__half>(A, layout, num_tokens, st);
  else e = launch_norm<float>(A, layout, num_tokens, st);
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
