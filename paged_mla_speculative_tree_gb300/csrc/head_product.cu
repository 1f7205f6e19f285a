// One matrix product a head: the absorption of queries into the latent space,
// the values of latent outputs and the expansion of latents to every head's
// keys and values (the latent form: "The Glue That Binds" -- "The Broader
// Engineering Effort").
#include <stdint.h>

#include "mla_layer_ops.h"
#include "mtv_internal.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

struct ProductArgs {
  const void* x;
  const void* w;
  void* out;
  int64_t x_tok, x_head, w_head, w_k, w_n, out_tok, out_head, tokens;
  int heads, k_dim, n_dim;
};

// The plain form, for any strides: a block a tile of 64 tokens x 64 outputs of
// one head, 16 k at a time through shared memory, 4 x 4 sums a thread.
constexpr int kTile = 64, kStep = 16;

template <typename T>
__global__ void __launch_bounds__(256) head_product_plain_kernel(const ProductArgs A) {
  __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
  const int h = blockIdx.y, n0 = blockIdx.z * kTile, tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kTile;
  const T* x = static_cast<const T*>(A.x) + int64_t(h) * A.x_head;
  const T* w = static_cast<const T*>(A.w) + int64_t(h) * A.w_head;
  const int tx = tid % 16, ty = tid / 16;
  float sum[4][4] = {};
  for (int k0 = 0; k0 < A.k_dim; k0 += kStep) {
    for (int i = tid; i < kStep * kTile; i += 256) {
      const int k = i % kStep, t = i / kStep;
      xs[k][t] = (k0 + k < A.k_dim && t0 + t < A.tokens) ? to_float(x[(t0 + t) * A.x_tok + k0 + k]) : 0.f;
    }
    for (int i = tid; i < kStep * kTile; i += 256) {
      const int n = i % kTile, k = i / kTile;
      ws[k][n] = (k0 + k < A.k_dim && n0 + n < A.n_dim) ? to_float(w[(k0 + k) * A.w_k + (n0 + n) * A.w_n]) : 0.f;
    }
    __syncthreads();
    // values of k past the end are zero on both sides
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], sum[i][j]);
    __syncthreads();
  }
  T* out = static_cast<T*>(A.out) + int64_t(h) * A.out_head;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty + 16 * i;
      const int n = n0 + tx + 16 * j;
      if (t < A.tokens && n < A.n_dim) out[t * A.out_tok + n] = from_float<T>(sum[i][j]);
    }
}

template <typename T> cudaError_t launch_plain(const ProductArgs& A, cudaStream_t st) {
  const dim3 grid(unsigned((A.tokens + kTile - 1) / kTile), unsigned(A.heads), unsigned((A.n_dim + kTile - 1) / kTile));
  head_product_plain_kernel<T><<<grid, 256, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mtv

extern "C" int mla_head_product(const void* x, int64_t x_tok_stride, int64_t x_head_stride, const void* w,
                                int64_t w_head_stride, int64_t w_k_stride, int64_t w_n_stride, void* out,
                                int64_t out_tok_stride, int64_t out_head_stride, int64_t num_tokens, int num_heads,
                                int k_dim, int n_dim, int dtype, void* stream) {
  using namespace mtv;
  if (num_tokens < 0 || num_tokens > INT32_MAX || num_heads < 0 || num_heads > MTV_MAX_HEADS || k_dim < 1 ||
      k_dim > MTV_MAX_HEAD_DIM || n_dim < 1 || n_dim > MTV_MAX_HEAD_DIM ||
      (dtype != MTV_DTYPE_BF16 && dtype != MTV_DTYPE_FP16))
    return MTV_E_BAD_ARGUMENT;
  if (num_tokens == 0 || num_heads == 0) return MTV_OK;
  if (!x || !w || !out) return MTV_E_NULL_POINTER;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(out)) & 1)
    return MTV_E_BAD_ARGUMENT;
  const ProductArgs A{x,          w,          out,        x_tok_stride,   x_head_stride,   w_head_stride,
                      w_k_stride, w_n_stride, out_tok_stride, out_head_stride, num_tokens, num_heads, k_dim, n_dim};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MTV_DTYPE_BF16 ? launch_plain<__nv_bfloat16>(A, st) : launch_plain<__half>(A, st);
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
