// Causal attention of new tokens over keys and values expanded from latents
// (head parts of 128 + 64 and 128): the form for prompts, where every query
// row has many neighbours.
#include <math.h>
#include <stdint.h>

#include "mla_layer_ops.h"
#include "mtv_internal.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

constexpr int kNope = 128, kRope = 64, kQK = kNope + kRope, kV = 128;

struct PrefillArgs {
  const void* q;
  const void* k_nope;
  const void* k_rope;
  const void* v;
  void* out;
  float* lse;
  const int64_t* qo_indptr;
  const int32_t* kv_indptr;
  uint32_t* err;
  int64_t q_tok, q_head, k_tok, k_head, kr_tok, v_tok, v_head, o_tok, o_head, num_q, num_kv, max_q, max_kv;
  float scale;
  int bs, heads, causal;
};

struct PrefillReq {
  int64_t q0, k0, n, len;
};

// The request's rows, checked against the buffers and the bounds; n = 0 where
// they do not hold.
__device__ __forceinline__ PrefillReq load_prefill_req(const PrefillArgs& A, int r, bool report) {
  const int64_t q0 = A.qo_indptr[r], q1 = A.qo_indptr[r + 1], k0 = A.kv_indptr[r], k1 = A.kv_indptr[r + 1];
  PrefillReq R{q0, k0, q1 - q0, k1 - k0};
  if (q0 < 0 || q1 < q0 || q1 > A.num_q || k0 < 0 || k1 < k0 || k1 > A.num_kv || R.n > A.max_q || R.len > A.max_kv) {
    if (report && A.err) atomicOr(A.err, MTV_DEVERR_INDPTR);
    R.n = 0;
  }
  return R;
}

// A warp a query row of one head, a key at a time.
template <typename T>
__global__ void __launch_bounds__(128) prefill_plain_kernel(const PrefillArgs A) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y, r = blockIdx.z;
  const PrefillReq R = load_prefill_req(A, r, threadIdx.x == 0);
  const int64_t i = int64_t(blockIdx.x) * 4 + warp;
  if (i >= R.n) return;
  const T* q = static_cast<const T*>(A.q) + (R.q0 + i) * A.q_tok + h * A.q_head;
  float x[6], acc[4] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int u = 0; u < 6; ++u) x[u] = to_float(q[lane + 32 * u]) * A.scale;
  const int64_t end = A.causal ? min(R.len, R.len - R.n + i + 1) : R.len;
  for (int64_t j = 0; j < end; ++j) {
    const T* kn = static_cast<const T*>(A.k_nope) + (R.k0 + j) * A.k_tok + h * A.k_head;
    const T* kr = static_cast<const T*>(A.k_rope) + (R.k0 + j) * A.kr_tok;
    const T* v = static_cast<const T*>(A.v) + (R.k0 + j) * A.v_tok + h * A.v_head;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) s = fmaf(x[u], to_float(kn[lane + 32 * u]), s);
#pragma unroll
    for (int u = 0; u < 2; ++u) s = fmaf(x[4 + u], to_float(kr[lane + 32 * u]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    l = l * keep + p;
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[u] = acc[u] * keep + p * to_float(v[lane + 32 * u]);
    m = top;
  }
  T* out = static_cast<T*>(A.out) + (R.q0 + i) * A.o_tok + h * A.o_head;
#pragma unroll
  for (int u = 0; u < 4; ++u) out[lane + 32 * u] = from_float<T>(end > 0 ? acc[u] / l : 0.f);
  if (A.lse && lane == 0) A.lse[(R.q0 + i) * A.heads + h] = end > 0 ? m + logf(l) : -INFINITY;
}

template <typename T> cudaError_t launch_prefill(const PrefillArgs& A, cudaStream_t st) {
  const dim3 grid(unsigned((A.max_q + 3) / 4), unsigned(A.heads), unsigned(A.bs));
  prefill_plain_kernel<T><<<grid, 128, 0, st>>>(A);
  return cudaGetLastError();
}

uint64_t workspace_bytes_of(int nsplit, int64_t num_q, int heads) {
  return nsplit > 1 ? uint64_t(nsplit) * uint64_t(num_q) * uint64_t(heads) * uint64_t(kV + 1) * 4u : 0u;
}

}  // namespace
}  // namespace mtv

extern "C" int mla_prefill_workspace(int num_sms, int bs, int64_t max_q, int64_t max_kv, int64_t num_q, int num_heads,
                                     int* nsplit_out, uint64_t* bytes_out) {
  using namespace mtv;
  if (!nsplit_out || !bytes_out) return MTV_E_NULL_POINTER;
  if (num_sms < 1 || bs < 0 || bs > MTV_MAX_HEADS || max_q < 0 || max_kv < 0 || num_q < 0 || num_q > INT32_MAX ||
      max_q > INT32_MAX || max_kv > INT32_MAX || num_heads < 0 || num_heads > MTV_MAX_HEADS)
    return MTV_E_BAD_ARGUMENT;
  *nsplit_out = 1;
  *bytes_out = workspace_bytes_of(*nsplit_out, num_q, num_heads);
  return MTV_OK;
}

extern "C" int mla_prefill_run(const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k_nope,
                               int64_t k_tok_stride, int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
                               const void* v, int64_t v_tok_stride, int64_t v_head_stride, const int64_t* qo_indptr,
                               const int32_t* kv_indptr, int bs, int64_t max_q, int64_t max_kv, int64_t num_q,
                               int64_t num_kv, int num_heads, int dtype, float scale, int causal, void* out,
                               int64_t out_tok_stride, int64_t out_head_stride, float* lse, int nsplit,
                               void* workspace, uint64_t workspace_bytes, uint32_t* err, void* stream) {
  using namespace mtv;
  if (bs < 0 || bs > MTV_MAX_HEADS || max_q < 0 || max_kv < 0 || max_q > INT32_MAX || max_kv > INT32_MAX ||
      num_q < 0 || num_kv < 0 || num_q > INT32_MAX || num_kv > INT32_MAX || num_heads < 0 ||
      num_heads > MTV_MAX_HEADS || (dtype != MTV_DTYPE_BF16 && dtype != MTV_DTYPE_FP16) || !isfinite(scale) ||
      !(scale > 0) || (causal != 0 && causal != 1) || nsplit < 1 || nsplit > MTV_MAX_PREFILL_SPLITS)
    return MTV_E_BAD_ARGUMENT;
  if (nsplit > 1) {
    if (!workspace) return MTV_E_NULL_POINTER;
    if (workspace_bytes < workspace_bytes_of(nsplit, num_q, num_heads)) return MTV_E_WORKSPACE_SMALL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return MTV_E_WORKSPACE_ALIGN;
  }
  if (bs == 0 || max_q == 0 || num_q == 0 || num_heads == 0) return MTV_OK;
  if (!q || !out || !qo_indptr || !kv_indptr || (num_kv > 0 && (!k_nope || !k_rope || !v))) return MTV_E_NULL_POINTER;
  uintptr_t bits = 0;
  for (const void* p : {q, k_nope, k_rope, v, static_cast<const void*>(out)}) bits |= reinterpret_cast<uintptr_t>(p);
  for (int64_t s : {q_tok_stride, q_head_stride, k_tok_stride, k_head_stride, k_rope_stride, v_tok_stride,
                    v_head_stride, out_tok_stride, out_head_stride})
    bits |= uintptr_t(s) * 2;
  if (bits & 15) return MTV_E_BAD_ARGUMENT;
  const PrefillArgs A{q, k_nope, k_rope, v, out, lse, qo_indptr, kv_indptr, err, q_tok_stride, q_head_stride,
                      k_tok_stride, k_head_stride, k_rope_stride, v_tok_stride, v_head_stride, out_tok_stride,
                      out_head_stride, num_q, num_kv, max_q, max_kv, scale, bs, num_heads, causal};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MTV_DTYPE_BF16 ? launch_prefill<__nv_bfloat16>(A, st) : launch_prefill<__half>(A, st);
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
