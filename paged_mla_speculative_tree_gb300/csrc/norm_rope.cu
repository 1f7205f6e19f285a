// Root-mean-square norms of the latent part and of query heads, the rotary
// positions of both, and the write of the latent rows into the paged pool, in
// one pass over a token's projections.
#include <math.h>
#include <stdint.h>

#include "mla_layer_ops.h"
#include "launch.cuh"
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

// The vector form: a block a token, eight lanes a head, in 16-byte units: of the
// plain part every eighth unit a lane, of the rotated part every eighth unit or,
// in the half layout, every eighth pair of units half a part apart, so that a
// head is read once, its sum of squares takes three shuffles, and a lane turns
// what it holds.  One more warp has the latent row.  Every load of the first 32
// heads is issued before the angles are computed and before the token is known
// to be valid.  Its conditions (whole units everywhere, at most NN and NR units
// a lane) are checked by the launch; the plain form above takes what is left.
//
// What bounds it (one GB300, 64 heads of 128 + 64): for many tokens the bytes of the
// heads, read and written once (8,191 tokens in fp16 77 us, 5.5 TB/s; the plain form
// 257); for few the launch (8 tokens 2.1 us).  Four blocks an SM in 56 registers
// (three in 72: 84 us; 16 heads a block, six an SM: 76, but 1,024 tokens 9.3 us in
// place of 8.0); streaming loads and stores were slower.
constexpr int kVecThreads = 288, kGroups = 32;

template <int N> __device__ __forceinline__ void load_floats(const float* from, float* to) {
  static_assert(N % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < N; i += N % 4 ? 2 : 4) {
    if constexpr (N % 4 == 0) {
      const float4 v = *reinterpret_cast<const float4*>(from + i);
      to[i] = v.x, to[i + 1] = v.y, to[i + 2] = v.z, to[i + 3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(from + i);
      to[i] = v.x, to[i + 1] = v.y;
    }
  }
}

// 2 V values of a rotated part, turned: two units half a part apart (half
// layout), or one and nothing.
template <int V, bool kHalf>
__device__ __forceinline__ void turn_unit(float* x, int unit, const float* cos_s, const float* sin_s) {
  constexpr int P = kHalf ? V : V / 2;
  float c[P], s[P];
  load_floats<P>(cos_s + unit * P, c);
  load_floats<P>(sin_s + unit * P, s);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int j = kHalf ? i : 2 * i, k = kHalf ? i + V : 2 * i + 1;
    const float x1 = x[j], x2 = x[k];
    x[j] = x1 * c[i] - x2 * s[i];
    x[k] = x1 * s[i] + x2 * c[i];
  }
}

__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }

// NN, NR: units of the plain part and units (half layout: pairs of them) of the
// rotated part that a lane may hold.
template <typename T, bool kHalf, int NN, int NR>
__global__ void __launch_bounds__(kVecThreads, NN <= 2 ? (sizeof(T) == 4 ? 3 : 4) : 1) norm_rope_vec_kernel(const NormArgs A) {
  constexpr int V = 16 / int(sizeof(T)), M = kHalf ? 2 : 1;
  constexpr int kLatentUnits = kDLat / V / 32;
  __shared__ __align__(16) float cos_s[MTV_MAX_ROPE_DIM / 2], sin_s[MTV_MAX_ROPE_DIM / 2];
  launched_after();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, l = tid & 7, group = tid >> 3;
  const bool queries = A.q_in && tid < kGroups * 8, latents = A.pool && tid >= kGroups * 8;
  const int turned = A.rope_dim / V / M, apart = A.rope_dim / 2;  // units or pairs of a rotated part
  const int plain = A.q_weight ? A.nope_dim / V : 0;              // units of the plain part, where it is read

  const T* q = static_cast<const T*>(A.q_in) + t * A.q_tok;
  const T* weight = static_cast<const T*>(A.q_weight);
  uint4 xn[NN > 0 ? NN : 1], xr[NR][M];
  auto load_head = [&](const T* head) {
#pragma unroll
    for (int i = 0; i < NN; ++i)
      if (l + 8 * i < plain) xn[i] = load16(head + (l + 8 * i) * V);
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (l + 8 * i < turned) xr[i][m] = load16(head + A.nope_dim + (l + 8 * i) * V + m * apart);
  };
  uint4 c[kLatentUnits], cw[kLatentUnits], k[M];
  int64_t slot = -1;
  if (queries) {
    if (group < A.num_heads) load_head(q + group * A.q_head);
  } else if (latents) {
    slot = A.out_cache_loc[t];
#pragma unroll
    for (int i = 0; i < kLatentUnits; ++i) {
      c[i] = load16(static_cast<const T*>(A.c_in) + t * A.c_tok + (lane + 32 * i) * V);
      if (A.c_weight) cw[i] = load16(static_cast<const T*>(A.c_weight) + (lane + 32 * i) * V);
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (lane < turned) k[m] = load16(static_cast<const T*>(A.k_in) + t * A.k_tok + lane * V + m * apart);
  }
  const int64_t valid = A.num_valid ? *A.num_valid : INT64_MAX;
  angles(A, t, tid, kVecThreads, cos_s, sin_s);
  __syncthreads();
  if (t >= valid) return;

  if (queries) {
    for (int h = group; h - group < A.num_heads; h += kGroups) {  // whole warps stay together
      const bool mine = h < A.num_heads;
      if (h != group && mine) load_head(q + h * A.q_head);
      float r = 1.f;
      if (weight) {
        float sum = 0.f;
        auto add = [&](const uint4& u) {
          float f[V];
          expand<T>(u, f);
#pragma unroll
          for (int d = 0; d < V; ++d) sum = fmaf(f[d], f[d], sum);
        };
#pragma unroll
        for (int i = 0; i < NN; ++i)
          if (mine && l + 8 * i < plain) add(xn[i]);
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int m = 0; m < M; ++m)
            if (mine && l + 8 * i < turned) add(xr[i][m]);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        r = rsqrtf(sum / float(A.nope_dim + A.rope_dim) + A.eps);
      }
      if (!mine) continue;
      // a lane writes what it has read, so outputs may be the inputs
      auto scale = [&](float* f, int at) {  // the weights are in L1 from the blocks before
        float g[V];
        expand<T>(load16(weight + at), g);
#pragma unroll
        for (int d = 0; d < V; ++d) f[d] = f[d] * r * g[d];
      };
      T* nope = static_cast<T*>(A.q_nope) + t * A.nope_tok + h * A.nope_head;
      T* rope = static_cast<T*>(A.q_rope) + t * A.rope_tok + h * A.rope_head;
#pragma unroll
      for (int i = 0; i < NN; ++i) {
        if (l + 8 * i >= plain) continue;
        float f[V];
        expand<T>(xn[i], f);
        scale(f, (l + 8 * i) * V);
        *reinterpret_cast<uint4*>(nope + (l + 8 * i) * V) = pack<T>(f);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (l + 8 * i >= turned) continue;
        float f[2 * V];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          expand<T>(xr[i][m], f + m * V);
          if (weight) scale(f + m * V, A.nope_dim + (l + 8 * i) * V + m * apart);
        }
        turn_unit<V, kHalf>(f, l + 8 * i, cos_s, sin_s);
#pragma unroll
        for (int m = 0; m < M; ++m) *reinterpret_cast<uint4*>(rope + (l + 8 * i) * V + m * apart) = pack<T>(f + m * V);
      }
    }
    return;
  }
  if (!latents) return;
  if (slot < 0 || slot >= A.num_slots) {
    if (lane == 0 && A.err) atomicOr(A.err, MTV_DEVERR_SLOT_RANGE);
    return;
  }
  __nv_bfloat16* row = A.pool + slot * kDQK;
  float r = 1.f;
  if (A.c_weight) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kLatentUnits; ++i) {
      float f[V];
      expand<T>(c[i], f);
#pragma unroll
      for (int d = 0; d < V; ++d) sum = fmaf(f[d], f[d], sum);
    }
    r = rsqrtf(warp_sum(sum) / float(kDLat) + A.eps);
  }
#pragma unroll
  for (int i = 0; i < kLatentUnits; ++i) {
    float f[V], g[V];
    expand<T>(c[i], f);
    if (A.c_weight) {
      expand<T>(cw[i], g);
#pragma unroll
      for (int d = 0; d < V; ++d) f[d] = f[d] * r * g[d];
    }
    store_bf16<V>(row + (lane + 32 * i) * V, f);
  }
  if (lane < turned) {
    float f[2 * V];
#pragma unroll
    for (int m = 0; m < M; ++m) expand<T>(k[m], f + m * V);
    turn_unit<V, kHalf>(f, lane, cos_s, sin_s);
#pragma unroll
    for (int m = 0; m < M; ++m) store_bf16<V>(row + kDLat + lane * V + m * apart, f + m * V);
  }
}

// Whether every address that the vector form touches is 16-byte aligned.
template <typename T> bool vector_form(const NormArgs& A) {
  constexpr int64_t v = 16 / int64_t(sizeof(T));
  uint64_t bits = 0;
  auto at = [&](const void* p) { bits |= reinterpret_cast<uintptr_t>(p); };
  auto stride = [&](int64_t s) { bits |= s % v != 0; };
  if (A.q_in) {
    at(A.q_in), at(A.q_weight), at(A.q_nope), at(A.q_rope);
    stride(A.q_tok), stride(A.q_head), stride(A.rope_tok), stride(A.rope_head);
    if (A.q_nope) stride(A.nope_tok), stride(A.nope_head);
    stride(A.nope_dim);
  }
  if (A.pool) at(A.c_in), at(A.c_weight), at(A.k_in), stride(A.c_tok), stride(A.k_tok);
  return (bits & 15) == 0 && A.rope_dim % (2 * v) == 0 && A.num_heads <= INT32_MAX / 2;
}

template <typename T, bool kHalf> cudaError_t launch_norm_layout(const NormArgs& A, int64_t tokens, cudaStream_t st) {
  constexpr int v = 16 / int(sizeof(T));
  const unsigned grid = unsigned(tokens);
  const int plain = A.q_weight ? (A.nope_dim / v + 7) / 8 : 0, turned = (A.rope_dim / v / (kHalf ? 2 : 1) + 7) / 8;
  if (!vector_form<T>(A) || plain > 8 || turned > 2) {
    norm_rope_plain_kernel<T, kHalf><<<grid, kPlainThreads, 0, st>>>(A);
    return cudaGetLastError();
  }
  auto kernel = plain == 0                  ? norm_rope_vec_kernel<T, kHalf, 0, 2>
                : plain <= 2 && turned == 1 ? norm_rope_vec_kernel<T, kHalf, 2, 1>
                : plain <= 4                ? norm_rope_vec_kernel<T, kHalf, 4, 2>
                                            : norm_rope_vec_kernel<T, kHalf, 8, 2>;
  return launch_early(kernel, dim3(grid), kVecThreads, 0, st, A);
}

template <typename T> cudaError_t launch_norm(const NormArgs& A, int layout, int64_t tokens, cudaStream_t st) {
  return layout == MTV_ROPE_HALF ? launch_norm_layout<T, true>(A, tokens, st) : launch_norm_layout<T, false>(A, tokens, st);
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
  if (e != cudaSuccess) cudaGetLastError();  // or a later launch reports it
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
