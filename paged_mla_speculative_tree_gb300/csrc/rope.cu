// Rotary positions of the queries' rope part and the write of new latent rows
// into the paged pool, and the frequency table they read (the 64 rope dims of
// a latent row: "The Glue That Binds" -- "The Broader Engineering Effort").
#include <math.h>
#include <stdint.h>

#include "mla_step_ops.h"
#include "mtv_internal.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
  const uint64_t* turns;
  const int64_t* positions;
  const int64_t* num_valid;
  const void* q_in;
  void* q_out;
  const void* k_in;
  const void* c_in;
  const int64_t* out_cache_loc;
  __nv_bfloat16* pool;
  uint32_t* err;
  int64_t q_in_tok, q_in_head, q_out_tok, q_out_head, k_tok, c_tok, num_slots;
  float amplitude;
  int rope_dim, num_heads, inverse;
};

// One block a token.  Pair i's angle is position * turns[i] modulo one turn in
// 64-bit fixed point (the multiplication's wrap drops the whole turns exactly),
// of which the high 32 bits, signed, go to sincospi as half turns: the angle is
// off by at most 2^-25 half turns from rounding them to fp32, at any position.
// Each angle is computed once a token and serves all heads.
//
// What bounds it: for many tokens the bytes of the queries' rotary part, read
// and written once (128-byte pieces of 1152-byte rows); for few the chain
// position -> angle -> barrier -> store, so every load of the token, whether
// it turns out valid or not, is issued before the first use of any.  8 tokens
// of 64 heads take 2.3 us, 1,024 4.5 us, 8,191 28 us (5.4 TB/s).
//
// Vector form: a thread's unit is 4 or 8 pairs in two 16-byte pieces
// (neighbours when interleaved, a half apart otherwise).  Its conditions
// (16-byte alignment of every address, whole units a head) are checked by the
// launch; the plain form below takes any strides and any even length, a pair
// at a time (8,191 tokens: 73 us in place of 28).
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_write_vec_kernel(const RopeArgs A) {
  constexpr int V = 16 / int(sizeof(T));             // values of 16 bytes: pairs a unit
  constexpr int kItems = sizeof(T) == 4 ? 4 : 2;     // units in flight a thread
  constexpr int kLatent = kDLat / (kRopeThreads / 2);  // 8 latent values each for half of the threads
  __shared__ __align__(16) float cos_s[MTV_MAX_ROPE_DIM / 2], sin_s[MTV_MAX_ROPE_DIM / 2];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, pairs = A.rope_dim / 2, units = pairs / V;
  const int second = kHalf ? pairs : V;
  auto first = [&](int u) { return kHalf ? u * V : 2 * u * V; };

  const int total = A.q_in ? A.num_heads * units : 0;
  const T* q_in = static_cast<const T*>(A.q_in) + t * A.q_in_tok;
  T* q_out = static_cast<T*>(A.q_out) + t * A.q_out_tok;
  uint4 qa[kItems], qb[kItems];
  auto load_q = [&](int base) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = base + i * kRopeThreads;
      if (x < total) {
        const int h = x / units, d = first(x - h * units);
        qa[i] = *reinterpret_cast<const uint4*>(q_in + h * A.q_in_head + d);
        qb[i] = *reinterpret_cast<const uint4*>(q_in + h * A.q_in_head + d + second);
      }
    }
  };
  load_q(tid);
  uint4 la = make_uint4(0, 0, 0, 0), lb = la;  // the latent part, or a unit of the key part
  int64_t slot = -1;
  const bool latent = A.pool && tid < kRopeThreads / 2;
  const bool key = A.pool && tid >= kRopeThreads / 2 && tid - kRopeThreads / 2 < units;
  const int key_unit = tid - kRopeThreads / 2;
  if (A.pool) slot = A.out_cache_loc[t];
  if (latent) {
    const T* c = static_cast<const T*>(A.c_in) + t * A.c_tok + tid * kLatent;
    la = *reinterpret_cast<const uint4*>(c);
    if (V == 4) lb = *reinterpret_cast<const uint4*>(c + 4);
  } else if (key) {
    const T* k = static_cast<const T*>(A.k_in) + t * A.k_tok + first(key_unit);
    la = *reinterpret_cast<const uint4*>(k);
    lb = *reinterpret_cast<const uint4*>(k + second);
  }
  const int64_t valid = A.num_valid ? *A.num_valid : INT64_MAX;
  const uint64_t pos = uint64_t(A.positions[t]);
  for (int i = tid; i < pairs; i += kRopeThreads) {
    float s, c;
    sincospif(float(int32_t((pos * A.turns[i]) >> 32)) * 0x1p-31f, &s, &c);
    cos_s[i] = c * A.amplitude;
    sin_s[i] = (A.inverse ? -s : s) * A.amplitude;
  }
  __syncthreads();
  if (t >= valid) return;

  // pairs u * V .. of a unit; interleaved ones alternate through both registers
  auto turn = [&](const uint4& a, const uint4& b, int u, float* y) {
    float x[2 * V], c[V], s[V];
    expand<T>(a, x);
    expand<T>(b, x + V);
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 cc = *reinterpret_cast<const float4*>(&cos_s[u * V + i]);
      const float4 ss = *reinterpret_cast<const float4*>(&sin_s[u * V + i]);
      c[i] = cc.x, c[i + 1] = cc.y, c[i + 2] = cc.z, c[i + 3] = cc.w;
      s[i] = ss.x, s[i + 1] = ss.y, s[i + 2] = ss.z, s[i + 3] = ss.w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = kHalf ? i : 2 * i, k = kHalf ? i + V : 2 * i + 1;
      y[j] = x[j] * c[i] - x[k] * s[i];
      y[k] = x[j] * s[i] + x[k] * c[i];
    }
  };
  for (int base = tid; base < total; base += kItems * kRopeThreads) {
    if (base != tid) load_q(base);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = base + i * kRopeThreads;
      if (x < total) {
        const int h = x / units, u = x - h * units, d = first(u);
        float y[2 * V];
        turn(qa[i], qb[i], u, y);
        *reinterpret_cast<uint4*>(q_out + h * A.q_out_head + d) = pack<T>(y);
        *reinterpret_cast<uint4*>(q_out + h * A.q_out_head + d + second) = pack<T>(y + V);
      }
    }
  }
  if (!A.pool) return;
  if (slot < 0 || slot >= A.num_slots) {
    if (tid == 0 && A.err) atomicOr(A.err, MTV_DEVERR_SLOT_RANGE);
    return;
  }
  __nv_bfloat16* row = A.pool + slot * kDQK;
  if (latent) {
    float x[2 * V];
    expand<T>(la, x);
    if (V == 4) expand<T>(lb, x + 4);
    store_bf16<kLatent>(row + tid * kLatent, x);
  } else if (key) {
    float y[2 * V];
    turn(la, lb, key_unit, y);
    store_bf16<V>(row + kDLat + first(key_unit), y);
    store_bf16<V>(row + kDLat + first(key_unit) + second, y + V);
  }
}

template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs A) {
  __shared__ float cos_s[MTV_MAX_ROPE_DIM / 2], sin_s[MTV_MAX_ROPE_DIM / 2];
  const int64_t t = blockIdx.x;
  if (A.num_valid && t >= *A.num_valid) return;
  const int tid = threadIdx.x, pairs = A.rope_dim / 2;
  const uint64_t pos = uint64_t(A.positions[t]);
  for (int i = tid; i < pairs; i += kRopeThreads) {
    float s, c;
    sincospif(float(int32_t((pos * A.turns[i]) >> 32)) * 0x1p-31f, &s, &c);
    cos_s[i] = c * A.amplitude;
    sin_s[i] = (A.inverse ? -s : s) * A.amplitude;
  }
  __syncthreads();
  auto turn = [&](float x1, float x2, int i, float* y1, float* y2) {
    *y1 = x1 * cos_s[i] - x2 * sin_s[i];
    *y2 = x1 * sin_s[i] + x2 * cos_s[i];
  };
  auto first = [&](int i) { return kHalf ? i : 2 * i; };
  const int second = kHalf ? pairs : 1;

  if (A.q_in) {
    const T* in = static_cast<const T*>(A.q_in) + t * A.q_in_tok;
    T* out = static_cast<T*>(A.q_out) + t * A.q_out_tok;
    for (int64_t x = tid; x < int64_t(A.num_heads) * pairs; x += kRopeThreads) {
      const int64_t h = x / pairs;
      const int i = int(x - h * pairs), d = first(i);
      float y1, y2;
      turn(to_float(in[h * A.q_in_head + d]), to_float(in[h * A.q_in_head + d + second]), i, &y1, &y2);
      out[h * A.q_out_head + d] = from_float<T>(y1);
      out[h * A.q_out_head + d + second] = from_float<T>(y2);
    }
  }
  if (A.pool) {
    const int64_t slot = A.out_cache_loc[t];
    if (slot < 0 || slot >= A.num_slots) {
      if (tid == 0 && A.err) atomicOr(A.err, MTV_DEVERR_SLOT_RANGE);
      return;
    }
    __nv_bfloat16* row = A.pool + slot * kDQK;
    const T* c = static_cast<const T*>(A.c_in) + t * A.c_tok;
    for (int x = tid; x < kDLat; x += kRopeThreads) row[x] = __float2bfloat16_rn(to_float(c[x]));
    const T* k = static_cast<const T*>(A.k_in) + t * A.k_tok;
    for (int i = tid; i < pairs; i += kRopeThreads) {
      const int d = first(i);
      float y1, y2;
      turn(to_float(k[d]), to_float(k[d + second]), i, &y1, &y2);
      row[kDLat + d] = __float2bfloat16_rn(y1);
      row[kDLat + d + second] = __float2bfloat16_rn(y2);
    }
  }
}

// Whether every address that the vector form touches is 16-byte aligned.
template <typename T> bool vector_form(const RopeArgs& A) {
  constexpr int64_t v = 16 / int64_t(sizeof(T));
  uint64_t bits = 0;
  if (A.q_in)
    bits |= reinterpret_cast<uintptr_t>(A.q_in) | reinterpret_cast<uintptr_t>(A.q_out) |
            uint64_t((A.q_in_tok | A.q_in_head | A.q_out_tok | A.q_out_head) % v != 0);
  if (A.pool)
    bits |= reinterpret_cast<uintptr_t>(A.k_in) | reinterpret_cast<uintptr_t>(A.c_in) |
            uint64_t((A.k_tok | A.c_tok) % v != 0);
  return (bits & 15) == 0 && A.rope_dim % (2 * v) == 0 && int64_t(A.num_heads) * A.rope_dim < INT32_MAX / 2;
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& A, int layout, int64_t tokens, cudaStream_t st) {
  const bool half = layout == MTV_ROPE_HALF, vec = vector_form<T>(A);
  auto kernel = vec ? (half ? rope_write_vec_kernel<T, true> : rope_write_vec_kernel<T, false>)
                    : (half ? rope_write_kernel<T, true> : rope_write_kernel<T, false>);
  kernel<<<unsigned(tokens), kRopeThreads, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mtv

extern "C" int mla_rope_freqs(int rope_dim, double base, const mtv_rope_scaling_t* scaling, uint64_t* turns,
                              float* amplitude) {
  if (!turns || !amplitude) return MTV_E_NULL_POINTER;
  if (rope_dim < 2 || rope_dim > MTV_MAX_ROPE_DIM || (rope_dim & 1) || !(base > 1.0) || !isfinite(base))
    return MTV_E_BAD_ARGUMENT;
  mtv_rope_scaling_t s = {};
  s.factor = 1.0;
  if (scaling) s = *scaling;
  if (s.kind < MTV_ROPE_SCALE_NONE || s.kind > MTV_ROPE_SCALE_WAVELENGTH || s.reserved != 0 ||
      !isfinite(s.amplitude) || s.amplitude < 0)
    return MTV_E_BAD_ARGUMENT;
  if (s.kind != MTV_ROPE_SCALE_NONE && !(s.factor >= 1.0 && isfinite(s.factor))) return MTV_E_BAD_ARGUMENT;
  const bool by_length = s.kind == MTV_ROPE_SCALE_YARN || s.kind == MTV_ROPE_SCALE_WAVELENGTH;
  if (by_length && !(s.original_len > 0 && isfinite(s.original_len))) return MTV_E_BAD_ARGUMENT;
  if (s.kind == MTV_ROPE_SCALE_YARN && !(s.beta_slow > 0 && s.beta_fast > s.beta_slow && isfinite(s.beta_fast)))
    return MTV_E_BAD_ARGUMENT;
  if (s.kind == MTV_ROPE_SCALE_WAVELENGTH &&
      !(s.low_turns > 0 && s.high_turns > s.low_turns && isfinite(s.high_turns)))
    return MTV_E_BAD_ARGUMENT;
  const double two_pi = 6.283185307179586476925286766559;
  double lo = 0, hi = 0;
  if (s.kind == MTV_ROPE_SCALE_YARN) {
    // the pair index that turns b times in original_len, solved from base^(-2i/d)
    auto at = [&](double b) { return rope_dim * log(s.original_len / (b * two_pi)) / (2.0 * log(base)); };
    lo = fmax(floor(at(s.beta_fast)), 0.0);
    hi = fmin(ceil(at(s.beta_slow)), double(rope_dim - 1));
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < rope_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rope_dim);
    if (s.kind == MTV_ROPE_SCALE_LINEAR) {
      f /= s.factor;
    } else if (s.kind == MTV_ROPE_SCALE_YARN) {
      const double ramp = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f = f / s.factor * ramp + f * (1.0 - ramp);
    } else if (s.kind == MTV_ROPE_SCALE_WAVELENGTH) {
      const double n = s.original_len * f / two_pi;
      const double keep = fmin(fmax((n - s.low_turns) / (s.high_turns - s.low_turns), 0.0), 1.0);
      f = (1.0 - keep) * f / s.factor + keep * f;
    }
    turns[i] = uint64_t(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  double amp = s.amplitude;
  if (amp == 0) amp = s.kind == MTV_ROPE_SCALE_YARN ? 0.1 * log(s.factor) + 1.0 : 1.0;
  *amplitude = float(amp);
  return MTV_OK;
}

extern "C" int mla_rope_write(const uint64_t* turns, int rope_dim, float amplitude, int layout, int inverse,
                              const int64_t* positions, int64_t num_tokens, const int64_t* num_valid, int dtype,
                              const void* q_in, int64_t q_in_tok_stride, int64_t q_in_head_stride, void* q_out,
                              int64_t q_out_tok_stride, int64_t q_out_head_stride, int num_heads, const void* k_in,
                              int64_t k_tok_stride, const void* c_in, int64_t c_tok_stride,
                              const int64_t* out_cache_loc, void* kv_pool, int64_t num_slots, uint32_t* err,
                              void* stream) {
  using namespace mtv;
  if (rope_dim < 2 || rope_dim > MTV_MAX_ROPE_DIM || (rope_dim & 1) || !isfinite(amplitude) ||
      (layout != MTV_ROPE_INTERLEAVED && layout != MTV_ROPE_HALF) || (inverse != 0 && inverse != 1) ||
      num_tokens < 0 || num_heads < 0 || num_slots < 0 || dtype < MTV_DTYPE_BF16 || dtype > MTV_DTYPE_FP32)
    return MTV_E_BAD_ARGUMENT;
  if (num_tokens > INT32_MAX) return MTV_E_UNSUPPORTED;
  if ((q_in == nullptr) != (q_out == nullptr)) return MTV_E_NULL_POINTER;
  if (kv_pool) {
    if (rope_dim != kDRope) return MTV_E_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(kv_pool) & 15) return MTV_E_BAD_ARGUMENT;
  }
  if (num_tokens == 0 || (!kv_pool && (!q_in || num_heads == 0))) return MTV_OK;
  if (!turns || !positions || (kv_pool && (!k_in || !c_in || !out_cache_loc))) return MTV_E_NULL_POINTER;
  const uintptr_t size = dtype == MTV_DTYPE_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(q_in) | reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k_in) |
       reinterpret_cast<uintptr_t>(c_in)) & (size - 1))
    return MTV_E_BAD_ARGUMENT;
  const RopeArgs A{turns,  positions, num_valid, q_in, q_out, k_in, c_in, out_cache_loc,
                   static_cast<__nv_bfloat16*>(kv_pool), err, q_in_tok_stride, q_in_head_stride, q_out_tok_stride,
                   q_out_head_stride, k_tok_stride, c_tok_stride, num_slots, amplitude, rope_dim, num_heads, inverse};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MTV_DTYPE_BF16) e = launch_rope<__nv_bfloat16>(A, layout, num_tokens, st);
  else if (dtype == MTV_DTYPE_FP16) e = launch_rope<__half>(A, layout, num_tokens, st);
  else e = launch_rope<float>(A, layout, num_tokens, st);
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
