// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits: the target's prediction that the acceptance walk follows ("The Glue
// That Connects" -- "What the Edit Actually Does") and what a server returns
// beside it.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "mla_step_ops.h"
#include "mtv_internal.cuh"

namespace mtv {
namespace {

namespace cg = cooperative_groups;

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

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

__device__ __forceinline__ bool usable_temperature(float s) { return s > 0.f && s < INFINITY; }

// ---------------------------------------------------------------------------
// A row is read once, by a cluster of 1 to 8 blocks that each take a
// contiguous share of it in groups of 64 bytes.  Per thread: the sums S = sum
// 2^t and U = sum 2^t t of t = c x - ref, c = log2(e) / temperature, relative
// to a reference that moves only when a logit passes it by 2^29, and the
// largest group maximum with its group.  Every group's maximum also goes to
// shared memory, so the top k needs no second pass: the k-th largest maximum of
// 64 buckets of groups bounds the k-th logit from below, only groups whose
// maximum reaches it are read again (about k of thousands), and the survivors'
// order is counted.
//
// What bounds it: the bytes of the logits (4,864 rows of 131,072 bf16: 208 us,
// 6.1 TB/s), read by 4 blocks an SM with 64 bytes a thread in flight (3 or 5
// blocks: 225 and 208 us, 1,024 rows 59 and 57 in place of 53); then issue
// slots, about 6 instructions a logit with the fp32 work in pairs (f32x2) and
// one MUFU exponential each.  The top k adds 2 us to a wave of blocks and
// 1.7 us to the latency of few rows (8 x 32,000: 5.6 us).
// ---------------------------------------------------------------------------
constexpr int kMaxGroups = 8192;      // groups a block: their maxima fill 16 or 32 KB
constexpr int kListed = 256;          // groups that may reach the bound before they are searched by rank
constexpr int kPicked = MTV_MAX_TOP;  // groups read again at most
constexpr int kMaxGroup = 32;         // logits a group at most
constexpr int kEdge = 64;             // logits before and after the aligned groups, under 32 each
constexpr int kCand = kPicked * kMaxGroup + kEdge;  // logits found at most
constexpr int kFewCand = 128;         // 4 MTV_MAX_TOP: found from 64 buckets of 4 threads with one logit each
constexpr int kBuckets = 64;
constexpr int kBucketThreads = kLpThreads / kBuckets;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes of logits in four registers.  Maxima stay in one register of the
// logits' type (two of them for 16-bit types) until one value is needed.
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
  static constexpr uint32_t kNone = 0xff80ff80u;  // -inf
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(pair(a), pair(b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float value(uint32_t m) {
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) {
    return make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
  static __device__ __forceinline__ __nv_bfloat16 narrow(float x) {  // x is one already
    return __ushort_as_bfloat16(uint16_t(__float_as_uint(x) >> 16));
  }
};
template <> struct Chunk<__half> {
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2_nan(pair(a), pair(b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float value(uint32_t m) {
    const float2 p = __half22float2(pair(m));
    return max_nan(p.x, p.y);
  }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) { return __half22float2(pair(v[i])); }
  static __device__ __forceinline__ __half2 pair(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
  static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
};
template <> struct Chunk<float> {
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m); }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) {
    return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
  }
  static __device__ __forceinline__ float narrow(float x) { return x; }
};

__device__ __forceinline__ void load16(const void* p, uint32_t* v) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "l"(p));
}

// Pairs of fp32 in one 64-bit register: one instruction for two values.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Sums S and U whose reference moves by d: t becomes t + d.
struct Sums {
  float s, u;
  __device__ __forceinline__ Sums moved(float d) const {
    const float w = exp2_approx(d);
    return w > 0.f ? Sums{s * w, (u + s * d) * w} : Sums{0.f, 0.f};
  }
};

constexpr float kRefSlack = 29.f;
constexpr float kLowest = -3.402823466e38f;

struct LpShared {
  uint64_t cand[kCand];
  uint64_t bucket[kBuckets];
  uint64_t round[2][kLpWarps];
  uint16_t listed[kListed], picked[kPicked];
  float wm[kLpWarps], ws[kLpWarps], wu[kLpWarps];
  // written by every block of the cluster into the first one's
  float part_m[kMaxCluster], part_s[kMaxCluster], part_u[kMaxCluster];
  int part_bad[kMaxCluster], part_found[kMaxCluster];
  uint64_t part_key[kMaxCluster][MTV_MAX_TOP];
  uint64_t bound;
  int num_listed, num_cand;
};

// Groups in the order of larger maxima and then lower groups: larger keys first.
__device__ __forceinline__ uint64_t group_key(float m, int g) { return order_key(m, uint32_t(g)); }

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_rows_kernel(const LogprobArgs A, int blocks) {
  extern __shared__ __align__(16) unsigned char dyn[];
  T* group_max = reinterpret_cast<T*>(dyn);
  __shared__ LpShared sh;
  constexpr int kChunks = 4;                       // of 16 bytes: a group's, and a thread's of a step
  constexpr int kGroup = 64 / int(sizeof(T));      // logits a group
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = blocks > 1 ? int(blockIdx.x % unsigned(blocks)) : 0;
  const int64_t r = blocks > 1 ? int64_t(blockIdx.x / unsigned(blocks)) : int64_t(blockIdx.x);
  cg::cluster_group cluster = cg::this_cluster();
  if (blocks > 1) cluster.barrier_arrive();
  grid_launch_dependents();

  const T* x = static_cast<const T*>(A.logits) + r * A.row_stride;
  const float scale = A.inv_temperature ? A.inv_temperature[r] : 1.f;
  // the token that this row scores, fetched ahead of its use
  float token_x = 0.f;
  int token = -1;
  const bool scores = rank == 0 && tid == 0 && A.tokens && !A.token_rows && r < A.num_tokens;
  if (scores) {
    token = A.tokens[r];
    if (token >= 0 && token < A.vocab) token_x = to_float(x[token]);
  }
  // aligned groups [g0, g0 + n) of this block; logits before and after them
  const int skew = int(reinterpret_cast<uintptr_t>(x) & 63) / int(sizeof(T));
  const int head = min(skew ? 64 / int(sizeof(T)) - skew : 0, A.vocab);
  const int all = (A.vocab - head) / kGroup;
  const int share = (all + blocks - 1) / blocks;
  const int g0 = min(rank * share, all), n = min(share, all - g0);
  const T* body = x + head + int64_t(g0) * kGroup;

  Sums acc{0.f, 0.f};
  float ref = kLowest;
  const float c2 = scale * kLog2e;
  // a difference of logits in powers of two; scale * log2(e) passes fp32's range
  // before scale does, and a difference of 0 has to stay 0
  auto powers = [&](float d) { return c2 < INFINITY ? d * c2 : d * scale * kLog2e; };
  float tmax = -INFINITY, tnext = -INFINITY;  // largest and second largest group maximum
  float worst = -INFINITY;  // NaN or +inf once a logit was
  int tgroup = 0xffff;
  bool bad = !usable_temperature(scale);
  const uint64_t c22 = pack2(c2, c2);
  uint64_t s2 = 0, u2 = 0;
  auto fold = [&]() {
    const float2 a = unpack2(s2), b = unpack2(u2);
    acc.s += a.x + a.y;
    acc.u += b.x + b.y;
    s2 = u2 = 0;
  };
  // A step of a warp is 32 neighbouring groups, as kChunks runs of 32 chunks: a
  // lane loads chunk `lane` of each run.  A group's maximum is put together
  // from the lanes that hold its chunks; lane l ends up with group own + step.
  const int own = w * 32 + (lane % kChunks) * (32 / kChunks) + lane / kChunks;
  auto process = [&](const uint32_t* v, int step) {
    uint32_t c[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      c[i] = Chunk<T>::larger(Chunk<T>::larger(v[4 * i], v[4 * i + 1]), Chunk<T>::larger(v[4 * i + 2], v[4 * i + 3]));
    const float m = Chunk<T>::value(Chunk<T>::larger(Chunk<T>::larger(c[0], c[1]), Chunk<T>::larger(c[2], c[3])));
    worst = max_nan(worst, m);
    // run r of the maxima goes to the lanes with lane % kChunks == r, halving the runs each time
#pragma unroll
    for (int h = kChunks / 2; h > 0; h >>= 1) {
      const bool upper = (lane & h) != 0;
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? c[i] : c[i + h], h);
        c[i] = Chunk<T>::larger(upper ? c[i + h] : c[i], other);
      }
    }
    const float gm = Chunk<T>::value(c[0]);
    const int g = own + step;
    if (g < n) {
      group_max[g] = Chunk<T>::narrow(gm);
      tnext = fmaxf(tnext, fminf(gm, tmax));
      if (gm > tmax) {
        tmax = gm;
        tgroup = g;
      }
    }
    const float z = m * c2;
    if (z > ref + kRefSlack) {
      fold();
      acc = acc.moved(ref - z);
      ref = z;
    }
    const uint64_t ref2 = pack2(-ref, -ref);
    uint64_t ug = 0;
#pragma unroll
    for (int i = 0; i < kGroup / 2; ++i) {
      const float2 p = Chunk<T>::get(v, i);
      const uint64_t t2 = fma2(pack2(p.x, p.y), c22, ref2);
      const float2 t = unpack2(t2);
      const uint64_t e = pack2(exp2_approx(t.x), exp2_approx(t.y));
      s2 = add2(s2, e);
      ug = fma2(e, t2, ug);
    }
    const float2 h = unpack2(ug);
    if (isnan(h.x + h.y)) {  // 0 * -inf: a logit at -inf, or so low that t is
      ug = 0;
      if (m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kGroup / 2; ++i) {
          const float2 p = Chunk<T>::get(v, i);
          const float2 t = unpack2(fma2(pack2(p.x, p.y), c22, ref2));
          const float tx = fmaxf(t.x, -1000.f), ty = fmaxf(t.y, -1000.f);  // 2^-1000 is 0
          ug = fma2(pack2(exp2_approx(tx), exp2_approx(ty)), pack2(tx, ty), ug);
        }
      }
    }
    u2 = add2(u2, ug);
  };
  constexpr int kChunkLogits = 16 / int(sizeof(T));
#pragma unroll 1
  for (int step = 0; w * 32 + step < n; step += kLpThreads) {
    const int from = w * 32 + step;
    const T* at = body + int64_t(from) * kGroup + lane * kChunkLogits;
    uint32_t v[4 * kChunks];
    if (from + 32 <= n) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) load16(at + i * 32 * kChunkLogits, v + 4 * i);
    } else {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (from + (i * 32 + lane) / kChunks < n) load16(at + i * 32 * kChunkLogits, v + 4 * i);
        else v[4 * i] = v[4 * i + 1] = v[4 * i + 2] = v[4 * i + 3] = Chunk<T>::kNone;
      }
    }
    process(v, step);
  }
  fold();
  bad |= !(worst < INFINITY);
  // the edges: thread tid < kEdge of the first block takes one logit
  const int tail0 = head + all * kGroup;
  float edge = -INFINITY;
  int edge_id = -1;
  if (rank == 0 && tid < head) edge_id = tid;
  else if (rank == 0 && tid >= kEdge / 2 && tail0 + tid - kEdge / 2 < A.vocab && tid < kEdge) edge_id = tail0 + tid - kEdge / 2;
  if (edge_id >= 0) {
    edge = to_float(x[edge_id]);
    bad |= !(edge < INFINITY);
    const float z = edge * c2;
    if (z > ref + kRefSlack) {
      acc = acc.moved(ref - z);
      ref = z;
    }
    const float t = fmaf(edge, c2, -ref), e = exp2_approx(t);
    acc.s += e;
    acc.u += e > 0.f ? e * t : 0.f;
  }

  // The block's maximum and the buckets' largest group keys.  A bucket is a few
  // neighbouring threads: the k-th largest of 64 buckets' keys is reached by k
  // groups at least, and by 1.4 k on average at k = 32.
  auto fill_bucket = [&](uint64_t key) {  // the largest of a bucket's threads' keys
#pragma unroll
    for (int o = 1; o < kBucketThreads; o <<= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (tid % kBucketThreads == 0) sh.bucket[tid / kBucketThreads] = key;
  };
  auto find_bound = [&]() {  // the k-th largest bucket: a bucket's threads count its rank
    const uint64_t mine = sh.bucket[tid / kBucketThreads];
    int above = 0;
#pragma unroll
    for (int j = 0; j < kBuckets; j += kBucketThreads) above += sh.bucket[j + tid % kBucketThreads] > mine;
#pragma unroll
    for (int o = 1; o < kBucketThreads; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (above == A.top_k - 1 && tid % kBucketThreads == 0) sh.bound = mine;
  };
  float m = fmaxf(tmax, edge);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.wm[w] = m;
  if (A.top_k > 0) {
    // threads without a group above -inf rank last, each apart from the others
    const uint64_t key = tmax > -INFINITY ? group_key(tmax, tgroup) : group_key(-INFINITY, kMaxGroups + tid);
    fill_bucket(key);
    if (tid == 0) sh.num_listed = sh.num_cand = 0;
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int i = 0; i < kLpWarps; ++i) m = fmaxf(m, sh.wm[i]);
  // sums relative to the block's maximum: t = c (x - m)
  Sums total{0.f, 0.f};
  if (m > -INFINITY && !bad) {
    if (fabsf(m * c2) < 0x1p30f) {
      total = acc.moved(fmaf(-c2, m, ref));
    } else {
      // so far from 0 that a reference's rounding (2^-24 of it) is no longer a
      // small t, or c2 is no number: once more, from differences to the maximum
      for (int i = tid; i < n * kGroup; i += kLpThreads) {
        const float t = powers(to_float(body[i]) - m), e = exp2_approx(t);
        total.s += e;
        total.u += e > 0.f ? e * t : 0.f;
      }
      if (edge_id >= 0) {
        const float t = powers(edge - m), e = exp2_approx(t);
        total.s += e;
        total.u += e > 0.f ? e * t : 0.f;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total.s += __shfl_xor_sync(0xffffffffu, total.s, o);
    total.u += __shfl_xor_sync(0xffffffffu, total.u, o);
  }
  if (lane == 0) {
    sh.ws[w] = total.s;
    sh.wu[w] = total.u;
  }
  if (A.top_k > 0) find_bound();
  __syncthreads();
  total.s = total.u = 0.f;
#pragma unroll
  for (int i = 0; i < kLpWarps; ++i) {
    total.s += sh.ws[i];
    total.u += sh.wu[i];
  }
  LpShared* to = blocks > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
  if (blocks > 1) {
    cluster.barrier_wait();  // the first block is there
    if (tid == 0) {
      to->part_m[rank] = m;
      to->part_s[rank] = total.s;
      to->part_u[rank] = total.u;
      to->part_bad[rank] = bad;
    }
  }
  // What a single block knows of the row already, the first of several later:
  // m times the scale rounds; what that leaves goes into ln S, so that one
  // fused multiply-add z - zmax, less ln S, is right to the roundings of both
  float zmax, log_s, entropy;
  auto finish = [&]() {
    zmax = m * scale;
    bad |= m > -INFINITY && !(fabsf(zmax) < INFINITY);
    if (bad) {
      log_s = entropy = zmax = NAN;
    } else if (m == -INFINITY) {
      log_s = -INFINITY;
      entropy = 0.f;
    } else {
      const float l = logf(total.s);
      log_s = l + fmaf(m, scale, -zmax);
      entropy = l - kLn2 * (total.u / total.s);
    }
    if (tid == 0) {
      A.stats[r] = zmax;
      A.stats[A.num_rows + r] = log_s;
      A.stats[2 * A.num_rows + r] = entropy;
      uint32_t word = bad ? MTV_DEVERR_LOGITS : 0;
      if (scores) {
        float lp = 0.f;
        if (token < -1 || token >= A.vocab) {
          lp = NAN;
          word |= MTV_DEVERR_TOKEN;
        } else if (token >= 0) {
          lp = token_x == -INFINITY && !bad ? -INFINITY : fmaf(token_x, scale, -zmax) - log_s;
        }
        A.logprobs[r] = lp;
      }
      if (word) set_err(A.err, word);
    }
  };
  auto write_top = [&](int k, uint64_t key) {
    A.top_tokens[k * A.num_rows + r] = int32_t(~uint32_t(key));
    A.top_logprobs[k * A.num_rows + r] = fmaf(key_logit(key), scale, -zmax) - log_s;
  };
  auto write_none = [&](int from) {
    for (int k = from + tid; k < A.top_k; k += kLpThreads) {
      A.top_tokens[k * A.num_rows + r] = -1;
      A.top_logprobs[k * A.num_rows + r] = bad ? NAN : -INFINITY;
    }
  };
  if (blocks == 1) finish();
  if (A.top_k == 0 && blocks == 1) return;

  // the block's top k: groups that reach the bound, their logits, their order
  int found = 0;
  if (A.top_k > 0 && !bad) {
    const uint64_t bound = sh.bound;
    const float least = key_logit(bound);
    auto list = [&](float v, int at) {
      if (v > -INFINITY && group_key(v, at) >= bound) {
        const int i = atomicAdd(&sh.num_listed, 1);
        if (i < kListed) sh.listed[i] = uint16_t(at);
      }
    };
    list(tmax, tgroup);
    if (tnext > -INFINITY && tnext >= least) {  // rare: a second group of the thread
      for (int at = own; at < n; at += kLpThreads)
        if (at != tgroup) list(to_float(group_max[at]), at);
    }
    if (edge > -INFINITY) sh.cand[atomicAdd(&sh.num_cand, 1)] = order_key(edge, uint32_t(edge_id));
    __syncthreads();
    const int listed = sh.num_listed;
    const uint16_t* pick = sh.listed;
    int picked = listed;
    if (listed > kListed) {  // the large logits sit in few buckets, or many are equal: one search a rank
      uint64_t below = ~uint64_t(0);
      for (picked = 0; picked < A.top_k; ++picked) {
        uint64_t best = 0;
        for (int at = tid; at < n; at += kLpThreads) {
          const uint64_t key = group_key(to_float(group_max[at]), at);
          if (key < below && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
          best = other > best ? other : best;
        }
        if (lane == 0) sh.round[picked & 1][w] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLpWarps; ++i) best = sh.round[picked & 1][i] > best ? sh.round[picked & 1][i] : best;
        if (best == 0 || key_logit(best) == -INFINITY) break;
        below = best;
        if (tid == 0) sh.picked[picked] = uint16_t(~uint32_t(best));
      }
      pick = sh.picked;
      __syncthreads();
    } else if (listed > kPicked) {  // the first k of them
      for (int i = tid; i < listed; i += kLpThreads) {
        const int at = sh.listed[i];
        const uint64_t key = group_key(to_float(group_max[at]), at);
        int above = 0;
        for (int j = 0; j < listed; ++j) above += group_key(to_float(group_max[sh.listed[j]]), sh.listed[j]) > key;
        if (above < A.top_k) sh.picked[above] = uint16_t(at);
      }
      picked = A.top_k;
      pick = sh.picked;
      __syncthreads();
    }
    for (int i0 = tid; i0 < picked * kGroup; i0 += 4 * kLpThreads) {  // four loads in flight
      float v[4];
      int id[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = i0 + b * kLpThreads;
        v[b] = -INFINITY;
        if (i < picked * kGroup) {
          id[b] = head + (g0 + pick[i / kGroup]) * kGroup + i % kGroup;
          v[b] = to_float(x[id[b]]);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (v[b] >= least && v[b] > -INFINITY) sh.cand[atomicAdd(&sh.num_cand, 1)] = order_key(v[b], uint32_t(id[b]));
    }
    __syncthreads();
    found = sh.num_cand;
    // Many logits of few groups (a small vocabulary, a mask that leaves little):
    // the bound once more, over the logits.  k buckets of 4 threads with c logits
    // each leave 128 c of over 256 (c - 1) at most, so this ends.
    while (found > kFewCand) {
      uint64_t mine[(kCand + kLpThreads - 1) / kLpThreads], best = 0;
#pragma unroll
      for (int q = 0; q < (kCand + kLpThreads - 1) / kLpThreads; ++q) {
        const int i = tid + q * kLpThreads;
        mine[q] = i < found ? sh.cand[i] : 0;
        best = mine[q] > best ? mine[q] : best;
      }
      fill_bucket(best);
      __syncthreads();
      find_bound();
      if (tid == 0) sh.num_cand = 0;
      __syncthreads();
      const uint64_t at_least = sh.bound;
#pragma unroll
      for (int q = 0; q < (kCand + kLpThreads - 1) / kLpThreads; ++q)
        if (mine[q] != 0 && mine[q] >= at_least) sh.cand[atomicAdd(&sh.num_cand, 1)] = mine[q];
      __syncthreads();
      found = sh.num_cand;
    }
  }
  if (A.top_k > 0) {
    for (int i0 = 0; i0 < found; i0 += kLpThreads / 4) {  // four threads count a logit's rank
      const int i = i0 + (tid >> 2);
      const uint64_t key = i < found ? sh.cand[i] : 0;
      int above = 0;
      for (int j = tid & 3; j < found; j += 4) above += sh.cand[j] > key;
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      above += __shfl_xor_sync(0xffffffffu, above, 2);
      if ((tid & 3) == 0 && i < found && above < A.top_k) {
        if (blocks == 1) write_top(above, key);
        else to->part_key[rank][above] = key;
      }
    }
    if (blocks == 1) {
      write_none(min(found, A.top_k));
      return;
    }
    for (int i = found + tid; i < A.top_k; i += kLpThreads) to->part_key[rank][i] = 0;
    if (tid == 0) to->part_found[rank] = min(found, A.top_k);
  }
  cluster.sync();
  if (rank != 0) return;

  // the row, from its blocks' shares
  for (int i = 0; i < blocks; ++i) {
    m = fmaxf(m, sh.part_m[i]);
    bad |= sh.part_bad[i] != 0;
  }
  total = Sums{0.f, 0.f};
  for (int i = 0; i < blocks && m > -INFINITY; ++i) {
    const Sums p = Sums{sh.part_s[i], sh.part_u[i]}.moved(powers(sh.part_m[i] - m));
    total.s += p.s;
    total.u += p.u;
  }
  finish();
  // ranks over the blocks' sorted lists; keys of different logits differ
  for (int i = tid; i < A.top_k * blocks && !bad; i += kLpThreads) {
    const int b = i / A.top_k, k = i - b * A.top_k;
    const uint64_t key = sh.part_key[b][k];
    int above = k;
    for (int o = 0; o < blocks; ++o) {
      if (o == b) continue;
      int lo = 0, hi = A.top_k;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sh.part_key[o][mid] > key) lo = mid + 1;
        else hi = mid;
      }
      above += lo;
    }
    if (key != 0 && above < A.top_k) write_top(above, key);
  }
  if (A.top_k > 0) {
    int have = 0;  // logits above -inf; the ranks behind them have none
    for (int b = 0; b < blocks && !bad; ++b) have += sh.part_found[b];
    write_none(have);
  }
}

// Tokens scored by rows of their own choice, from the rows' stats: a
// programmatic dependent of the rows' kernel, so that its launch and its reads
// of the inputs are done by the time the stats are there.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_tokens_kernel(const LogprobArgs A) {
  const int64_t i = int64_t(blockIdx.x) * kLpThreads + threadIdx.x;
  const bool live = i < A.num_tokens;
  const int64_t r = live ? int64_t(A.token_rows[i]) : -1;
  const int tok = live ? A.tokens[i] : -1;
  const bool known = r >= 0 && r < A.num_rows;
  float x = 0.f, scale = 1.f;
  if (known && tok >= 0 && tok < A.vocab) {
    x = to_float(static_cast<const T*>(A.logits)[r * A.row_stride + tok]);
    if (A.inv_temperature) scale = A.inv_temperature[r];
  }
  grid_dependency_wait();
  if (!live) return;
  float lp = NAN;
  if (!known || tok < -1 || tok >= A.vocab) {
    set_err(A.err, MTV_DEVERR_TOKEN);
  } else if (tok < 0) {
    lp = 0.f;
  } else {
    const float log_s = A.stats[A.num_rows + r];
    lp = x == -INFINITY && !isnan(log_s) ? -INFINITY : fmaf(x, scale, -A.stats[r]) - log_s;
  }
  A.logprobs[i] = lp;
}

// Blocks a row: doubled while a block's groups do not fit its shared memory,
// and while there are SMs for more blocks and each keeps enough of the row to
// pay for the cluster and one more top k.  Measured (us; blocks 1, 2, 4, 8):
//   8 x 32,000 bf16      5.6   6.0   5.9   6.3      64 x 131,072 bf16   16.0  11.8  10.0  11.5
//   8 x 131,072 bf16    12.6   9.9   8.1   7.8     152 x 131,072 bf16   18.5  14.7  19.1  24.1
//   1 x 64,000 bf16      7.9   7.3   6.7   7.1     304 x 131,072 bf16   21.4  19.9  29.1  39.8
//   8 x 131,072 fp32    17.2  12.5   9.2   8.6     304 x 32,000 bf16     9.1  11.5  19.0  32.0
// The bounds on a block's bytes are those of measured sizes, with no margin:
// 128 KB is 131,072 bf16 in two, 32,000 bytes 64,000 bf16 in four.  A little
// less, 129,280 bf16 say, falls to the rule's other side (one block a row from
// 153 rows on, in place of two), of which nothing has been measured.
int blocks_per_row(int64_t rows, int vocab, int size) {
  const int groups = vocab / (64 / size);
  int b = 1;
  for (; b < kMaxCluster; b *= 2) {
    const int share = vocab * size / (2 * b);  // bytes a block with twice as many
    const int64_t most = share >= 128 * 1024 ? 608 : share >= 48 * 1024 ? 304 : share >= 32000 && b > 1 ? 152 : 0;
    if (groups <= b * kMaxGroups && rows * b * 2 > most) break;
  }
  return b;
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs& A, cudaStream_t st) {
  if (A.num_rows > 0) {
    const int blocks = blocks_per_row(A.num_rows, A.vocab, int(sizeof(T)));
    const int share = (A.vocab / (64 / int(sizeof(T))) + blocks - 1) / blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(A.num_rows) * unsigned(blocks));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = size_t(share) * sizeof(T);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(blocks), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    // within the 48 KB that need no leave (a block's groups: MTV_MAX_VOCAB over 8 blocks at most)
    static_assert(sizeof(LpShared) + kMaxGroups * sizeof(float) <= 48 * 1024);
    static_assert(MTV_MAX_VOCAB / (64 / sizeof(T)) <= kMaxGroups * kMaxCluster);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, logprob_rows_kernel<T>, A, blocks);
    if (e != cudaSuccess) return e;
  }
  if (A.num_tokens > 0 && A.token_rows) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((A.num_tokens + kLpThreads - 1) / kLpThreads));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = A.num_rows > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logprob_tokens_kernel<T>, A);
  }
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
  if (num_rows > INT32_MAX / mtv::kMaxCluster || num_tokens > INT32_MAX) return MTV_E_UNSUPPORTED;
  if (num_rows == 0 && num_tokens == 0) return MTV_OK;
  if ((num_rows > 0 && (!logits || !stats)) || (num_tokens > 0 && (!tokens || !logprobs)) ||
      (top_k > 0 && num_rows > 0 && (!top_tokens || !top_logprobs)))
    return MTV_E_NULL_POINTER;
  const uintptr_t size = dtype == MTV_DTYPE_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) & (size - 1)) return MTV_E_BAD_ARGUMENT;
  const LogprobArgs A{logits, inv_temperature, tokens, token_rows, logprobs, stats, top_tokens, top_logprobs,
                      err,    num_rows,        row_stride, num_tokens, vocab,  top_k};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MTV_DTYPE_BF16) e = launch_logprobs<__nv_bfloat16>(A, st);
  else if (dtype == MTV_DTYPE_FP16) e = launch_logprobs<__half>(A, st);
  else e = launch_logprobs<float>(A, st);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
