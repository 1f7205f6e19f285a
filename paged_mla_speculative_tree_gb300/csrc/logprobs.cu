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
// contiguous share of it in groups of 16 logits (one or two 32-byte loads of a
// thread).  Per thread: the sums S and U = sum e^d d of d = z - ref relative to
// a reference that moves only when a logit passes it by 20, and the largest
// group maximum with its group.  Every group's maximum also goes to shared
// memory, so the top k needs no second pass: the k-th largest of the threads'
// maxima (by value, then lower group) bounds the k-th logit from below, only
// groups whose maximum reaches it are read again (about k of thousands), and
// the survivors' order is counted.
//
// What bounds it: the bytes of the logits; then issue slots -- about 5
// instructions a logit, with the fp32 work in pairs (f32x2) and one MUFU
// exponential each.
// ---------------------------------------------------------------------------
constexpr int kGroup = 16;            // logits a group
constexpr int kMaxGroups = 8192;      // groups a block: their maxima fill 16 or 32 KB
constexpr int kOwners = 48;           // most threads whose maxima may reach the bound
constexpr int kPicked = 64;           // most groups read again
constexpr int kEdge = 32;             // logits before and after the aligned groups, at most 15 each
constexpr int kListed = kOwners * (kMaxGroups / kLpThreads);
constexpr int kMaxCluster = 8;

template <typename T> struct Groups;  // one group in registers
template <> struct Groups<__nv_bfloat16> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ float max(const uint32_t* v) {
    __nv_bfloat162 m = pair(v[0]);
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = __hmax2_nan(m, pair(v[i]));
    return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
  }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) {
    return make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
  static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Groups<__half> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ float max(const uint32_t* v) {
    __half2 m = pair(v[0]);
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = __hmax2_nan(m, pair(v[i]));
    return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
  }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) { return __half22float2(pair(v[i])); }
  static __device__ __forceinline__ __half2 pair(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
  static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
};
template <> struct Groups<float> {
  static constexpr int kWords = 16;
  static __device__ __forceinline__ float max(const uint32_t* v) {
    float m = __uint_as_float(v[0]);
#pragma unroll
    for (int i = 1; i < kWords; ++i)
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(__uint_as_float(v[i])));
    return m;
  }
  static __device__ __forceinline__ float2 get(const uint32_t* v, int i) {
    return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
  }
  static __device__ __forceinline__ float narrow(float x) { return x; }
};

__device__ __forceinline__ void load32(const void* p, uint32_t* v) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// Sums relative to a reference ref: S = sum e^(z - ref), U = sum e^(z - ref) (z - ref).
struct Sums {
  float ref, s, u;
  __device__ __forceinline__ void move_to(float to) {  // to > -inf
    if (ref > -INFINITY) {
      const float d = ref - to, w = exp2_approx(d * kLog2e);
      u = w > 0.f ? (u + s * d) * w : 0.f;
      s *= w;
    }
    ref = to;
  }
  __device__ __forceinline__ void add(const Sums& o) {  // o has the same reference, or none
    if (o.ref > -INFINITY) {
      s += o.s;
      u += o.u;
    }
  }
};

constexpr float kRefSlack = 20.f;

struct LpShared {
  uint64_t cand[kPicked * kGroup + kEdge];
  float thread_max[kLpThreads];
  uint16_t thread_group[kLpThreads];
  uint16_t listed[kListed];
  uint16_t picked[kPicked];
  float wm[kLpWarps], ws[kLpWarps], wu[kLpWarps];
  // written by every block of the cluster into the first one's
  float part_m[kMaxCluster], part_s[kMaxCluster], part_u[kMaxCluster];
  int part_bad[kMaxCluster], part_found[kMaxCluster];
  uint64_t part_key[kMaxCluster][MTV_MAX_TOP];
  float bound;
  int bound_group, num_listed, num_cand;
};

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

// Warp 0: a bound (value, group) that at least k and at most kOwners of the
// threads' (maximum, first group of it) pairs reach, in the order of larger
// values and then lower groups; -inf and any group when fewer than k threads
// have a maximum above -inf.  Bisection over the values' ordered bits, and
// over the groups among equal values.
__device__ __forceinline__ void select_bound(LpShared& sh, int k) {
  const int lane = threadIdx.x;
  constexpr int kPer = kLpThreads / 32;
  uint32_t v[kPer];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = ordered(sh.thread_max[i * 32 + lane]);
    top = v[i] > top ? v[i] : top;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  auto count_from = [&](uint32_t x) {
    unsigned c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += v[i] >= x;
    return int(__reduce_add_sync(0xffffffffu, c));
  };
  const uint32_t none = ordered(-INFINITY);
  uint32_t lo = none + 1, hi = top;  // the bound's bits lie in [lo, hi]
  int g = 0xffff, c = 0;
  if (top <= none || (c = count_from(lo)) < k) {
    lo = none;
  } else {
    // invariant: count_from(lo) >= k
    while (lo < hi && c > kOwners) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int cm = count_from(mid);
      if (cm >= k) {
        lo = mid;
        c = cm;
      } else {
        hi = mid - 1;
      }
    }
    if (c > kOwners) {  // equal values: the lowest groups among them
      const int above = lo == 0xffffffffu ? 0 : count_from(lo + 1);
      int g0 = 0, g1 = 0xffff;
      uint16_t grp[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) grp[i] = sh.thread_group[i * 32 + lane];
      while (g0 < g1) {
        const int mid = (g0 + g1) / 2;
        unsigned n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) n += v[i] == lo && grp[i] <= mid;
        if (above + int(__reduce_add_sync(0xffffffffu, n)) >= k) g1 = mid;
        else g0 = mid + 1;
      }
      g = g0;
    }
  }
  if (lane == 0) {
    sh.bound = lo == none ? -INFINITY : __uint_as_float((lo >> 31) ? (lo & 0x7fffffffu) : ~lo);
    sh.bound_group = g;
  }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_rows_kernel(const LogprobArgs A, int blocks) {
  extern __shared__ __align__(16) unsigned char dyn[];
  T* group_max = reinterpret_cast<T*>(dyn);
  __shared__ LpShared sh;
  constexpr int kWords = Groups<T>::kWords;
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
  const int skew = int(reinterpret_cast<uintptr_t>(x) & 31) / int(sizeof(T));
  const int head = min(skew ? 32 / int(sizeof(T)) - skew : 0, A.vocab);
  const int all = (A.vocab - head) / kGroup;
  const int share = (all + blocks - 1) / blocks;
  const int g0 = min(rank * share, all), n = min(share, all - g0);
  const T* body = x + head + int64_t(g0) * kGroup;

  Sums acc{-INFINITY, 0.f, 0.f};
  float tmax = -INFINITY;
  int tgroup = 0xffff;
  bool bad = !usable_temperature(scale);
  const uint64_t scale2 = pack2(scale, scale), log2e2 = pack2(kLog2e, kLog2e);
  uint64_t s2 = 0, u2 = 0;
  auto fold = [&]() {
    const float2 a = unpack2(s2), b = unpack2(u2);
    acc.s += a.x + a.y;
    acc.u += b.x + b.y;
    s2 = u2 = 0;
  };
  auto group = [&](const uint32_t* v, int g) {
    const float m = Groups<T>::max(v);
    group_max[g] = Groups<T>::narrow(m);
    bad |= !(m < INFINITY);
    if (m > tmax) {
      tmax = m;
      tgroup = g;
    }
    const float z = m * scale;
    if (!(z > -INFINITY)) return;
    if (z > acc.ref + kRefSlack) {
      fold();
      acc.move_to(z);
    }
    const uint64_t ref2 = pack2(-acc.ref, -acc.ref);
    uint64_t ug = 0;
#pragma unroll
    for (int i = 0; i < kGroup / 2; ++i) {
      const float2 p = Groups<T>::get(v, i);
      const uint64_t d = fma2(pack2(p.x, p.y), scale2, ref2);
      const float2 t = unpack2(mul2(d, log2e2));
      const uint64_t e = pack2(exp2_approx(t.x), exp2_approx(t.y));
      s2 = add2(s2, e);
      ug = fma2(e, d, ug);
    }
    const float2 h = unpack2(ug);
    if (isnan(h.x + h.y)) {  // a logit at -inf, or so low that z is: 0 * -inf
      ug = 0;
#pragma unroll
      for (int i = 0; i < kGroup / 2; ++i) {
        const float2 p = Groups<T>::get(v, i);
        const float2 d = unpack2(fma2(pack2(p.x, p.y), scale2, ref2));
        const float dx = fmaxf(d.x, -1000.f), dy = fmaxf(d.y, -1000.f);  // e^-1000 is 0
        ug = fma2(pack2(exp2_approx(dx * kLog2e), exp2_approx(dy * kLog2e)), pack2(dx, dy), ug);
      }
    }
    u2 = add2(u2, ug);
  };
  constexpr int kBatch = kWords == 8 ? 4 : 2;  // groups in flight a thread
  int g = tid;
  for (; g + (kBatch - 1) * kLpThreads < n; g += kBatch * kLpThreads) {
    uint32_t v[kBatch][kWords];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const T* at = body + int64_t(g + b * kLpThreads) * kGroup;
#pragma unroll
      for (int q = 0; q < kWords; q += 8) load32(at + q * (kGroup / kWords), &v[b][q]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) group(v[b], g + b * kLpThreads);
  }
  for (; g < n; g += kLpThreads) {
    uint32_t v[kWords];
    const T* at = body + int64_t(g) * kGroup;
#pragma unroll
    for (int q = 0; q < kWords; q += 8) load32(at + q * (kGroup / kWords), &v[q]);
    group(v, g);
  }
  fold();
  // the edges: thread tid < kEdge of the first block takes one logit
  const int tail0 = head + all * kGroup;
  float edge = -INFINITY;
  int edge_id = -1;
  if (rank == 0 && tid < head) edge_id = tid;
  else if (rank == 0 && tid >= kEdge / 2 && tail0 + tid - kEdge / 2 < A.vocab && tid < kEdge) edge_id = tail0 + tid - kEdge / 2;
  if (edge_id >= 0) {
    edge = to_float(x[edge_id]);
    bad |= !(edge < INFINITY);
    const float z = edge * scale;
    if (z > -INFINITY && z < INFINITY) {
      if (z > acc.ref + kRefSlack) acc.move_to(z);
      const float d = fmaf(edge, scale, -acc.ref), e = exp2_approx(d * kLog2e);
      acc.s += e;
      acc.u += e > 0.f ? e * d : 0.f;
    }
  }

  // the block's maximum and sums
  float m = fmaxf(tmax, edge);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.wm[w] = m;
  sh.thread_max[tid] = tmax;
  sh.thread_group[tid] = uint16_t(tgroup);
  if (tid == 0) sh.num_listed = sh.num_cand = 0;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int i = 0; i < kLpWarps; ++i) m = fmaxf(m, sh.wm[i]);
  // the reference of the results: one rounded product, so that one fused
  // multiply-add gives z - zmax to half a step of the difference
  float zmax = m * scale;
  const bool sums = m > -INFINITY && !bad && fabsf(zmax) < INFINITY;
  Sums total{zmax, 0.f, 0.f};
  if (sums) {
    if (acc.ref > -INFINITY) {
      acc.move_to(zmax);
      total.add(acc);
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
  }
  if (A.top_k > 0 && w == 0) select_bound(sh, A.top_k);
  __syncthreads();
  total.s = total.u = 0.f;
  if (sums) {
#pragma unroll
    for (int i = 0; i < kLpWarps; ++i) {
      total.s += sh.ws[i];
      total.u += sh.wu[i];
    }
  }

  // the block's top k
  int found = 0;
  if (A.top_k > 0 && !bad) {
    const float bound = sh.bound;
    const int bound_group = sh.bound_group;
    auto reaches = [&](float v, int at) { return v > -INFINITY && (v > bound || (v == bound && at <= bound_group)); };
    if (reaches(tmax, tgroup)) {
      for (int at = tid; at < n; at += kLpThreads)
        if (reaches(to_float(group_max[at]), at)) sh.listed[atomicAdd(&sh.num_listed, 1)] = uint16_t(at);
    }
    if (edge > -INFINITY) sh.cand[atomicAdd(&sh.num_cand, 1)] = order_key(edge, uint32_t(edge_id));
    __syncthreads();
    int picked = sh.num_listed;
    const uint16_t* list = sh.listed;
    if (picked > kPicked) {  // few threads own many large groups: the first k by (maximum, group)
      for (int i = tid; i < picked; i += kLpThreads) {
        const uint64_t key = order_key(to_float(group_max[sh.listed[i]]), sh.listed[i]);
        int above = 0;
        for (int j = 0; j < picked; ++j) above += order_key(to_float(group_max[sh.listed[j]]), sh.listed[j]) > key;
        if (above < A.top_k) sh.picked[above] = sh.listed[i];
      }
      __syncthreads();
      picked = A.top_k;
      list = sh.picked;
    }
    for (int i = tid; i < picked * kGroup; i += kLpThreads) {
      const int id = head + (g0 + list[i / kGroup]) * kGroup + i % kGroup;
      const float v = to_float(x[id]);
      if (v >= bound && v > -INFINITY) sh.cand[atomicAdd(&sh.num_cand, 1)] = order_key(v, uint32_t(id));
    }
    __syncthreads();
    found = sh.num_cand;
  }
  LpShared* to = blocks > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
  if (blocks > 1) cluster.barrier_wait();  // the first block is there
  if (A.top_k > 0) {
    for (int i = tid; i < found; i += kLpThreads) {
      const uint64_t key = sh.cand[i];
      int above = 0;
      for (int j = 0; j < found; ++j) above += sh.cand[j] > key;
      if (above < A.top_k) to->part_key[rank][above] = key;
    }
    for (int i = found + tid; i < A.top_k; i += kLpThreads) to->part_key[rank][i] = 0;
  }
  if (tid == 0) {
    to->part_m[rank] = m;
    to->part_s[rank] = total.s;
    to->part_u[rank] = total.u;
    to->part_bad[rank] = bad;
    to->part_found[rank] = min(found, A.top_k);
  }
  if (blocks > 1) {
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // the row
  for (int i = 0; i < blocks; ++i) {
    m = fmaxf(m, sh.part_m[i]);
    bad |= sh.part_bad[i] != 0;
  }
  zmax = m * scale;
  bad |= m > -INFINITY && !(fabsf(zmax) < INFINITY);
  float log_s, entropy;
  if (bad) {
    log_s = entropy = zmax = NAN;
  } else if (m == -INFINITY) {
    log_s = -INFINITY;
    entropy = 0.f;
  } else {
    Sums row{zmax, 0.f, 0.f};
    for (int i = 0; i < blocks; ++i) {
      const float zi = sh.part_m[i] * scale;
      if (zi > -INFINITY) {
        Sums p{zi, sh.part_s[i], sh.part_u[i]};
        p.move_to(zmax);
        row.add(p);
      }
    }
    log_s = logf(row.s);
    entropy = log_s - row.u / row.s;
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
  // ranks over the blocks' sorted lists; keys of different logits differ
  for (int i = tid; i < A.top_k * blocks; i += kLpThreads) {
    const int b = i / A.top_k, k = i - b * A.top_k;
    const uint64_t key = bad ? 0 : sh.part_key[b][k];
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
    if (key != 0 && above < A.top_k) {
      A.top_tokens[above * A.num_rows + r] = int32_t(~uint32_t(key));
      A.top_logprobs[above * A.num_rows + r] = fmaf(key_logit(key), scale, -zmax) - log_s;
    }
  }
  if (A.top_k > 0) {
    int have = 0;  // logits above -inf among the lists; the ranks behind them have none
    for (int b = 0; b < blocks && !bad; ++b) have += sh.part_found[b];
    for (int k = have + tid; k < A.top_k; k += kLpThreads) {
      A.top_tokens[k * A.num_rows + r] = -1;
      A.top_logprobs[k * A.num_rows + r] = bad ? NAN : -INFINITY;
    }
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

// Blocks a row: enough to give every SM work, as long as each keeps a few
// groups a thread, and so many that a block's groups fit its shared memory.
int blocks_per_row(int64_t rows, int vocab) {
  const int groups = vocab / kGroup;
  int b = 1;
  while (b < kMaxCluster && (groups > b * kMaxGroups || (rows * b * 2 <= 304 && groups >= b * 2 * 128))) b *= 2;
  return b;
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs& A, cudaStream_t st) {
  if (A.num_rows > 0) {
    const int blocks = blocks_per_row(A.num_rows, A.vocab);
    const int share = (A.vocab / kGroup + blocks - 1) / blocks;
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
    if (sizeof(LpShared) + cfg.dynamicSmemBytes > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(logprob_rows_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 int(cfg.dynamicSmemBytes));
      if (e != cudaSuccess) return e;
    }
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
