// Page tables and slot maps of the paged latent pool, built on the GPU from
// request lengths: the buffers that the verify kernels take their offsets
// from ("The Final Solder Joint" -- "The Investigation" gives their types).
#include <cooperative_groups.h>
#include <stdint.h>

#include "mla_step_ops.h"
#include "mtv_internal.cuh"

namespace mtv {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ void set_err(uint32_t* err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

// Division by a host-known divisor d >= 1 of numerators below 2^31:
// floor(x / d) = x * ceil(2^(31+s) / d) >> (31 + s) with 2^s >= d, since the
// product is too large by less than 2^31 * 2^s / 2^(31+s) = 1 (in units of 1/d).
struct FastDiv {
  uint32_t d, mul, shift;
};

FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
  return FastDiv{d, uint32_t(m), 31 + s};
}

__device__ __forceinline__ uint32_t fast_div(uint32_t x, FastDiv f) {
  return uint32_t((uint64_t(x) * f.mul) >> f.shift);
}

// Inclusive sum over the block of one 64-bit value a thread, in thread order.
// part: shared, one entry a warp.  Ends with every thread past the last read.
template <int kThreads>
__device__ __forceinline__ uint64_t block_inclusive_sum(uint64_t v, uint64_t* part, uint64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) part[w] = v;
  __syncthreads();
  constexpr int kWarps = kThreads / 32;
  uint64_t s = lane < kWarps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  const uint64_t before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
  *total = __shfl_sync(0xffffffffu, s, kWarps - 1);
  __syncthreads();
  return v + (w > 0 ? before : 0);
}

// Largest r in [lo, hi) with off[r] <= x (off non-decreasing, off[lo] <= x).
__device__ __forceinline__ int find_row(const uint32_t* off, int lo, int hi, uint32_t x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Page tables.  Released entries are numbered x = 0 .. R-1 and new entries y =
// 0 .. G-1 in (row, entry) order; F pages are free.  The stack after all
// pushes holds released entry x at F + R - 1 - x, and new entry y takes the
// element at F + R - 1 - y: released entry y while y < R, else
// free_pages[F - 1 - (y - R)].  Released entries x >= G stay on the stack.  So
// every page moves once, reads and writes never meet (a row releases or grows,
// not both; stack reads lie below F, writes at or above), and only held and
// num_free are updated in place: one cluster does the call, every block scans
// all rows itself, and the two are written after the cluster's barrier.
// ---------------------------------------------------------------------------
constexpr int kPageThreads = 1024;

struct PageArgs {
  const int32_t* lens;
  int32_t* table;
  int32_t* held;
  int32_t* free_pages;
  int32_t* num_free;
  uint32_t* err;
  int64_t stride, free_capacity;
  int32_t num_rows, page_size, max_pages;
};

__global__ void __launch_bounds__(kPageThreads) page_table_kernel(const PageArgs A) {
  extern __shared__ uint32_t sm[];
  uint32_t* rel_off = sm;                          // [num_rows + 1]
  uint32_t* grow_off = rel_off + A.num_rows + 1;   // [num_rows + 1]
  uint32_t* base = grow_off + A.num_rows + 1;      // [num_rows]: min(need, held)
  __shared__ uint64_t part[kPageThreads / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), blocks = int(cluster.num_blocks());
  const int tid = threadIdx.x;
  const int64_t F = *A.num_free;
  const bool stack_ok = F >= 0 && F <= A.free_capacity;
  uint32_t bad = stack_ok ? 0 : MTV_DEVERR_PAGES;

  uint64_t carry = 0;  // released entries in the high half, new ones in the low half
  if (tid == 0) rel_off[0] = grow_off[0] = 0;
  for (int r0 = 0; r0 < A.num_rows; r0 += kPageThreads) {
    const int r = r0 + tid;
    uint32_t rel = 0, grow = 0;
    if (r < A.num_rows && stack_ok) {
      const int32_t len = A.lens[r], held = A.held[r];
      int32_t need = held;
      if (held < 0 || held > A.max_pages) bad |= MTV_DEVERR_PAGES;
      else if (len < -1) bad |= MTV_DEVERR_INDPTR;
      else if (len >= 0) {
        need = len == 0 ? 0 : (len - 1) / A.page_size + 1;
        if (need > A.max_pages) {
          bad |= MTV_DEVERR_PAGES;
          need = held;
        }
        rel = need < held ? uint32_t(held - need) : 0;
        grow = need > held ? uint32_t(need - held) : 0;
      }
      base[r] = uint32_t(min(need, held));
    }
    uint64_t total;
    const uint64_t incl = block_inclusive_sum<kPageThreads>((uint64_t(rel) << 32) | grow, part, &total) + carry;
    carry += total;
    if (r < A.num_rows) {
      rel_off[r + 1] = uint32_t(incl >> 32);
      grow_off[r + 1] = uint32_t(incl);
    }
  }
  __syncthreads();
  const int64_t R = int64_t(carry >> 32);
  // rows grow in order until one does not fit: G is the last sum within F + R
  int64_t G = int64_t(uint32_t(carry));
  if (G > F + R) {
    bad |= MTV_DEVERR_PAGES;
    G = grow_off[find_row(grow_off, 0, A.num_rows + 1, uint32_t(F + R))];
  }
  if (F + R - G > A.free_capacity) bad |= MTV_DEVERR_PAGES;

  if (stack_ok) {
    const int64_t step = int64_t(blocks) * kPageThreads;
    for (int64_t y = int64_t(rank) * kPageThreads + tid; y < G; y += step) {
      const int r = find_row(grow_off, 0, A.num_rows, uint32_t(y));
      int32_t page;
      if (y < R) {
        const int s = find_row(rel_off, 0, A.num_rows, uint32_t(y));
        page = A.table[s * A.stride + base[s] + (y - rel_off[s])];
      } else {
        page = A.free_pages[F - 1 - (y - R)];
      }
      A.table[r * A.stride + base[r] + (y - grow_off[r])] = page;
    }
    for (int64_t x = G + int64_t(rank) * kPageThreads + tid; x < R; x += step) {
      const int s = find_row(rel_off, 0, A.num_rows, uint32_t(x));
      const int64_t at = F + R - 1 - x;
      if (at < A.free_capacity) A.free_pages[at] = A.table[s * A.stride + base[s] + (x - rel_off[s])];
    }
  }
  cluster.sync();  // every block has read held, num_free and the released entries
  if (stack_ok) {
    for (int r = rank * kPageThreads + tid; r < A.num_rows; r += blocks * kPageThreads) {
      const uint32_t rel = rel_off[r + 1] - rel_off[r], grow = grow_off[r + 1] - grow_off[r];
      if (rel) A.held[r] = int32_t(base[r]);
      else if (grow && int64_t(grow_off[r + 1]) <= G) A.held[r] = int32_t(base[r] + grow);
    }
    if (rank == 0 && tid == 0) *A.num_free = int32_t(min(F + R - G, A.free_capacity));
  }
  if (rank == 0 && bad) set_err(A.err, bad);
}

// ---------------------------------------------------------------------------
// Slot maps.  Every block scans all request lengths into shared memory (a few
// KB out of L2), then takes its share of the prefix keys by output position
// and every gridDim-th request's tree.
// ---------------------------------------------------------------------------
constexpr int kMapThreads = 512;
constexpr uint32_t kMaxSum = 0x7fffffffu;

struct MapArgs {
  const int32_t* table;
  const int32_t* rows;
  const int32_t* prefix;
  const int32_t* tree;
  const int32_t* parents;
  int32_t* kv_indptr;
  int64_t* kv_indices;
  int64_t* qo_indptr;
  int64_t* out_cache_loc;
  int64_t* positions;
  uint32_t* err;
  int64_t stride, num_rows, max_pages, num_pages, kv_capacity, q_capacity;
  FastDiv page;
  int32_t bs;
};

// Slot of token j of the request in table row `row`; -1 (and the error bits)
// where the table has none.
__device__ __forceinline__ int64_t slot_of(const MapArgs& A, int64_t row, uint32_t j, uint32_t* bad) {
  const uint32_t pg = fast_div(j, A.page);
  if (row < 0 || row >= A.num_rows || int64_t(pg) >= A.max_pages) {
    *bad |= MTV_DEVERR_PAGES;
    return -1;
  }
  const int32_t id = A.table[row * A.stride + pg];
  if (id < 0 || int64_t(id) >= A.num_pages) {
    *bad |= MTV_DEVERR_PAGES;
    return -1;
  }
  return int64_t(id) * A.page.d + (j - pg * A.page.d);
}

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const MapArgs A) {
  extern __shared__ uint32_t sm[];
  uint32_t* kv_off = sm;                // [bs + 1]
  uint32_t* q_off = kv_off + A.bs + 1;  // [bs + 1]
  __shared__ uint64_t part[kMapThreads / 32];
  __shared__ int up[2][kMapThreads], dep[2][kMapThreads];
  const int tid = threadIdx.x;
  uint32_t bad = 0;

  uint64_t kv_carry = 0, q_carry = 0;
  if (tid == 0) kv_off[0] = q_off[0] = 0;
  for (int r0 = 0; r0 < A.bs; r0 += kMapThreads) {
    const int r = r0 + tid;
    int32_t p = 0, n = 0;
    if (r < A.bs) {
      p = A.prefix[r];
      n = A.tree ? A.tree[r] : 0;
      if (p < 0 || n < 0) bad |= MTV_DEVERR_INDPTR;
    }
    uint64_t total;
    const uint64_t a = block_inclusive_sum<kMapThreads>(uint64_t(max(p, 0)), part, &total) + kv_carry;
    kv_carry += total;
    const uint64_t b = block_inclusive_sum<kMapThreads>(uint64_t(max(n, 0)), part, &total) + q_carry;
    q_carry += total;
    if (r < A.bs) {
      kv_off[r + 1] = uint32_t(a < kMaxSum ? a : kMaxSum);
      q_off[r + 1] = uint32_t(b < kMaxSum ? b : kMaxSum);
    }
  }
  __syncthreads();
  if (kv_carry > kMaxSum || q_carry > kMaxSum) bad |= MTV_DEVERR_INDPTR;
  if (A.kv_indices && int64_t(kv_off[A.bs]) > A.kv_capacity) bad |= MTV_DEVERR_INDPTR;
  if ((A.out_cache_loc || A.positions) && int64_t(q_off[A.bs]) > A.q_capacity) bad |= MTV_DEVERR_INDPTR;
  if (blockIdx.x == 0) {
    for (int r = tid; r <= A.bs; r += kMapThreads) {
      A.kv_indptr[r] = int32_t(kv_off[r]);
      A.qo_indptr[r] = int64_t(q_off[r]);
    }
  }

  // trees: slots of their tokens, and positions from their depths
  if (A.out_cache_loc || A.positions) {
    for (int r = blockIdx.x; r < A.bs; r += gridDim.x) {
      const int64_t q0 = q_off[r];
      const int64_t n = min(int64_t(q_off[r + 1]), A.q_capacity) - q0;
      const uint32_t p = kv_off[r + 1] - kv_off[r];
      const int64_t row = A.rows ? A.rows[r] : r;
      for (int64_t t0 = 0; t0 < n; t0 += kMapThreads) {
        const int64_t t = t0 + tid;
        const bool live = t < n;
        if (live && A.out_cache_loc) {
          const int64_t j = int64_t(p) + t;
          if (j > kMaxSum) bad |= MTV_DEVERR_PAGES;
          A.out_cache_loc[q0 + t] = j > kMaxSum ? -1 : slot_of(A, row, uint32_t(j), &bad);
        }
        if (!A.positions) continue;
        if (!A.parents) {
          if (live) A.positions[q0 + t] = int64_t(p) + t;
          continue;
        }
        // Depth by doubling over this run of nodes: up = an ancestor inside
        // the run, dep = steps to it.  A parent in an earlier run has its
        // position written already.
        __syncthreads();
        int u = -1, d = 0;
        if (live) {
          int64_t par = A.parents[q0 + t];
          if (par < -1 || par >= t) {
            bad |= MTV_DEVERR_PARENT;
            par = -1;
          }
          if (par >= t0) {
            u = int(par - t0);
            d = 1;
          } else if (par >= 0) {
            d = int(A.positions[q0 + par] - p) + 1;
          }
        }
        int buf = 0;
        up[0][tid] = u;
        dep[0][tid] = d;
        while (__syncthreads_or(u >= 0)) {
          if (u >= 0) {
            d += dep[buf][u];
            u = up[buf][u];
          }
          up[buf ^ 1][tid] = u;
          dep[buf ^ 1][tid] = d;
          buf ^= 1;
        }
        if (live) A.positions[q0 + t] = int64_t(p) + d;
      }
    }
  }

  // prefix keys by output position
  if (A.kv_indices) {
    const int64_t total = min(int64_t(kv_off[A.bs]), A.kv_capacity);
    const int64_t step = int64_t(gridDim.x) * kMapThreads;
    for (int64_t y = int64_t(blockIdx.x) * kMapThreads + tid; y < total; y += step) {
      const int r = find_row(kv_off, 0, A.bs, uint32_t(y));
      const int64_t row = A.rows ? A.rows[r] : r;
      A.kv_indices[y] = slot_of(A, row, uint32_t(y) - kv_off[r], &bad);
    }
  }
  if (bad) set_err(A.err, bad);
}

// Dynamic shared memory above 48 KB has to be allowed for a kernel first.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;  // static arrays come on top
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

int launch_code(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}

}  // namespace
}  // namespace mtv

extern "C" int mla_page_table_update(const int32_t* lens, int num_rows, int page_size, int32_t* page_table,
                                     int64_t table_stride, int64_t max_pages, int32_t* held, int32_t* free_pages,
                                     int64_t free_capacity, int32_t* num_free, uint32_t* err, void* stream) {
  using namespace mtv;
  if (num_rows < 0 || page_size < 1 || max_pages < 0 || table_stride < max_pages || free_capacity < 0 ||
      free_capacity > INT32_MAX)
    return MTV_E_BAD_ARGUMENT;
  if (num_rows > MTV_MAX_REQUESTS) return MTV_E_UNSUPPORTED;
  if (num_rows > 0 && max_pages > INT32_MAX / num_rows) return MTV_E_UNSUPPORTED;
  if (num_rows == 0) return MTV_OK;
  if (!lens || !held || !num_free || (!page_table && max_pages > 0) || (!free_pages && free_capacity > 0))
    return MTV_E_NULL_POINTER;
  const PageArgs A{lens,  page_table,   held,          free_pages, num_free,  err,
                   table_stride, free_capacity, num_rows,   page_size, int32_t(max_pages)};
  const size_t smem = (3 * size_t(num_rows) + 2) * 4;
  cudaError_t e = allow_smem(page_table_kernel, smem);
  if (e != cudaSuccess) return launch_code(e);
  const unsigned blocks = int64_t(num_rows) * max_pages > 8192 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kPageThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {blocks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_code(cudaLaunchKernelEx(&cfg, page_table_kernel, A));
}

extern "C" int mla_slot_map_build(const int32_t* page_table, int64_t table_stride, int64_t num_rows,
                                  int64_t max_pages, int64_t num_pages, int page_size, const int32_t* rows,
                                  const int32_t* prefix_lens, const int32_t* tree_sizes, const int32_t* parents,
                                  int bs, int32_t* kv_indptr, int64_t* kv_indices, int64_t kv_capacity,
                                  int64_t* qo_indptr, int64_t* out_cache_loc, int64_t* positions,
                                  int64_t q_capacity, uint32_t* err, void* stream) {
  using namespace mtv;
  if (bs < 0 || page_size < 1 || table_stride < 0 || num_rows < 0 || max_pages < 0 || num_pages < 0 ||
      kv_capacity < 0 || q_capacity < 0 || (table_stride < max_pages && num_rows > 1))
    return MTV_E_BAD_ARGUMENT;
  if (bs > MTV_MAX_REQUESTS) return MTV_E_UNSUPPORTED;
  if (!kv_indptr || !qo_indptr || (bs > 0 && !prefix_lens) || (!page_table && num_rows > 0 && max_pages > 0))
    return MTV_E_NULL_POINTER;
  const MapArgs A{page_table, rows,         prefix_lens, tree_sizes, parents,   kv_indptr, kv_indices,
                  qo_indptr,  out_cache_loc, positions,   err,        table_stride, num_rows,  max_pages,
                  num_pages,  kv_capacity,   q_capacity,  make_fast_div(uint32_t(page_size)), bs};
  const size_t smem = 2 * (size_t(bs) + 1) * 4;
  cudaError_t e = allow_smem(slot_map_kernel, smem);
  if (e != cudaSuccess) return launch_code(e);
  int64_t blocks = kv_indices ? (kv_capacity + kMapThreads - 1) / kMapThreads : 0;
  if (blocks < bs) blocks = bs;
  if (blocks > 608) blocks = 608;
  if (blocks < 1) blocks = 1;
  slot_map_kernel<<<unsigned(blocks), kMapThreads, smem, static_cast<cudaStream_t>(stream)>>>(A);
  return launch_code(cudaSuccess);
}
