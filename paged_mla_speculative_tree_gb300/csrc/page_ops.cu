// Page tables and slot maps of the paged latent pool, built on the GPU from
// request lengths: the buffers that the verify kernels take their offsets
// from ("The Final Solder Joint" -- "The Investigation" gives their types).
#include <stdint.h>

#include <type_traits>

#include "mla_step_ops.h"
#include "mtv_internal.cuh"

namespace mtv {
namespace {

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

__device__ __forceinline__ void set_err(uint32_t* err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

// Division by a host-known divisor d of numerators below 2^31: with 2^s >= d,
// s >= 1, floor(x / d) = x * ceil(2^(31+s) / d) >> (31 + s), since the product
// is too large by less than 2^31 * 2^s / 2^(31+s) = 1 (in units of 1/d); the
// high word of the product, shifted by s - 1.  mul == 0 stands for d == 1.
struct FastDiv {
  uint32_t d, mul, shift;
};

FastDiv make_fast_div(uint32_t d) {
  if (d == 1) return FastDiv{1, 0, 0};
  uint32_t s = 1;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
  return FastDiv{d, uint32_t(m), s - 1};
}

__device__ __forceinline__ uint32_t fast_div(uint32_t x, FastDiv f) {
  return f.mul ? __umulhi(x, f.mul) >> f.shift : x;
}

// Inclusive sums over the block of one or two 64-bit values a thread, in
// thread order.  part: shared, an entry a warp for each.  Ends with every
// thread past the last read.
template <int kThreads>
__device__ __forceinline__ void block_inclusive_sum(uint64_t* a, uint64_t* b, uint64_t* part, uint64_t* a_total,
                                                    uint64_t* b_total) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto warp_sum = [&](uint64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  *a = warp_sum(*a);
  if (lane == 31) part[w] = *a;
  if (b) {
    *b = warp_sum(*b);
    if (lane == 31) part[kWarps + w] = *b;
  }
  __syncthreads();
  auto before = [&](const uint64_t* p, uint64_t* total) {
    const uint64_t s = warp_sum(lane < kWarps ? p[lane] : 0);
    *total = __shfl_sync(0xffffffffu, s, kWarps - 1);
    const uint64_t left = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
    return w > 0 ? left : 0;
  };
  *a += before(part, a_total);
  if (b) *b += before(part + kWarps, b_total);
  __syncthreads();
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
// num_free are updated in place: every block scans all rows itself, and the
// two are written at the end -- by the one block of a small table, or by one
// more block behind a grid, its programmatic dependent, whose own scan is done
// by the time the grid is.  (One cluster of 16 blocks with its barrier in
// place of the second launch took 33 us where the grid takes 10, for 1 M pages
// in and out.)
// ---------------------------------------------------------------------------
constexpr int kPageThreads = 512;
constexpr int kRun = 512;     // entries (runs of 32 throughout: 34 us in place of 10.5 for 1 M pages in and out)
constexpr int kFewRows = 4;   // of a run that is copied row by row (every entry searched: 14.6 us)
constexpr int kSearches = 4;  // entries a lane has in flight otherwise
constexpr int64_t kPageBlocks = 152;  // of the grid: one an SM
// Tables that one block does, for one launch in place of two.  Measured on one
// table of 256 rows (5,888 entries), up and back: 12 us against 15 called from
// Python, which is why; 8.9 against 7.9 in a graph, where the grid would win.
constexpr int64_t kBlockEntries = 1 << 14;

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

enum PageMode {
  kAll,    // one block does the call
  kMoves,  // a grid moves the pages ...
  kState,  // ... and one block behind it writes held and num_free
};

template <int kMode> __global__ void __launch_bounds__(kPageThreads) page_table_kernel(const PageArgs A) {
  extern __shared__ uint32_t sm[];
  uint32_t* rel_off = sm;                          // [num_rows + 1]
  uint32_t* grow_off = rel_off + A.num_rows + 1;   // [num_rows + 1]
  uint32_t* base = grow_off + A.num_rows + 1;      // [num_rows]: min(need, held)
  __shared__ uint64_t part[kPageThreads / 32];
  const int tid = threadIdx.x;
  if (kMode == kMoves) grid_launch_dependents();
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
    uint64_t incl = (uint64_t(rel) << 32) | grow, total;
    block_inclusive_sum<kPageThreads>(&incl, nullptr, part, &total, nullptr);
    incl += carry;
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

  if (kMode != kState && stack_ok) {
    // A warp moves runs of 32 or 512 entries.  A run inside a few rows, with
    // all its pages from the stack (or to it), is copied row by row with up to
    // 16 loads a lane in flight; any other one searches each entry's row.
    const int lane = tid & 31;
    const int64_t warp = int64_t(blockIdx.x) * (kPageThreads / 32) + (tid >> 5);
    const int64_t warps = int64_t(gridDim.x) * (kPageThreads / 32);
    auto copy = [&](int32_t* to, int to_step, const int32_t* from, int from_step, int64_t lo, int64_t hi) {
      for (int64_t z0 = lo; z0 < hi; z0 += kRun) {  // to[to_step * z] = from[from_step * z]
        int32_t page[kRun / 32];
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) {
          const int64_t z = z0 + i * 32 + lane;
          if (z < hi) page[i] = from[from_step * z];
        }
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) {
          const int64_t z = z0 + i * 32 + lane;
          if (z < hi) to[to_step * z] = page[i];
        }
      }
    };
    const int64_t grow_run = G > warps * 64 ? kRun : 32, rel_run = R - G > warps * 64 ? kRun : 32;
    for (int64_t y0 = warp * grow_run; y0 < G; y0 += warps * grow_run) {
      const int64_t y1 = min(y0 + grow_run, G);
      int r0 = 0, r1 = A.num_rows - 1;
      if (grow_run == kRun) {
        r0 = find_row(grow_off, 0, A.num_rows, uint32_t(y0));
        r1 = find_row(grow_off, r0, A.num_rows, uint32_t(y1 - 1));
      }
      if (grow_run == kRun && y0 >= R && r1 - r0 < kFewRows) {
        for (int r = r0; r <= r1; ++r)
          copy(A.table + r * A.stride + (int64_t(base[r]) - grow_off[r]), 1, A.free_pages + (F - 1 + R), -1,
               max(y0, int64_t(grow_off[r])), min(y1, int64_t(grow_off[r + 1])));
        continue;
      }
      for (int64_t y = y0 + lane; y < y1; y += 32 * kSearches) {
        const int32_t* from[kSearches];
        int32_t* to[kSearches];
        int32_t page[kSearches];
#pragma unroll
        for (int i = 0; i < kSearches; ++i) {
          const uint32_t z = uint32_t(y) + i * 32;
          from[i] = nullptr;
          if (z < y1) {
            const int r = find_row(grow_off, r0, r1 + 1, z);
            to[i] = A.table + r * A.stride + base[r] + (z - grow_off[r]);
            if (z < R) {
              const int s = find_row(rel_off, 0, A.num_rows, z);
              from[i] = A.table + s * A.stride + base[s] + (z - rel_off[s]);
            } else {
              from[i] = A.free_pages + (F - 1 - (z - R));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kSearches; ++i)
          if (from[i]) page[i] = *from[i];
#pragma unroll
        for (int i = 0; i < kSearches; ++i)
          if (from[i]) *to[i] = page[i];
      }
    }
    const int64_t top = F + R - 1;  // released entry x goes to top - x
    for (int64_t x0 = G + warp * rel_run; x0 < R; x0 += warps * rel_run) {
      const int64_t x1 = min(x0 + rel_run, R);
      int s0 = 0, s1 = A.num_rows - 1;
      if (rel_run == kRun) {
        s0 = find_row(rel_off, 0, A.num_rows, uint32_t(x0));
        s1 = find_row(rel_off, s0, A.num_rows, uint32_t(x1 - 1));
      }
      const int64_t lo = max(x0, top - A.free_capacity + 1);  // (those before it would pass the capacity)
      if (rel_run == kRun && s1 - s0 < kFewRows) {
        for (int s = s0; s <= s1; ++s)
          copy(A.free_pages + top, -1, A.table + s * A.stride + (int64_t(base[s]) - rel_off[s]), 1,
               max(lo, int64_t(rel_off[s])), min(x1, int64_t(rel_off[s + 1])));
        continue;
      }
      for (int64_t x = x0 + lane; x < x1; x += 32 * kSearches) {
        int32_t page[kSearches];
#pragma unroll
        for (int i = 0; i < kSearches; ++i) {
          const uint32_t z = uint32_t(x) + i * 32;
          if (z >= lo && z < x1) {
            const int s = find_row(rel_off, s0, s1 + 1, z);
            page[i] = A.table[s * A.stride + base[s] + (z - rel_off[s])];
          }
        }
#pragma unroll
        for (int i = 0; i < kSearches; ++i) {
          const uint32_t z = uint32_t(x) + i * 32;
          if (z >= lo && z < x1) A.free_pages[top - z] = page[i];
        }
      }
    }
  }
  if (kMode == kMoves) return;
  // every thread or block of the moves has read held and num_free
  if (kMode == kAll) __syncthreads();
  else grid_dependency_wait();
  if (stack_ok) {
    for (int r = tid; r < A.num_rows; r += kPageThreads) {  // (one block is left)
      const uint32_t rel = rel_off[r + 1] - rel_off[r], grow = grow_off[r + 1] - grow_off[r];
      if (rel) A.held[r] = int32_t(base[r]);
      else if (grow && int64_t(grow_off[r + 1]) <= G) A.held[r] = int32_t(base[r] + grow);
    }
    if (tid == 0) *A.num_free = int32_t(min(F + R - G, A.free_capacity));
  }
  if (bad) set_err(A.err, bad);
}

// ---------------------------------------------------------------------------
// Slot maps.  Every block scans all request lengths into shared memory (a few
// KB out of L2), then takes its share of the prefix keys by output position
// and every gridDim-th request's tree.  Bound by the 8 bytes stored a key:
// 256 x (131,072 + 64) in pages of 64 takes 47.5 us (5.7 TB/s, of which 4 us
// are scan and trees; bare stores in this order take 41 to 43), 4 x (5,760 +
// 16) takes 3.9 us of launch, scan and depths.
// ---------------------------------------------------------------------------
constexpr int kMapThreads = 256;
constexpr int kPairs = 4;        // keys a lane searches at a time
constexpr int kUnroll = 4;       // steps with their loads in flight together
constexpr int kMaxSteps = 32;    // of 64 keys, in a run
// Requests of a run that is written request by request (192 ragged ones: 8.8 us;
// every key of a run across requests searched: 11.2; all keys searched: 13.4,
// and 84 in place of 47 us for 256 long ones).
constexpr int kFewRequests = 4;
constexpr int kMapBlocks = 608;  // four on each of 152 SMs
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

// A lane's pairs of keys in steps of 64 keys a warp, from token j on: slots of
// tokens j + 64 i and the next one.  kInside: both always lie in one page.
// Returns whether an entry was no page (its slots are then wrong).
template <bool kInside>
__device__ __forceinline__ bool write_steps(longlong2* out, const int32_t* pages, uint32_t j, int steps, FastDiv page,
                                            uint32_t limit) {
  const int32_t d = int32_t(page.d);
  bool none = false;
  auto batch = [&](auto count) {
    constexpr int kCount = decltype(count)::value;
    uint32_t at[kCount];
    int32_t id[kCount], next[kCount];
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
      at[u] = fast_div(j + u * 64, page);
      id[u] = __ldg(pages + at[u]);
      // the second key may start the next page
      if (!kInside) next[u] = j + u * 64 + 1 == (at[u] + 1) * page.d ? __ldg(pages + at[u] + 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
      none |= uint32_t(id[u]) >= limit;
      const int64_t x = int64_t(id[u] - int32_t(at[u])) * d + (j + u * 64);  // id d + j mod d
      int64_t y = x + 1;
      if (!kInside && j + u * 64 + 1 == (at[u] + 1) * page.d) {
        none |= uint32_t(next[u]) >= limit;
        y = int64_t(next[u]) * d;
      }
      out[u * 32] = make_longlong2(x, y);
    }
    out += kCount * 32;
    j += kCount * 64;
  };
  int i = 0;
#pragma unroll 1
  for (; i + kUnroll <= steps; i += kUnroll) batch(std::integral_constant<int, kUnroll>());
#pragma unroll 1
  for (; i < steps; ++i) batch(std::integral_constant<int, 1>());
  return none;
}

__global__ void __launch_bounds__(kMapThreads, 4) slot_map_kernel(const MapArgs A) {
  extern __shared__ uint32_t sm[];
  uint32_t* kv_off = sm;                // [bs + 1]
  uint32_t* q_off = kv_off + A.bs + 1;  // [bs + 1]
  int32_t* row_of = reinterpret_cast<int32_t*>(q_off + A.bs + 1);  // [bs]
  __shared__ uint64_t part[2 * kMapThreads / 32];
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
      row_of[r] = A.rows ? A.rows[r] : r;
      if (p < 0 || n < 0) bad |= MTV_DEVERR_INDPTR;
    }
    uint64_t a = uint64_t(max(p, 0)), b = uint64_t(max(n, 0)), a_total, b_total;
    block_inclusive_sum<kMapThreads>(&a, &b, part, &a_total, &b_total);
    a += kv_carry;
    b += q_carry;
    kv_carry += a_total;
    q_carry += b_total;
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
    // (the last blocks first: the prefix keys' remainder falls to the first ones)
    for (int r = gridDim.x - 1 - blockIdx.x; r < A.bs; r += gridDim.x) {
      const int64_t q0 = q_off[r];
      const int64_t n = min(int64_t(q_off[r + 1]), A.q_capacity) - q0;
      // (sums that are held have lost the prefix's length, and with a shorter one
      // the tree's slots would be those of cached tokens)
      const uint32_t p = kv_carry > kMaxSum ? uint32_t(max(A.prefix[r], 0)) : kv_off[r + 1] - kv_off[r];
      const int64_t row = row_of[r];
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

  // Prefix keys by output position: a warp writes runs of 64 to 2048 keys.
  // A run inside a few requests goes request by request, its row and pages
  // checked as a whole, in steps of two neighbouring keys a lane (16 bytes);
  // any other one (of many short requests) searches each key's request.
  if (A.kv_indices) {
    const int lane = tid & 31;
    const int64_t total = min(int64_t(kv_off[A.bs]), A.kv_capacity);
    const uint32_t limit = uint32_t(min(A.num_pages, int64_t(1) << 31));  // of an entry; negative ones wrap past it
    // runs short enough to give every warp one, of 64 to 2048 keys
    const int run = 64 * int(min(max(total / (64 * int64_t(gridDim.x) * (kMapThreads / 32)), int64_t(1)), int64_t(kMaxSteps)));
    const int64_t step = int64_t(gridDim.x) * (kMapThreads / 32) * run;
    for (int64_t y0 = (int64_t(blockIdx.x) * (kMapThreads / 32) + (tid >> 5)) * run; y0 < total; y0 += step) {
      const int64_t y1 = min(y0 + run, total);
      const int r0 = find_row(kv_off, 0, A.bs, uint32_t(y0));
      const int r1 = find_row(kv_off, r0, A.bs, uint32_t(y1 - 1));
      if (r1 - r0 >= kFewRequests) {
        for (int64_t y = y0 + lane; y < y1; y += 32 * kPairs) {
          int64_t slot[kPairs];
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const int64_t z = y + i * 32;
            if (z < y1) {
              const int r = find_row(kv_off, r0, r1 + 1, uint32_t(z));
              slot[i] = slot_of(A, row_of[r], uint32_t(z) - kv_off[r], &bad);
            }
          }
#pragma unroll
          for (int i = 0; i < kPairs; ++i)
            if (y + i * 32 < y1) A.kv_indices[y + i * 32] = slot[i];
        }
        continue;
      }
      for (int r = r0; r <= r1; ++r) {
        const int64_t lo = max(y0, int64_t(kv_off[r])), hi = min(y1, int64_t(kv_off[r + 1]));
        if (lo >= hi) continue;
        const int64_t row = row_of[r];
        const uint32_t j0 = uint32_t(lo) - kv_off[r], keys = uint32_t(hi - lo);  // tokens [j0, j0 + keys)
        if (row < 0 || row >= A.num_rows || int64_t(fast_div(j0 + keys - 1, A.page)) >= A.max_pages) {
          for (int64_t y = lo + lane; y < hi; y += 32)
            A.kv_indices[y] = slot_of(A, row, uint32_t(y) - kv_off[r], &bad);
          continue;
        }
        const int32_t* pages = A.table + row * A.stride;
        int64_t* to = A.kv_indices + lo;
        const int count = int(keys), shift = int(reinterpret_cast<uintptr_t>(to) >> 3) & 1;
        const int whole = (count - shift) / 64;  // steps of 64 keys on 16-byte boundaries
        const uint32_t d = A.page.d;
        auto one = [&](int k) { to[k] = slot_of(A, row, j0 + uint32_t(k), &bad); };
        longlong2* out = reinterpret_cast<longlong2*>(to + shift) + lane;
        const uint32_t j = j0 + uint32_t(shift) + 2 * lane;
        bool none = false;  // an entry that is no page
        if (d % 2 == 0 && (j0 + uint32_t(shift)) % 2 == 0)
          none = write_steps<true>(out, pages, j, whole, A.page, limit);
        else
          none = write_steps<false>(out, pages, j, whole, A.page, limit);
        if (__any_sync(0xffffffffu, none)) {
          __syncwarp();  // other lanes have stored to these addresses: a vote orders no memory
          for (int k = lane; k < count; k += 32) one(k);
        } else {
          if (shift && lane == 0) one(0);
          for (int k = shift + whole * 64 + lane; k < count; k += 32) one(k);
        }
      }
    }
  }
  if (bad) set_err(A.err, bad);
}

// Dynamic shared memory above 48 KB has to be allowed for a kernel first.  The
// limit belongs to the process and not to the call, so it is the one that the
// largest call needs: a call's own bytes would lower it for another host
// thread's call, or for a graph that is still to be instantiated.
constexpr size_t step_smem(size_t requests) { return (3 * requests + 2) * 4; }

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;  // static arrays come on top
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(step_smem(MTV_MAX_REQUESTS)));
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
  const size_t smem = step_smem(size_t(num_rows));
  const int64_t entries = int64_t(num_rows) * max_pages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (entries <= kBlockEntries) {
    const cudaError_t e = allow_smem(page_table_kernel<kAll>, smem);
    if (e != cudaSuccess) return launch_code(e);
    page_table_kernel<kAll><<<1, kPageThreads, smem, st>>>(A);
    return launch_code(cudaSuccess);
  }
  cudaError_t e = allow_smem(page_table_kernel<kMoves>, smem);
  if (e == cudaSuccess) e = allow_smem(page_table_kernel<kState>, smem);
  if (e != cudaSuccess) return launch_code(e);
  const int64_t blocks = (entries + kPageThreads - 1) / kPageThreads;
  page_table_kernel<kMoves><<<unsigned(blocks < kPageBlocks ? blocks : kPageBlocks), kPageThreads, smem, st>>>(A);
  e = cudaGetLastError();
  if (e != cudaSuccess) return launch_code(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPageThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_code(cudaLaunchKernelEx(&cfg, page_table_kernel<kState>, A));
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
  const size_t smem = step_smem(size_t(bs));
  cudaError_t e = allow_smem(slot_map_kernel, smem);
  if (e != cudaSuccess) return launch_code(e);
  int64_t blocks = kv_indices ? (kv_capacity + 64 * (kMapThreads / 32) - 1) / (64 * (kMapThreads / 32)) : 0;
  if (blocks < bs) blocks = bs;
  if (blocks > kMapBlocks) blocks = kMapBlocks;
  if (blocks < 1) blocks = 1;
  slot_map_kernel<<<unsigned(blocks), kMapThreads, smem, static_cast<cudaStream_t>(stream)>>>(A);
  return launch_code(cudaSuccess);
}
