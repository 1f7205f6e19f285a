// One matrix product a head: the absorption of queries into the latent space,
// the values of latent outputs and the expansion of latents to every head's
// keys and values (the latent form: "The Glue That Binds" -- "The Broader
// Engineering Effort").
//
// head_product_kernel.  A unit is 128 tokens x nt outputs of one head; a block
// takes a run of units, of which those of one (head, nt outputs) follow each
// other, so that their weights (all of k, at most 128 KB) are loaded once and
// stay in shared memory while the tokens stream through a ring of slots of
// 128 tokens x 64 k.  Roles: one warp issues the copies, one the MMAs, four
// take the sums (two TMEM buffers) through shared memory to bulk stores.  What
// lies outside a tensor reads as zero and is not stored, so odd sizes need no
// code of their own.
//
// Weights dense in k are a K-major operand (chunks of 64 k x nt rows), weights
// dense in n an MN-major one (blocks of 64 n x 64 k).
//
// What bounds it (one GB300, 64 heads; replays of one graph, which find part of their
// bytes in L2): the bytes where each head has rows of its own (1,024 tokens: queries
// to the latent space 14.6 us, latent outputs to values 13.9, floors 13.8, but 18.7 for
// the first called on and on over changing inputs; 4,000 tokens 70 and 57, floors 50,
// but the first writes 262 MB, which a plain fill does in 68); for few tokens the chain
// launch -> copies -> sums -> stores (8 tokens to the latent space 4.2 us, 1.3 of
// bytes; 64 to values 4.9, 2.0 of bytes); for one latent expanded to all heads the
// copies of x under way beside 128 KB of weights, each value of which meets 128
// outputs (8,191 tokens to 64 x 256: 104 us, 115 over changing inputs), so that many
// tokens go to pairs of SMs (head_product_pair_kernel: 88 us, 1,560 TFLOP/s, and 103;
// one library product of that shape 85 to 87).  Without pairs, sharing x between two
// blocks by multicast changed nothing (it is a block's own ring that binds, not L2);
// two chunks a wait (+ 10 %) and eight warps for the sums (+ 5 %) were slower.  Copies
// and MMAs are issued under warp-uniform branches by an elected thread: by lane 0
// of a divergent one they took two to four times as long (186 us).
//
// Every wait is bounded: one that gives up sets MTV_DEVERR_TIMEOUT and a flag
// that ends the block's other waits; copies and MMAs in flight are waited for
// (bounded too) before TMEM is freed.
#include <stdint.h>

#include <type_traits>

#include "mla_layer_ops.h"
#include "launch.cuh"
#include "mtv_internal.cuh"
#include "pipeline.cuh"
#include "tc_ptx.cuh"
#include "tma.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

using namespace ptx;

struct ProductArgs {
  const void* x;
  const void* w;
  void* out;
  uint32_t* err;
  int64_t x_tok, x_head, w_head, w_k, w_n, out_tok, out_head, tokens;
  int heads, k_dim, n_dim, give_up;
};

constexpr int kRows = 128, kChunk = 64;   // tokens a unit, k a chunk
constexpr int kMaxChunks = MTV_MAX_HEAD_DIM / kChunk, kMaxSlots = 8;
constexpr uint32_t kXSlot = kRows * kChunk * 2, kMaxWeights = 131072;
constexpr uint32_t kBlockBytes = 32 * 128;  // staged output: 32 rows x 64 columns
constexpr int kThreads = 192;
enum : int {
  B_XFULL = 0, B_XEMPTY = B_XFULL + kMaxSlots, B_WFULL = B_XEMPTY + kMaxSlots, B_WFREE = B_WFULL + kMaxChunks,
  B_ACC, B_ACCFREE = B_ACC + 2, B_FIN = B_ACCFREE + 2, B_COUNT
};
constexpr uint32_t kOffCtl = 8 * B_COUNT, kOffData = 1024;
static_assert(kOffCtl + sizeof(Ctl) <= kOffData, "barriers");

struct TensorArgs {
  CUtensorMap x, w, out;
  uint32_t* err;
  int give_up;             // tests: see init_ctl
  int64_t units, tokens;   // units: heads * n_tiles * m_tiles
  uint32_t x_bytes;        // of a chunk of x: 64 k of 128 tokens, or of as many as there are
  int m_tiles, n_tiles, nt, chunks, slots;
  int gx, gw, gw_log;      // chunks a copy of x (and a slot of the ring) and of w (dense in k) has: 1, 2 or 4
  int x_whole, w_whole;    // the maps are cut into chunks of 64
  int w_k_major, x_by_head, w_by_head, out_by_head, n_dim;
};

// A block's units in order: 128 tokens after 128 tokens of one (head, nt outputs),
// then the next such group.  Counted on, since 64-bit divisions by every role and
// chunk took longer than the chunk's products (8,191 tokens expanded: 186 us).
struct Units {
  int64_t left;
  int h, n, t;  // head, outputs' tile, tokens' tile
  bool fresh;   // the first of its group in this block
  __device__ __forceinline__ Units(int64_t first, int64_t last, const TensorArgs& A) : left(last - first) {
    const int64_t g = first / A.m_tiles;
    t = int(first % A.m_tiles), h = int(g / A.n_tiles), n = int(g % A.n_tiles);
    fresh = true;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ bool changes(const TensorArgs& A) const { return left > 1 && t + 1 == A.m_tiles; }
  __device__ __forceinline__ void next(const TensorArgs& A) {
    --left;
    fresh = ++t == A.m_tiles;
    if (!fresh) return;
    t = 0;
    if (++n == A.n_tiles) n = 0, ++h;
  }
};

// kFew: at most one tile of tokens, whose copies bring several chunks each.
// kTest: waits that give up for a test.
template <typename T, bool kFew, bool kTest>
__global__ void __launch_bounds__(kThreads, 1) head_product_kernel(const __grid_constant__ TensorArgs A) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (base - raw) + kOffCtl);
  auto bar = [&](int i) { return base + 8u * uint32_t(i); };
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const uint32_t w_chunk = uint32_t(A.nt) * 128u;
  const int gx = kFew ? A.gx : 1, gw = kFew ? A.gw : 1;
  const uint32_t x_chunk = kFew ? A.x_bytes : kXSlot, x_slot = uint32_t(gx) * x_chunk;
  const uint32_t off_x = kOffData + uint32_t(A.chunks) * w_chunk;
  const uint32_t off_out = off_x + uint32_t(A.slots) * x_slot + (kXSlot - x_chunk);  // the MMAs read 128 rows of the last chunk
  const int64_t first = A.units * blockIdx.x / gridDim.x, last = A.units * (blockIdx.x + 1) / gridDim.x;
  const uint32_t cols = A.nt <= 64 ? 128u : 2u * uint32_t(A.nt);

  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i == B_ACCFREE || i == B_ACCFREE + 1 ? 4 : 1);
    init_ctl<kTest>(ctl, A.give_up);
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem), cols);
    tmem_relinquish();
  }
  launched_after();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    int slot = 0, items = 0, loads = 0, asked = 0;  // loads of weights, and chunks of the last one
    uint32_t phase = 1;                             // of the slots' releases: the first round waits for none
    const uint32_t data = uniform(base);
    auto released = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for_call<kTest>(bar(b), parity, ctl, A.err)) != 0;
    };
    bool ok = true;
    for (Units u(first, last, A); u.more() && ok; u.next(A)) {
      const int xh = A.x_by_head ? u.h : 0, wh = A.w_by_head ? u.h : 0, n0 = u.n * A.nt, t0 = u.t * kRows;
      for (int c = 0; c < A.chunks && ok; ++c) {
        if ((c & (gx - 1)) == 0) {
          if (items >= A.slots) ok = released(B_XEMPTY + slot, phase);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t full = data + 8 * (B_XFULL + slot);
            mbar_arrive_expect_tx(full, x_slot);
            const uint32_t dst = data + off_x + slot * x_slot;
            if constexpr (kFew) tma_load_4d(dst, &A.x, A.x_whole ? 0 : c * kChunk, xh, t0, A.x_whole ? c : 0, full);
            else tma_load_3d(dst, &A.x, c * kChunk, xh, t0, full);
          }
          items = items < A.slots ? items + 1 : items;
          if (++slot == A.slots) slot = 0, phase ^= 1;
        }
        if (!u.fresh || (c & (gw - 1)) != 0) continue;
        if (c == 0) {
          if (loads > 0) ok = released(B_WFREE, uint32_t(loads - 1) & 1);
          if (!ok) break;
          ++loads, asked = 0;
        }
        ++asked;
        if (elect_one()) {
          const uint32_t dst = data + kOffData + c * w_chunk, full = data + 8 * (B_WFULL + (kFew ? c >> A.gw_log : c));
          mbar_arrive_expect_tx(full, uint32_t(gw) * w_chunk);
          if constexpr (kFew) {
            if (A.w_k_major) tma_load_4d(dst, &A.w, A.w_whole ? 0 : c * kChunk, wh, n0, A.w_whole ? c : 0, full);
            else if (A.w_whole) tma_load_4d(dst, &A.w, 0, wh, c * kChunk, n0 / 64, full);
            else for (int b = 0; b < A.nt; b += 64) tma_load_4d(dst + b * 128, &A.w, n0 + b, wh, c * kChunk, 0, full);
          } else {
            if (A.w_k_major) tma_load_3d(dst, &A.w, c * kChunk, wh, n0, full);
            else for (int b = 0; b < A.nt; b += 64) tma_load_3d(dst + b * 128, &A.w, n0 + b, wh, c * kChunk, full);
          }
        }
      }
    }
    // what was asked for lands before the block ends, read or not: the last items, slot by slot backwards
    if (elect_one()) {
      const long long since = clock64();
      for (int i = 0; i < items; ++i) {
        if (--slot < 0) slot = A.slots - 1, phase ^= 1;
        drain(bar(B_XFULL + slot), phase ^ 1, since, A.err);
      }
      for (int c = 0; c < asked; ++c) drain(bar(B_WFULL + c), uint32_t(loads - 1) & 1, since, A.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    const uint32_t id = std::is_same<T, __nv_bfloat16>::value ? idesc_bf16_f32(kRows, A.nt, 0, A.w_k_major ? 0 : 1)
                                                              : idesc_fp16_f32(kRows, A.nt, 0, A.w_k_major ? 0 : 1);
    const uint32_t w_step = A.w_k_major ? 32u : 2048u, acc = uniform(tmem), data = uniform(base);
    auto arrived = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for_call<kTest>(bar(b), parity, ctl, A.err)) != 0;
    };
    int slot = 0, loads = 0, n = 0;
    uint32_t phase = 0;  // of the ring's slots
    bool ok = true;
    for (Units u(first, last, A); u.more() && ok; u.next(A), ++n) {
      if (u.fresh) ++loads;
      const int buf = n & 1;
      if (n >= 2) ok = arrived(B_ACCFREE + buf, uint32_t(n / 2 - 1) & 1);
      int in = 0;  // chunk of the slot
      for (int c = 0; c < A.chunks && ok; ++c) {
        if (u.fresh && (!kFew || (c & (gw - 1)) == 0)) ok = arrived(B_WFULL + (kFew ? c >> A.gw_log : c), uint32_t(loads - 1) & 1);
        if (ok && (!kFew || in == 0)) ok = arrived(B_XFULL + slot, phase);
        if (!ok) break;
        tc_fence_after();
        const bool done = !kFew || in + 1 == gx || c + 1 == A.chunks;  // with the slot
        if (elect_one()) {
          const uint64_t a = smem_desc(data + off_x + slot * x_slot + (kFew ? in * x_chunk : 0), 16, 1024, kSwizzle128B);
          const uint64_t b = smem_desc(data + kOffData + c * w_chunk, A.w_k_major ? 16 : 8192, 1024, kSwizzle128B);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(acc + uint32_t(A.nt) * buf, desc_add(a, 32 * k), desc_add(b, w_step * k), id, c + k > 0);
          if (done) mma_commit(bar(B_XEMPTY + slot));
        }
        in = done ? 0 : in + 1;
        if (done && ++slot == A.slots) slot = 0, phase ^= 1;
      }
      if (!ok) break;
      if (elect_one()) {
        mma_commit(bar(B_ACC + buf));
        if (u.changes(A)) mma_commit(bar(B_WFREE));
      }
    }
    if (elect_one()) {
      mma_commit(bar(B_FIN));  // every MMA issued has run once this arrives
      drain(bar(B_FIN), 0, clock64(), A.err);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- sums to memory
    const int q = warp & 3;  // TMEM lane quarter
    const int blocks = A.nt > 128 ? 2 : 1;  // staged a warp
    const uint32_t stage = base + off_out + uint32_t(q * blocks) * kBlockBytes;
    int n = 0, block = 0;
    for (Units u(first, last, A); u.more(); u.next(A), ++n) {
      const int h = u.h, n0 = u.n * A.nt, buf = n & 1;
      const int64_t t0 = int64_t(u.t) * kRows + q * 32;
      const bool ok = wait_for_call<kTest>(bar(B_ACC + buf), uint32_t(n / 2) & 1, ctl, A.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int width = t0 < A.tokens ? min(A.nt, A.n_dim - n0) : 0;  // a store starts inside the tensor, which clips it
      for (int b = 0; b < width; b += 64, block ^= blocks - 1) {
        const uint32_t to = stage + uint32_t(block) * kBlockBytes;
        uint32_t y[64];
        tmem_ld64_sync(tmem + (uint32_t(q * 32) << 16) + uint32_t(A.nt) * buf + b, y);
        if (lane == 0) {  // the last store from this block has read it
          if (blocks > 1) bulk_wait_group_read<1>();
          else bulk_wait_group_read<0>();
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(y[e + i]);
          const uint4 v = pack<T>(f);
          st_shared_v4(to + lane * 128 + (((e / 8) ^ (lane & 7)) << 4), v.x, v.y, v.z, v.w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&A.out, n0 + b, A.out_by_head ? h : 0, int(t0), to);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_ACCFREE + buf));
    }
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
}

// Many tokens and k up to 512: a pair of SMs a unit of 256 tokens x 256 outputs, whose
// products meet 256 outputs with every value of x that an SM takes in (the form above:
// 128), so that the tensor cores are the bound.  Each CTA copies its 128 tokens and its
// 128 outputs' weights, all completing on the even CTA's barriers; that CTA issues the
// MMAs, whose commits arrive on both CTAs' barriers; each CTA stores its tokens' sums.
constexpr int kPairTokens = 2 * kRows, kPairN = 256, kPairChunks = 8;
constexpr uint32_t kPairW = 128 * kChunk * 2, kPairColumns = 512;

template <typename T, bool kTest>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) head_product_pair_kernel(const __grid_constant__ TensorArgs A) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (base - raw) + kOffCtl);
  auto bar = [&](int i) { return base + 8u * uint32_t(i); };
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const int rank = int(cluster_ctarank());
  const uint32_t off_x = kOffData + uint32_t(A.chunks) * kPairW, off_out = off_x + uint32_t(A.slots) * kXSlot;
  const int64_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int64_t first = A.units * pair / pairs, last = A.units * (pair + 1) / pairs;

  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i == B_ACCFREE || i == B_ACCFREE + 1 ? 8 : 1);
    init_ctl<kTest>(ctl, A.give_up, mapa(smem_u32(const_cast<int*>(&ctl->abort)), rank ^ 1));
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl->tmem), kPairColumns);
    tmem_relinquish_pair();
  }
  launched_after();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    int slot = 0, x_asked = 0, w_asked = 0;  // chunks
    uint32_t phase = 1, w_phase = 1;
    const uint32_t data = uniform(base), lead = uniform(mapa(base, 0));  // its barriers take both CTAs' copies
    auto released = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for_call<kTest>(bar(b), parity, ctl, A.err)) != 0;
    };
    bool ok = true;
    for (Units u(first, last, A); u.more() && ok; u.next(A)) {
      const int xh = A.x_by_head ? u.h : 0, wh = A.w_by_head ? u.h : 0;
      const int n0 = u.n * kPairN + rank * 128, t0 = u.t * kPairTokens + rank * kRows;
      for (int c = 0; c < A.chunks && ok; ++c) {
        if (x_asked >= A.slots) ok = released(B_XEMPTY + slot, phase);
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(data + 8 * (B_XFULL + slot), 2 * kXSlot);
          tma_load_3d_pair(data + off_x + slot * kXSlot, &A.x, c * kChunk, xh, t0, lead + 8 * (B_XFULL + slot));
        }
        ++x_asked;
        if (++slot == A.slots) slot = 0, phase ^= 1;
        if (!u.fresh) continue;
        if (c == 0) {
          if (w_asked > 0) ok = released(B_WFREE, w_phase);
          if (!ok) break;
          w_phase ^= 1;
        }
        if (elect_one()) {
          const uint32_t dst = data + kOffData + c * kPairW, full = lead + 8 * (B_WFULL + c);
          if (rank == 0) mbar_arrive_expect_tx(data + 8 * (B_WFULL + c), 2 * kPairW);
          if (A.w_k_major) tma_load_3d_pair(dst, &A.w, c * kChunk, wh, n0, full);
          else for (int b = 0; b < 128; b += 64) tma_load_3d_pair(dst + b * 128, &A.w, n0 + b, wh, c * kChunk, full);
        }
        ++w_asked;
      }
    }
    if (elect_one()) {
      const uint32_t to = mapa(smem_u32(&ctl->asked[2 * rank]), 0);
      st_cluster_u32(to, uint32_t(x_asked));
      st_cluster_u32(to + 4, uint32_t(w_asked));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    if (rank == 0) {
      const uint32_t id = std::is_same<T, __nv_bfloat16>::value ? idesc_bf16_f32(kPairTokens, kPairN, 0, A.w_k_major ? 0 : 1)
                                                                : idesc_fp16_f32(kPairTokens, kPairN, 0, A.w_k_major ? 0 : 1);
      const uint32_t w_step = A.w_k_major ? 32u : 2048u, acc = uniform(tmem), data = uniform(base);
      auto arrived = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for_call<kTest>(bar(b), parity, ctl, A.err)) != 0;
      };
      int slot = 0, loads = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (Units u(first, last, A); u.more() && ok; u.next(A), ++n) {
        if (u.fresh) ++loads;
        const int buf = n & 1;
        if (n >= 2) ok = __all_sync(0xffffffffu, wait_for_peer<kTest>(bar(B_ACCFREE + buf), uint32_t(n / 2 - 1) & 1, ctl, A.err)) != 0;
        for (int c = 0; c < A.chunks && ok; ++c) {
          if (u.fresh) ok = arrived(B_WFULL + c, uint32_t(loads - 1) & 1);
          if (ok) ok = arrived(B_XFULL + slot, phase);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = smem_desc(data + off_x + slot * kXSlot, 16, 1024, kSwizzle128B);
            const uint64_t b = smem_desc(data + kOffData + c * kPairW, A.w_k_major ? 16 : 8192, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_pair(acc + uint32_t(kPairN) * buf, desc_add(a, 32 * k), desc_add(b, w_step * k), id, c + k > 0);
            mma_commit_pair(bar(B_XEMPTY + slot));
          }
          if (++slot == A.slots) slot = 0, phase ^= 1;
        }
        if (!ok) break;
        if (elect_one()) {
          mma_commit_pair(bar(B_ACC + buf));
          if (u.changes(A)) mma_commit_pair(bar(B_WFREE));
        }
      }
      if (elect_one()) mma_commit_pair(bar(B_FIN));
    }
    if (elect_one()) drain(bar(B_FIN), 0, clock64(), A.err);  // the last of the commits that arrive here
    __syncwarp();
  } else {
    // ------------------------------------------------------------- sums to memory
    const int q = warp & 3;
    const uint32_t stage = base + off_out + uint32_t(q) * kBlockBytes;
    const uint32_t freed = mapa(bar(B_ACCFREE), 0);
    int n = 0;
    for (Units u(first, last, A); u.more(); u.next(A), ++n) {
      const int n0 = u.n * kPairN, buf = n & 1;
      const int64_t t0 = int64_t(u.t) * kPairTokens + rank * kRows + q * 32;
      const bool ok = wait_for_call<kTest>(bar(B_ACC + buf), uint32_t(n / 2) & 1, ctl, A.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int width = t0 < A.tokens ? min(kPairN, A.n_dim - n0) : 0;
      for (int b = 0; b < width; b += 64) {
        uint32_t y[64];
        tmem_ld64_sync(tmem + (uint32_t(q * 32) << 16) + uint32_t(kPairN) * buf + b, y);
        if (lane == 0) bulk_wait_group_read<0>();  // the last store has read the block
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(y[e + i]);
          const uint4 v = pack<T>(f);
          st_shared_v4(stage + lane * 128 + (((e / 8) ^ (lane & 7)) << 4), v.x, v.y, v.z, v.w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&A.out, n0 + b, A.out_by_head ? u.h : 0, int(t0), stage);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(freed + 8 * buf);
    }
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no product reads, and no commit writes, the other CTA's memory any more; no copy will be asked for
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kPairColumns);
  // After a wait that gave up, what either CTA asked for lands before one of them ends (else the products have taken
  // it all).  One may have asked for more than the other, by a ring at most, since a slot's release takes both sides'
  // copies: chunk i then has its barrier's open phase to itself, and the bytes that nobody asked for are made up or
  // not expected.
  if (ctl->abort && rank == 0 && warp == 0 && elect_one()) {
    const long long since = clock64();
    auto settle = [&](int full, int mine, int theirs, int ring, uint32_t bytes) {
      const int all = max(mine, theirs);
      for (int i = min(mine, theirs); i < all; ++i) {
        if (i < mine) mbar_complete_tx(bar(full + i % ring), bytes);
        else mbar_arrive_expect_tx(bar(full + i % ring), bytes);
      }
      for (int i = max(0, all - ring); i < all; ++i) drain(bar(full + i % ring), uint32_t(i / ring) & 1, since, A.err);
    };
    settle(B_XFULL, ctl->asked[0], ctl->asked[2], A.slots, kXSlot);
    settle(B_WFULL, ctl->asked[1], ctl->asked[3], A.chunks, kPairW);
  }
  __syncwarp();
  cluster_sync();
}

int sm_count() {
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms < 1)
    sms = 1;
  return sms;
}

// Whether tensor maps take the layout: 16-byte addresses and strides, w dense in k or n, and
// whole 16 bytes of outputs (a bulk store writes what is left of its last 16 bytes as zeros).
bool tensor_form(const ProductArgs& A) {
  if (A.n_dim % 8 != 0) return false;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(A.x) | reinterpret_cast<uintptr_t>(A.w) | reinterpret_cast<uintptr_t>(A.out);
  if (bits & 15) return false;
  const bool k_major = A.w_k == 1, n_major = A.w_n == 1;
  if (!k_major && !n_major) return false;
  const int64_t w_row = k_major ? A.w_n : A.w_k;
  const int64_t rows[] = {A.tokens, A.tokens, k_major ? A.n_dim : A.k_dim}, row[] = {A.x_tok, A.out_tok, w_row};
  for (int i = 0; i < 3; ++i)
    if (rows[i] > 1 && (!mappable_stride(row[i]) || row[i] == 0)) return false;
  if (A.heads > 1 && (!mappable_stride(A.x_head) || !mappable_stride(A.w_head) || !mappable_stride(A.out_head) || A.out_head == 0))
    return false;
  return tensor_map_encoder() != nullptr;
}

template <typename T> cudaError_t launch_tensor(const ProductArgs& A, cudaStream_t st) {
  TensorArgs P = {};
  const int sms = sm_count();
  P.chunks = (A.k_dim + kChunk - 1) / kChunk;
  P.m_tiles = int((A.tokens + kRows - 1) / kRows);
  // the narrowest tile that still gives every unit an SM of its own (20 heads: one token to the latent space
  // 4.1 us with 128, 4.6 with 256), else the widest whose weights fit, which reads x least often (1,024
  // tokens, 64 heads: 14.8 us with 256, 16.9 with 128)
  P.nt = 0;
  for (int nt = 64; nt <= 256; nt *= 2) {
    if (nt > 64 && (uint32_t(P.chunks) * nt * 128u > kMaxWeights || nt >= 2 * A.n_dim)) break;
    P.nt = nt;
    if (int64_t(A.heads) * ((A.n_dim + nt - 1) / nt) * P.m_tiles <= sms) break;
  }
  P.n_tiles = (A.n_dim + P.nt - 1) / P.nt;
  P.units = int64_t(A.heads) * P.n_tiles * P.m_tiles;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  // Pairs of SMs where the weights of 256 outputs do not fit one and fill two (n_dim 320 would leave a quarter of
  // the products empty: 4,000 tokens 64 us, not 55), where tokens do too (but for a ninth), from five units a pair on (8,191 tokens expanded to 64 x 256:
  // 104 -> 87 us; 4,000 with rows for each head 105 -> 74; 1,400, 5 units: 24 and 24; 800, 3 units: 16 and 18).
  const int pair_m = int((A.tokens + kPairTokens - 1) / kPairTokens), pair_n = (A.n_dim + kPairN - 1) / kPairN;
  const int64_t pair_units = int64_t(A.heads) * pair_n * pair_m, pairs = sms / 2;
  const bool pair = P.chunks > kPairChunks / 2 && P.chunks <= kPairChunks && (A.n_dim + 127) / 128 == 2 * pair_n &&
                    16 * pair_m <= 9 * P.m_tiles && pairs > 0 && pair_units >= 5 * pairs;
  if (pair) P.m_tiles = pair_m, P.n_tiles = pair_n, P.nt = kPairN, P.units = pair_units;
  P.w_k_major = A.w_k == 1;
  // A copy costs its issue (about 150 cycles) and its box, inside the tensor or not.  So one tile of tokens
  // takes several chunks of weights and of x with a copy, x in boxes as low as it is (what a slot holds below
  // such a box makes sums that nobody stores): values of 64 tokens 6.3 -> 5.3 us.  Many tokens stream chunk by
  // chunk, which keeps more copies under way (8,191 tokens expanded without pairs: 104 us, with the other form 142).
  const bool few = !pair && P.m_tiles == 1;
  const int x_rows = few ? int(A.tokens + 7) / 8 * 8 : kRows;
  P.x_bytes = uint32_t(x_rows) * kChunk * 2;
  P.x_whole = few && A.k_dim % kChunk == 0, P.w_whole = few && (P.w_k_major ? A.k_dim : A.n_dim) % 64 == 0;
  const int most = P.chunks % 4 == 0 ? 4 : P.chunks % 2 == 0 ? 2 : 1;
  P.gw = P.w_k_major && P.w_whole ? most : 1, P.gw_log = P.gw / 2;
  P.gx = P.x_whole ? most : 1;
  const uint32_t fixed = 1024 + kOffData + uint32_t(P.chunks) * P.nt * 128u + 4 * (P.nt > 128 ? 2 : 1) * kBlockBytes +
                         (kXSlot - P.x_bytes);
  while (P.gx > 1 && fixed + 2 * P.gx * P.x_bytes > 227u * 1024u) P.gx /= 2;
  P.slots = int((227u * 1024u - fixed) / (P.gx * P.x_bytes));
  if (P.slots > kMaxSlots) P.slots = kMaxSlots;
  const uint32_t smem = fixed + P.slots * P.gx * P.x_bytes;
  uint32_t pair_smem = 0;
  if (pair) {  // one staged block a warp: a slot more of x is worth more (87 us; four slots 89, three 97)
    const uint32_t pair_fixed = 1024 + kOffData + uint32_t(P.chunks) * kPairW + 4 * kBlockBytes;
    P.slots = int((227u * 1024u - pair_fixed) / kXSlot);
    if (P.slots > kMaxSlots) P.slots = kMaxSlots;
    pair_smem = pair_fixed + P.slots * kXSlot;
  }
  P.x_by_head = A.x_head != 0, P.w_by_head = A.w_head != 0, P.out_by_head = 1;
  if (A.heads == 1) P.x_by_head = P.w_by_head = P.out_by_head = 0;
  P.err = A.err, P.give_up = A.give_up, P.tokens = A.tokens, P.n_dim = A.n_dim;
  // weights: rows, their stride, their length, and the rows of a box
  const int64_t w_rows = P.w_k_major ? A.n_dim : A.k_dim, w_row = P.w_k_major ? A.w_n : A.w_k;
  const int w_dim = P.w_k_major ? A.k_dim : A.n_dim, w_box = P.w_k_major ? (pair ? 128 : P.nt) : 64;
  const bool maps =
      (few ? encode_chunked_map(&P.x, bf16, A.x, A.tokens, A.x_tok, A.heads, A.x_head, A.k_dim, P.x_whole, x_rows, P.gx) &&
                 encode_chunked_map(&P.w, bf16, A.w, w_rows, w_row, A.heads, A.w_head, w_dim, P.w_whole, w_box,
                                    P.w_k_major ? P.gw : P.nt / 64)
           : encode_heads_map(&P.x, bf16, A.x, A.tokens, A.x_tok, A.heads, A.x_head, A.k_dim, 64, kRows) &&
                 encode_heads_map(&P.w, bf16, A.w, w_rows, w_row, A.heads, A.w_head, w_dim, 64, w_box)) &&
      encode_heads_map(&P.out, bf16, A.out, A.tokens, A.out_tok, A.heads, A.out_head, A.n_dim, 64, 32);
  if (!maps) return cudaErrorInvalidValue;
  if (pair) {
    auto kernel = A.give_up ? head_product_pair_kernel<T, true> : head_product_pair_kernel<T, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3(2 * unsigned(pairs)), kThreads, pair_smem, st, P);
  }
  auto kernel = A.give_up ? (few ? head_product_kernel<T, true, true> : head_product_kernel<T, false, true>)
                          : (few ? head_product_kernel<T, true, false> : head_product_kernel<T, false, false>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(P.units < sms ? P.units : sms);
  return launch_early(kernel, dim3(grid), kThreads, smem, st, P);
}

// The plain form, for any strides: a block a tile of 64 tokens x 64 outputs of
// one head, 16 k at a time through shared memory, 4 x 4 sums a thread.  What it costs
// a caller whose rows are not in whole 16 bytes (64 heads): 8 tokens to the latent
// space 31 us, 64 to values 74, 1,024 to the latent space 355 (the tensor core: 4, 5, 15).
constexpr int kTile = 64, kSum = 16;

template <typename T>
__global__ void __launch_bounds__(256) head_product_plain_kernel(const ProductArgs A) {
  __shared__ float xs[kSum][kTile + 1], ws[kSum][kTile + 1];
  const int h = blockIdx.y, n0 = blockIdx.z * kTile, tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kTile;
  const T* x = static_cast<const T*>(A.x) + int64_t(h) * A.x_head;
  const T* w = static_cast<const T*>(A.w) + int64_t(h) * A.w_head;
  const int tx = tid % 16, ty = tid / 16;
  float sum[4][4] = {};
  for (int k0 = 0; k0 < A.k_dim; k0 += kSum) {
    for (int i = tid; i < kSum * kTile; i += 256) {
      const int k = i % kSum, t = i / kSum;
      xs[k][t] = (k0 + k < A.k_dim && t0 + t < A.tokens) ? to_float(x[(t0 + t) * A.x_tok + k0 + k]) : 0.f;
    }
    for (int i = tid; i < kSum * kTile; i += 256) {
      const int n = i % kTile, k = i / kTile;
      ws[k][n] = (k0 + k < A.k_dim && n0 + n < A.n_dim) ? to_float(w[(k0 + k) * A.w_k + (n0 + n) * A.w_n]) : 0.f;
    }
    __syncthreads();
    // values of k past the end are zero on both sides
#pragma unroll
    for (int k = 0; k < kSum; ++k)
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
                                int k_dim, int n_dim, int dtype, uint32_t* err, void* stream) {
  using namespace mtv;
  const int give_up = take_give_up(&dtype);
  if (num_tokens < 0 || num_tokens > INT32_MAX || num_heads < 0 || num_heads > MTV_MAX_HEADS || k_dim < 1 ||
      k_dim > MTV_MAX_HEAD_DIM || n_dim < 1 || n_dim > MTV_MAX_HEAD_DIM ||
      (dtype != MTV_DTYPE_BF16 && dtype != MTV_DTYPE_FP16))
    return MTV_E_BAD_ARGUMENT;
  if (num_tokens == 0 || num_heads == 0) return MTV_OK;
  if (!x || !w || !out) return MTV_E_NULL_POINTER;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(out)) & 1)
    return MTV_E_BAD_ARGUMENT;
  const ProductArgs A{x, w, out, err, x_tok_stride, x_head_stride, w_head_stride, w_k_stride, w_n_stride, out_tok_stride,
                      out_head_stride, num_tokens, num_heads, k_dim, n_dim, give_up};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MTV_DTYPE_BF16;
  cudaError_t e;
  if (tensor_form(A)) e = bf16 ? launch_tensor<__nv_bfloat16>(A, st) : launch_tensor<__half>(A, st);
  else e = bf16 ? launch_plain<__nv_bfloat16>(A, st) : launch_plain<__half>(A, st);
  if (e != cudaSuccess) cudaGetLastError();  // or a later launch reports it
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
