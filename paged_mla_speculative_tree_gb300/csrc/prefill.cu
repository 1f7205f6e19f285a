// Causal attention of new tokens over keys and values expanded from latents
// (head parts of 128 + 64 and 128): the form for prompts, where every query
// row has many neighbours.
//
// prefill_kernel.  A block owns 256 query rows of one head (two stages of 128)
// and walks the request's keys in tiles of 128, one pass with the running
// maximum and sum of a softmax:
//   S = Q K^T      12 k-steps of 16, both operands in shared memory, S in TMEM
//   P = 2^(S c - m c) in the input type, over S's columns in TMEM
//   O += P V       8 k-steps, P from TMEM, V as an MN-major operand
// Roles: a warp a stage issues the MMAs, one the TMA copies, and four warps a
// stage the softmax, a thread a row.  While one stage's softmax works, the tensor
// core computes the other's O += P V and next S; the stages take turns at it (see
// there).  MMAs of one thread run in order: S(j+1) may overwrite P(j) without a
// wait, and S(j+1) being there says that O holds everything up to j.
//
// Shared memory: Q 96 KB and a ring of eight 16 KB slots that K (three slots of
// 64 dims a tile) and V (two of 64 keys) pass through in the order of their
// use: K(0) V(0) K(1) V(1) ...  A copy has half of a tile's time (about 1,300 of
// 2,600 cycles at full rate) from its slot's release to its use; whole tiles of
// K and V do not fit twice beside Q.
// TMEM: S0, S1, O0, O1 of 128 columns each.
//
// The maximum that scores refer to moves only when a row's scores grow by more
// than 2^8 past it, so O is rarely rescaled.  P is rounded to the input type, which
// the tensor core takes; sums of weights stay in fp32: one of the weights, for the lse,
// and one of the rounded ones, by which O is divided, so that their rounding cancels
// in what the values have in common instead of scaling the output (up to half a step
// more: 300 equal values of 2 less a step came out a step too low).  The second sum is
// taken while the tensor core has the weights, with adds that read them as they are
// (8,192 tokens 780 -> 783 us, 2 x (1,000 after 5,760) 312 -> 317, the ragged fp16
// batch 168 -> 172, a prompt of 256 7.6 -> 8.1; unpacked first: 848, 328, 183, 8.5).
// fp16 weights are held 2^7 times as large, P = 2^(S c - m c + 7), at most 2^15: a
// weight is then off by 2^-32 of the row's largest at most.  Without that a long tail
// of keys below 2^-25 counted in the sum and not in O (one key 2^25.1 above 131,072
// others: outputs off by 240 of fp16's half steps in the median, now by 5, what fp32
// sums of that length leave).
//
// What bounds it (one GB300, 64 heads): the tensor core, for long prompts.  8,192
// tokens in one piece take 0.78 ms in short replays, 1,760 TFLOP/s of what the causal
// mask leaves (91 % of the measured bf16 rate), and 0.88 called on and on (1,570, 90 %
// of what the power cap leaves one library product); a pair of tiles 2,800 cycles of
// 2,600, a block 9,000 more for its first copies and its output.  What each step gave
// there, in short replays:
// MMAs and copies issued under warp-uniform branches by an elected thread (their
// operands stay in uniform registers) 1.41 -> 1.04 ms; a warp a stage for the MMAs
// -> 0.90; no spills in the softmax -> 0.87; turns -> 0.80; K's first slot filled
// before V's release -> 0.78.  Dropped: blocks that take the next one's number and
// start its copies early (more registers: 0.85 ms), 64 columns a softmax thread
// (0.95), P of both stages' rows in step (0.91).
//
// Every wait is bounded: one that gives up sets MTV_DEVERR_TIMEOUT and a flag
// that ends the block's other waits; copies and MMAs in flight are waited for
// (bounded too) before TMEM is freed.
//
// With few query rows the keys are split over blocks, and so are those of the last
// blocks where they would leave most SMs idle: each writes its normalised part and
// its lse, and combine_kernel joins them (60 rows over 32,768 keys of 8 heads: 31 us,
// 21 of them the keys' way from memory).  Letting both stages take the rows of such a
// block and its tiles in turn was no faster.  Few blocks of unsplit keys have 128
// rows, one stage, where 256 would leave half of the SMs idle.
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "mla_layer_ops.h"
#include "mtv_internal.cuh"
#include "launch.cuh"
#include "pipeline.cuh"
#include "tc_ptx.cuh"
#include "tma.cuh"
#include "vec_io.cuh"

namespace mtv {
namespace {

using namespace ptx;

constexpr int kNope = 128, kRope = 64, kQK = kNope + kRope, kV = 128;
constexpr int kStageRows = 128, kBlockRows = 2 * kStageRows, kKeys = 128;
constexpr int kThreads = 352;  // 4 + 4 softmax warps, 2 for the MMAs, 1 for the copies
constexpr uint32_t kSlot = 16384;
constexpr int kSlots = 8;
constexpr uint32_t kQStage = 3 * kSlot, kOffRing = 2 * kQStage, kOffBars = kOffRing + kSlots * kSlot;
// K and V tile j use the barriers j & 1; both stages release every tile
enum : int {
  B_Q = 0, B_KFULL = 2, B_VFULL = 4, B_KFREE = 6, B_VFREE = 8, B_S = 10, B_P = 12, B_O = 16, B_FIN = 18, B_TURN = 20, B_COUNT = 22
};
constexpr uint32_t kOffCtl = kOffBars + 8 * B_COUNT;
constexpr uint32_t kSmem = kOffCtl + sizeof(Ctl) + 1024;  // + slack for 1 KB alignment
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemS = 0, kTmemO = 256;
constexpr float kRescaleLog2 = 8.f;
// the reference's own weight, and its logarithm
template <typename T> constexpr float kWeight = std::is_same<T, __half>::value ? 128.f : 1.f;
template <typename T> constexpr float kWeightLog2 = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr int kSplitLast = MTV_PREFILL_SPLIT_LAST, kTailWaves = 8;

struct PrefillArgs {
  CUtensorMap q, k_nope, k_rope, v;
  void* out;
  float* lse;
  float* part;      // [nsplit, part_rows, 128], then the lse [nsplit, part_rows]
  const int64_t* qo_indptr;
  const int32_t* kv_indptr;
  uint32_t* err;
  int64_t o_tok, o_head, num_q, num_kv, max_q, max_kv, part_rows;
  float scale;
  int heads, causal, q_blocks;
  int give_up;       // tests: see init_ctl
  int block_rows;    // 256, or 128: the second stage idle
  int nsplit, last;  // the last blocks, whose keys are split
  unsigned whole;    // the blocks before them
  int by_block;      // rows of parts: 256 a split block; else num_q * heads
  int q_by_head, k_by_head, v_by_head;  // 0: one map for all heads
};

struct PrefillReq {
  int q0, k0, n, len;
};

// What block b of bs x heads x q_blocks works on: blocks of a head side by side, the longest first.
struct PrefillBlock {
  int r, h, row0;
  __device__ __forceinline__ PrefillBlock(const PrefillArgs& A, unsigned b) {
    row0 = (A.q_blocks - 1 - int(b % unsigned(A.q_blocks))) * A.block_rows;
    b /= unsigned(A.q_blocks);
    h = int(b % unsigned(A.heads)), r = int(b / unsigned(A.heads));
  }
};

// The request's rows, checked against the buffers and the bounds; n = 0 where
// they do not hold.
__device__ __forceinline__ PrefillReq load_prefill_req(const PrefillArgs& A, int r, bool report) {
  const int64_t q0 = A.qo_indptr[r], q1 = A.qo_indptr[r + 1], k0 = A.kv_indptr[r], k1 = A.kv_indptr[r + 1];
  PrefillReq R{int(q0), int(k0), int(q1 - q0), int(k1 - k0)};
  if (q0 < 0 || q1 < q0 || q1 > A.num_q || k0 < 0 || k1 < k0 || k1 > A.num_kv || q1 - q0 > A.max_q || k1 - k0 > A.max_kv) {
    if (report && A.err) atomicOr(A.err, MTV_DEVERR_INDPTR);
    R.n = R.len = 0;
  }
  return R;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds the two values of a packed pair to a and b, in fp32.
__device__ __forceinline__ void add_halves(uint32_t v, float& a, float& b, __nv_bfloat16) {
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n add.rn.f32.bf16 %0, x, %0;\n add.rn.f32.bf16 %1, y, %1;\n}"
      : "+f"(a), "+f"(b)
      : "r"(v));
}
__device__ __forceinline__ void add_halves(uint32_t v, float& a, float& b, __half) {
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n add.rn.f32.f16 %0, x, %0;\n add.rn.f32.f16 %1, y, %1;\n}"
      : "+f"(a), "+f"(b)
      : "r"(v));
}

// kTest: waits that give up for a test.
template <typename T, bool kTest>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs A) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (base - raw) + kOffCtl);
  auto bar = [&](int i) { return base + kOffBars + 8u * uint32_t(i); };
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;

  // blocks of all their keys, then the others' first parts, second parts, ...
  const bool split_keys = blockIdx.x >= A.whole && A.nsplit > 1;
  const unsigned tail = split_keys ? (blockIdx.x - A.whole) % unsigned(A.last) : 0u;
  const int split = split_keys ? int((blockIdx.x - A.whole) / unsigned(A.last)) : 0;
  const PrefillBlock B(A, split_keys ? A.whole + tail : blockIdx.x);
  const int row0 = B.row0, h = B.h;
  // the set-up needs nothing from memory
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i >= B_KFREE && i < B_S ? 2 : i >= B_P && i < B_O ? 4 : 1);
    init_ctl<kTest>(ctl, A.give_up);
    fence_mbar_init_cluster();
  }
  if (warp == 10 && lane == 0) {
    prefetch_map(&A.q);
    prefetch_map(&A.k_nope);
    prefetch_map(&A.k_rope);
    prefetch_map(&A.v);
  }
  launched_after();
  const PrefillReq R = load_prefill_req(A, B.r, tid == 0);
  if (row0 >= R.n) return;

  // key tiles of both stages: up to the last key that a stage's last row sees
  const int shift = R.len - R.n;  // query i sees keys up to shift + i
  auto tiles_of = [&](int s) -> int {
    const int first = row0 + s * kStageRows;
    if (first >= R.n || s * kStageRows >= A.block_rows) return 0;
    const int last = min(R.n, first + kStageRows) - 1;
    const int keys = A.causal ? max(0, min(R.len, shift + last + 1)) : R.len;
    return (keys + kKeys - 1) / kKeys;
  };
  const int tiles0 = tiles_of(0), tiles1 = tiles_of(1);
  const int parts = split_keys ? A.nsplit : 1, each = (max(tiles0, tiles1) + parts - 1) / parts, begin = split * each;
  auto mine = [&](int tiles) { return max(0, min(tiles - begin, each)); };
  const int T0 = mine(tiles0), T1 = mine(tiles1), TN = max(T0, T1);
  auto stage_tiles = [&](int s) { return s ? T1 : T0; };

  if (warp == 8) {
    tmem_alloc(smem_u32(&ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 10) {
    // ------------------------------------------------------------- copies
    if (TN > 0) {
      const int qh = A.q_by_head ? h : 0, kh = A.k_by_head ? h : 0, vh = A.v_by_head ? h : 0;
      const uint32_t data = uniform(base), bars = uniform(bar(0));
      auto released = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for<kTest>(bar(b), parity, ctl, A.err)) != 0;
      };
      auto load_q = [&](int s) {
        if (stage_tiles(s) > 0 && elect_one()) {
          mbar_arrive_expect_tx(bars + 8 * (B_Q + s), kQStage);
          for (int c = 0; c < 3; ++c)
            tma_load_3d(data + s * kQStage + c * kSlot, &A.q, 64 * c, qh, R.q0 + row0 + s * kStageRows, bars + 8 * (B_Q + s));
        }
      };
      bool ok = true;
      int k_asked = 0, v_asked = 0;
      load_q(0);
      for (int j = 0; j < TN; ++j) {
        // slots in the order of their use: K(j)'s first was K(j - 2)'s last, its others V(j - 2)'s, V(j)'s K(j - 1)'s first
        const int row = R.k0 + (begin + j) * kKeys;
        if (j >= 2) ok = released(B_KFREE + (j & 1), uint32_t(j / 2 - 1) & 1);
        if (!ok) break;
        const uint32_t kf = bars + 8 * (B_KFULL + (j & 1));
        if (elect_one()) {
          mbar_arrive_expect_tx(kf, 3 * kSlot);
          tma_load_3d(data + kOffRing + (5 * j) % kSlots * kSlot, &A.k_nope, 0, kh, row, kf);
        }
        ++k_asked;
        if (j >= 2) ok = released(B_VFREE + (j & 1), uint32_t(j / 2 - 1) & 1);
        if (elect_one()) {
          if (ok) {
            tma_load_3d(data + kOffRing + (5 * j + 1) % kSlots * kSlot, &A.k_nope, 64, kh, row, kf);
            tma_load_3d(data + kOffRing + (5 * j + 2) % kSlots * kSlot, &A.k_rope, 0, 0, row, kf);
          } else {
            mbar_complete_tx(kf, 2 * kSlot);  // the first is on its way: its barrier expects no more
          }
        }
        if (!ok) break;
        if (j == 0) load_q(1);
        if (j >= 1) ok = released(B_KFREE + ((j - 1) & 1), uint32_t((j - 1) / 2) & 1);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t vf = bars + 8 * (B_VFULL + (j & 1));
          mbar_arrive_expect_tx(vf, 2 * kSlot);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t dst = data + kOffRing + (5 * j + 3 + c) % kSlots * kSlot;
            tma_load_3d(dst, &A.v, 0, vh, row + 64 * c, vf);
            tma_load_3d(dst + kSlot / 2, &A.v, 64, vh, row + 64 * c, vf);
          }
        }
        ++v_asked;
      }
      // what was asked for lands before the block ends, read or not (a second stage's Q is asked for with the first tile)
      if (elect_one()) {
        const long long since = clock64();
        for (int s = 0; s < 2; ++s)
          if (stage_tiles(s) > 0) drain(bar(B_Q + s), 0, since, A.err);
        for (int j = max(0, k_asked - 2); j < k_asked; ++j) drain(bar(B_KFULL + (j & 1)), uint32_t(j / 2) & 1, since, A.err);
        for (int j = max(0, v_asked - 2); j < v_asked; ++j) drain(bar(B_VFULL + (j & 1)), uint32_t(j / 2) & 1, since, A.err);
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------- products
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t id_qk = kBf16 ? idesc_bf16_f32(128, 128, 0, 0) : idesc_fp16_f32(128, 128, 0, 0);
    constexpr uint32_t id_pv = kBf16 ? idesc_bf16_f32(128, 128, 0, 1) : idesc_fp16_f32(128, 128, 0, 1);
    const int s = warp - 8, Ts = stage_tiles(s);
    const uint32_t tmem_s = uniform(tmem) + kTmemS + 128 * s, tmem_o = uniform(tmem) + kTmemO + 128 * s, data = uniform(base);
    auto slot_of = [&](int item) { return data + kOffRing + uint32_t(item % kSlots) * kSlot; };
    auto arrived = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for<kTest>(bar(b), parity, ctl, A.err)) != 0;
    };
    // Where both stages have work they take turns, 0 1 0 1 ...: O += P V(j) and the next S are
    // one turn.  Left to themselves they drift into step, share the tensor core while both have
    // work for it and leave it idle while both compute weights (8,192 tokens: 914 us, not 805).
    const bool turns = T0 > 0 && T1 > 0;
    int step = 0;
    auto my_turn = [&]() -> bool {
      if (!turns) return true;
      const bool go = s ? arrived(B_TURN + 1, step & 1) : step == 0 || arrived(B_TURN, (step - 1) & 1);
      ++step;
      return go;
    };
    auto turn_over = [&]() {
      if (turns && elect_one()) mbar_arrive(bar(B_TURN + 1 - s));
    };
    auto qk = [&](int j) -> bool {  // S = Q K(j)^T
      if (!arrived(B_KFULL + (j & 1), uint32_t(j / 2) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const uint64_t a = smem_desc(data + s * kQStage + c * kSlot, 16, 1024, kSwizzle128B);
          const uint64_t b = smem_desc(slot_of(5 * j + c), 16, 1024, kSwizzle128B);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss(tmem_s, desc_add(a, 32 * k), desc_add(b, 32 * k), id_qk, c + k > 0);
        }
        mma_commit(bar(B_S + s));
        if (turns) mbar_arrive(bar(B_TURN + 1 - s));
        mma_commit(bar(B_KFREE + (j & 1)));
      }
      return true;
    };
    auto pv = [&](int j) -> bool {  // O += P V(j)
      if (!arrived(B_VFULL + (j & 1), uint32_t(j / 2) & 1)) return false;
      const int keys = min(kKeys, R.len - (begin + j) * kKeys);
      const uint64_t v0 = smem_desc(slot_of(5 * j + 3), kSlot / 2, 1024, kSwizzle128B);
      const uint64_t v1 = smem_desc(slot_of(5 * j + 4), kSlot / 2, 1024, kSwizzle128B);
      if (keys == kKeys) {
        if (!arrived(B_P + 2 * s, j & 1) || !my_turn()) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ts(tmem_o, tmem_s + 8 * k, desc_add(v0, 2048 * k), id_pv, j > 0 || k > 0);
        }
        if (!arrived(B_P + 2 * s + 1, j & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 4; k < 8; ++k) mma_ts(tmem_o, tmem_s + 8 * k, desc_add(v1, 2048 * (k & 3)), id_pv, 1);
          mma_commit(bar(B_VFREE + (j & 1)));
          if (j + 1 == Ts) mma_commit(bar(B_O + s));
        }
        return true;
      }
      // the request's last tile: only k-steps that hold keys; the rows of V behind
      // the last key may hold anything (another request's, or nobody's) and are
      // zeroed, by both stages alike, since a weight of 0 times NaN is NaN
      const int steps = (keys + 15) / 16;
      for (int u = 16 * keys + lane; u < 256 * steps; u += 32) {  // 16-byte units, 16 a row
        const int key = u / 16, part = u % 16;
        st_shared_v4(slot_of(5 * j + 3 + key / 64) + (part / 8) * (kSlot / 2) + (key % 64) * 128 + (part % 8) * 16, 0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (!arrived(B_P + 2 * s, j & 1) || !arrived(B_P + 2 * s + 1, j & 1) || !my_turn()) return false;
      tc_fence_after();
      if (elect_one()) {
        for (int k = 0; k < steps; ++k)
          mma_ts(tmem_o, tmem_s + 8 * k, desc_add(k < 4 ? v0 : v1, 2048 * (k & 3)), id_pv, j > 0 || k > 0);
        mma_commit(bar(B_VFREE + (j & 1)));
        if (j + 1 == Ts) mma_commit(bar(B_O + s));
      }
      return true;
    };
    // a tile that this stage has no use for is released as soon as it is there
    auto pass_k = [&](int j) -> bool {
      if (!arrived(B_KFULL + (j & 1), uint32_t(j / 2) & 1)) return false;
      if (elect_one()) mbar_arrive(bar(B_KFREE + (j & 1)));
      turn_over();
      return true;
    };
    auto pass_v = [&](int j) -> bool {
      if (!arrived(B_VFULL + (j & 1), uint32_t(j / 2) & 1) || !my_turn()) return false;
      if (elect_one()) mbar_arrive(bar(B_VFREE + (j & 1)));
      return true;
    };
    bool ok = Ts == 0 || arrived(B_Q + s, 0);
    if (ok && TN > 0) ok = my_turn() && (Ts > 0 ? qk(0) : pass_k(0));
    for (int j = 0; j < TN && ok; ++j) {
      ok = j < Ts ? pv(j) : pass_v(j);
      if (!ok) break;
      if (j + 1 >= TN) turn_over();
      else ok = j + 1 < Ts ? qk(j + 1) : pass_k(j + 1);
    }
    if (Ts > 0 && elect_one()) {  // every MMA issued has run once this arrives
      mma_commit(bar(B_FIN + s));
      drain(bar(B_FIN + s), 0, clock64(), A.err);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int s = warp >> 2;
    const int i0 = row0 + s * kStageRows + (warp & 3) * 32, i = i0 + lane;  // rows of the request
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const int Ts = stage_tiles(s);
    const float c = A.scale * kLog2e, grow = kRescaleLog2 / c;
    // keys before `end` are this row's; tiles that end before `clear` need no mask in this warp
    int end = A.causal ? max(0, min(R.len, shift + i + 1)) : R.len;
    int clear = A.causal ? max(0, min(R.len, shift + i0 + 1)) : R.len;
    end -= begin * kKeys, clear -= begin * kKeys;  // from the block's first tile on
    float m = -INFINITY, l = 0.f, taken = 0.f;  // taken: the weights' sum as the product takes them
    bool ok = true;
    for (int j = 0; j < Ts; ++j) {
      uint32_t x[128];
      ok = wait_for<kTest>(bar(B_S + s), j & 1, ctl, A.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      tmem_ld128_sync(tmem + lanes + kTmemS + 128 * s, x);
      const int k0 = j * kKeys;
      if (k0 + kKeys > clear) {
        const int live = end - k0;
#pragma unroll
        for (int u = 0; u < 128; ++u) x[u] = u < live ? x[u] : 0xff800000u;
      }
      float top0 = -INFINITY, top1 = -INFINITY, top2 = -INFINITY, top3 = -INFINITY;
#pragma unroll
      for (int u = 0; u < 128; u += 8) {
        top0 = max3(top0, __uint_as_float(x[u]), __uint_as_float(x[u + 1]));
        top1 = max3(top1, __uint_as_float(x[u + 2]), __uint_as_float(x[u + 3]));
        top2 = max3(top2, __uint_as_float(x[u + 4]), __uint_as_float(x[u + 5]));
        top3 = max3(top3, __uint_as_float(x[u + 6]), __uint_as_float(x[u + 7]));
      }
      const float top = fmaxf(max3(top0, top1, top2), top3);
      const bool move = top > m + grow || m == -INFINITY;  // the first maximum is taken as it is
      if (__any_sync(0xffffffffu, move && j > 0)) {
        // O holds all tiles before this one (its scores come after them)
        const float keep = move ? (m == -INFINITY ? 0.f : ex2((m - top) * c)) : 1.f;
        l *= keep, taken *= keep;
        const uint32_t o = tmem + lanes + kTmemO + 128 * s;
#pragma unroll 1
        for (int u = 0; u < 128; u += 16) {
          uint32_t y[16];
          tmem_ld16_sync(o + u, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
          tmem_st16_sync(o + u, y);
        }
      }
      if (move) m = top;
      const float ref = m == -INFINITY ? 0.f : fmaf(-m, c, kWeightLog2<T>);
      const uint64_t c2 = f2_pack(c, c), ref2 = f2_pack(ref, ref);
      uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          float a, b;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(x[64 * half + 2 * u]), __uint_as_float(x[64 * half + 2 * u + 1])), c2, ref2), a, b);
          a = ex2(a), b = ex2(b);
          if (u & 1) sum1 = f2_add(sum1, f2_pack(a, b));
          else sum0 = f2_add(sum0, f2_pack(a, b));
          x[64 * half + u] = join(a, b, T());  // in place: the register is read already
        }
        tmem_st32_sync(tmem + lanes + kTmemS + 128 * s + 32 * half, reinterpret_cast<const uint32_t(&)[32]>(x[64 * half]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P + 2 * s + half));
      }
      float a, b;
      f2_unpack(f2_add(sum0, sum1), a, b);
      l += a + b;
      float t0 = 0.f, t1 = 0.f, t2 = 0.f, t3 = 0.f;
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        add_halves(x[u], t0, t1, T());
        add_halves(x[64 + u], t2, t3, T());
      }
      taken += (t0 + t1) + (t2 + t3);
    }
    if (ok && Ts > 0) ok = __all_sync(0xffffffffu, wait_for<kTest>(bar(B_O + s), 0, ctl, A.err));
    const int live = s * kStageRows < A.block_rows ? min(32, R.n - i0) : 0;  // rows of this warp
    const int64_t at = int64_t(R.q0 + i0) * A.heads + h;
    const int64_t part_at = split * A.part_rows + (A.by_block ? int64_t(tail) * kBlockRows + (i0 - row0) : at);
    const int part_step = A.by_block ? 1 : A.heads;
    float* part_lse = A.part + A.nsplit * A.part_rows * kV + part_at;
    // a part that a wait gave up on makes its rows NaN, not what the workspace holds
    if (!ok && split_keys && lane < live) part_lse[int64_t(lane) * part_step] = __uint_as_float(0x7fffffffu);
    if (ok && live > 0) {
      const bool some = l != 0.f;  // true for a NaN too, which the row then shows
      const float inv = some ? __frcp_rn(taken) : 0.f;
      tc_fence_after();
      // rows to memory through this stage's part of Q (every product that read it has run), so
      // that a warp stores whole rows; 16-byte units are swizzled by the row.  In short loops: a
      // block runs this once, and straight code waits for its instructions (4,000 cycles)
      const uint32_t mine_s = base + s * kQStage + uint32_t((warp & 3) * 32) * 256u;
      // parts are in fp32, 64 columns at a time
#pragma unroll 1
      for (int u0 = 0; u0 < 128; u0 += split_keys ? 64 : 128) {
        const int u1 = u0 + (split_keys ? 64 : 128);
#pragma unroll 1
        for (int u = u0; u < u1; u += 32) {
          uint32_t y[32];  // anything, where the stage had no tile
          tmem_ld32_sync(tmem + lanes + kTmemO + 128 * s + u, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = some ? __float_as_uint(__uint_as_float(y[e]) * inv) : 0u;
          if (split_keys) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              st_shared_v4(mine_s + lane * 256 + ((((u - u0 + e) / 4) ^ (lane & 15)) << 4), y[e], y[e + 1], y[e + 2], y[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const uint4 w = pack<T>(reinterpret_cast<const float*>(y) + e);
              st_shared_v4(mine_s + lane * 256 + ((((u + e) / 8) ^ (lane & 15)) << 4), w.x, w.y, w.z, w.w);
            }
          }
        }
        __syncwarp();
        // half a warp a row of 256 bytes
        unsigned char* to;
        int64_t pitch;
        if (split_keys) {
          to = reinterpret_cast<unsigned char*>(A.part + part_at * kV + u0);
          pitch = int64_t(part_step) * kV * 4;
        } else {
          to = reinterpret_cast<unsigned char*>(static_cast<T*>(A.out) + int64_t(R.q0 + i0) * A.o_tok + int64_t(h) * A.o_head);
          pitch = A.o_tok * int64_t(sizeof(T));
        }
        to += (lane >> 4) * pitch + (lane & 15) * 16;
#pragma unroll 4
        for (int rr = lane >> 4; rr < 32; rr += 2, to += 2 * pitch) {
          const float4 w = ld_shared_f4(mine_s + rr * 256 + (((lane & 15) ^ (rr & 15)) << 4));
          if (rr < live) *reinterpret_cast<float4*>(to) = w;
        }
        __syncwarp();
      }
      if (lane < live) {
        const float lse = some ? m * A.scale + logf(l * (1.f / kWeight<T>)) : -INFINITY;
        if (split_keys) part_lse[int64_t(lane) * part_step] = lse;
        else if (A.lse) A.lse[at + int64_t(lane) * A.heads] = lse;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the parts of split keys by their lse.  Up to 8 parts: a warp a row, four
// rows a block; more: a block a row, whose four warps take every fourth part.  Either
// way eight loads are in flight (one warp a row with four took 6 us for 38 parts; a block a row for 14,336 rows of two parts
// 16 us, a warp a row 6).
constexpr int kWarpParts = 8;

template <typename T, bool kWarpRow>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ PrefillArgs A) {
  __shared__ float4 sums[4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PrefillBlock B(A, A.whole + blockIdx.x);
  const int row = kWarpRow ? int(blockIdx.y) * 4 + warp : int(blockIdx.y), h = B.h, i = B.row0 + row;
  launched_after();
  const PrefillReq R = load_prefill_req(A, B.r, false);
  if (i >= R.n) return;
  const int64_t at = int64_t(R.q0 + i) * A.heads + h, all = A.part_rows;
  const int64_t part_at = A.by_block ? int64_t(blockIdx.x) * kBlockRows + row : at;
  const float* lse = A.part + A.nsplit * all * kV + part_at;
  const float a = lane < A.nsplit ? lse[lane * all] : -INFINITY;
  const float b = !kWarpRow && lane + 32 < A.nsplit ? lse[(lane + 32) * all] : -INFINITY;
  float top = fmaxf(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  const float wa = expf(a - ref), wb = expf(b - ref);
  float sum = wa + wb;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;  // NaN stays
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kStep = kWarpRow ? 1 : 4;
  for (int k0 = kWarpRow ? 0 : warp; k0 < A.nsplit; k0 += 8 * kStep) {
    float4 v[8];
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + kStep * e;
      w[e] = __shfl_sync(0xffffffffu, k < 32 ? wa : wb, k & 31) * inv;
      if (k >= A.nsplit) w[e] = 0.f;
      v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      // a part of weight 0 is not read
      if (w[e] != 0.f) v[e] = *reinterpret_cast<const float4*>(A.part + (k * all + part_at) * kV + 4 * lane);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc.x = fmaf(w[e], v[e].x, acc.x), acc.y = fmaf(w[e], v[e].y, acc.y);
      acc.z = fmaf(w[e], v[e].z, acc.z), acc.w = fmaf(w[e], v[e].w, acc.w);
    }
  }
  if constexpr (!kWarpRow) {
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int e = 1; e < 4; ++e) {
      const float4 v = sums[e][lane];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
  }
  T* out = static_cast<T*>(A.out) + int64_t(R.q0 + i) * A.o_tok + int64_t(h) * A.o_head;
  *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(join(acc.x, acc.y, T()), join(acc.z, acc.w, T()));
  if (A.lse && lane == 0) A.lse[at] = sum != 0.f ? ref + logf(sum) : -INFINITY;
}

template <typename T> cudaError_t launch_prefill(const PrefillArgs& A, cudaStream_t st) {
  const unsigned blocks = A.whole + unsigned(A.last) * unsigned(A.nsplit);
  auto kernel = A.give_up ? prefill_kernel<T, true> : prefill_kernel<T, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  e = launch_early(kernel, dim3(blocks), kThreads, kSmem, st, A);
  if (e != cudaSuccess || A.nsplit == 1) return e;
  const bool warp_row = A.nsplit <= kWarpParts;
  const unsigned rows = unsigned(A.max_q < kBlockRows ? A.max_q : kBlockRows);
  return launch_early(warp_row ? combine_kernel<T, true> : combine_kernel<T, false>,
                      dim3(unsigned(A.last), warp_row ? (rows + 3) / 4 : rows), 128, 0, st, A);
}

int sm_count() {
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return 0;
  return sms;
}

// nsplit's two numbers, of `blocks` blocks: how many of the last ones are split
// (0 in it: all), and whether their parts have rows of their own.
struct Splits {
  int count;
  int64_t last, rows;
  bool by_block;
  Splits(int nsplit, int64_t blocks, int64_t num_q, int heads) {
    count = nsplit % kSplitLast, last = nsplit / kSplitLast;
    by_block = last > 0;
    if (!by_block || last > blocks) last = blocks;
    rows = by_block ? last * kBlockRows : num_q * heads;
  }
  uint64_t bytes() const { return count > 1 ? uint64_t(count) * uint64_t(rows) * uint64_t(kV + 1) * 4u : 0u; }
};

}  // namespace
}  // namespace mtv

extern "C" int mla_prefill_workspace(int num_sms, int bs, int64_t max_q, int64_t max_kv, int64_t num_q, int num_heads,
                                     int* nsplit_out, uint64_t* bytes_out) {
  using namespace mtv;
  if (!nsplit_out || !bytes_out) return MTV_E_NULL_POINTER;
  if (num_sms < 1 || bs < 0 || bs > MTV_MAX_HEADS || max_q < 0 || max_kv < 0 || num_q < 0 ||
      num_q > MTV_MAX_PREFILL_ROWS || max_q > MTV_MAX_PREFILL_ROWS || max_kv > MTV_MAX_PREFILL_ROWS || num_heads < 0 || num_heads > MTV_MAX_HEADS)
    return MTV_E_BAD_ARGUMENT;
  // as many splits as leave every block an SM, of four key tiles at least (a split costs a second launch
  // and its parts' way through memory)
  const int64_t blocks = int64_t(bs) * num_heads * ((max_q + kBlockRows - 1) / kBlockRows);
  int64_t n = blocks > 0 ? num_sms / blocks : 1, worth = (max_kv + kKeys - 1) / kKeys / 4;
  // More blocks than SMs: those of a last wave that fills half of the SMs at most are split over all of them
  // (256 new after 8,192, 160 heads: 233 -> 148 us; 2 x (1,000 after 5,760), 64 heads: 336 -> 311).  Blocks of
  // a head start longest first, so what counts is the shortest one's tiles: below 16 the join costs what the
  // split gives (3 x (256 after 1,024), 64 heads: 47 us, split 48; 2,048 new: 82 and 85).  After 8 waves the
  // blocks have drifted apart (15 waves: 1,066 us, split 1,087; 5: 374 and 340).
  const int64_t over = blocks > num_sms ? blocks % num_sms : 0;
  const int64_t shortest = (max_kv - max_q + kBlockRows) / kKeys;
  const bool tail = over > 0 && 2 * over <= num_sms && blocks < kTailWaves * int64_t(num_sms) && shortest >= 16;
  if (tail) n = num_sms / over, worth = shortest / 4;
  if (n > worth) n = worth;
  // Blocks of 128 rows (below) give as much as two parts: 256 new after 3,700 keys, 64 heads, 45 us either way,
  // 256 after 3,000 39 and 41, 900 new, 16 heads, 14 and 20; 200 after 8,000 85 and 72
  if (!tail && n == 2 && max_q > kStageRows && max_kv < 28 * kKeys) n = 1;
  if (n > MTV_MAX_PREFILL_SPLITS) n = MTV_MAX_PREFILL_SPLITS;
  *nsplit_out = n < 2 ? 1 : int(n + (tail ? over * kSplitLast : 0));
  *bytes_out = Splits(*nsplit_out, blocks, num_q, num_heads).bytes();
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
  const int give_up = take_give_up(&dtype);
  if (bs < 0 || bs > MTV_MAX_HEADS || max_q < 0 || max_kv < 0 || num_q < 0 || num_kv < 0 ||
      max_q > MTV_MAX_PREFILL_ROWS || max_kv > MTV_MAX_PREFILL_ROWS || num_q > MTV_MAX_PREFILL_ROWS ||
      num_kv > MTV_MAX_PREFILL_ROWS || num_heads < 0 ||
      num_heads > MTV_MAX_HEADS || (dtype != MTV_DTYPE_BF16 && dtype != MTV_DTYPE_FP16) || !isfinite(scale * mtv::kLog2e) ||
      !(scale > 0) || (causal != 0 && causal != 1) || nsplit < 1 || nsplit % kSplitLast < 1 ||
      nsplit % kSplitLast > MTV_MAX_PREFILL_SPLITS)
    return MTV_E_BAD_ARGUMENT;
  const int64_t q_blocks = (max_q + kBlockRows - 1) / kBlockRows;
  const Splits splits(nsplit, q_blocks * num_heads * bs, num_q, num_heads);
  if (splits.count > 1) {
    if (!workspace) return MTV_E_NULL_POINTER;
    if (workspace_bytes < splits.bytes()) return MTV_E_WORKSPACE_SMALL;
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
  // strides that a tensor map takes: no negative ones, rows apart
  for (int64_t s : {q_tok_stride, q_head_stride, k_tok_stride, k_head_stride, k_rope_stride, v_tok_stride, v_head_stride})
    if (!mappable_stride(s)) return MTV_E_BAD_ARGUMENT;
  if ((num_q > 1 && q_tok_stride == 0) || (num_kv > 1 && (k_tok_stride == 0 || k_rope_stride == 0 || v_tok_stride == 0)))
    return MTV_E_BAD_ARGUMENT;
  if (q_blocks * num_heads * bs + splits.last * (splits.count - 1) > INT32_MAX)
    return MTV_E_UNSUPPORTED;
  PrefillArgs A;
  const bool bf16 = dtype == MTV_DTYPE_BF16;
  const int64_t kv_rows = num_kv > 0 ? num_kv : 1;  // without keys nothing is copied: any valid map will do
  const void* kn = num_kv > 0 ? k_nope : q;
  const void* kr = num_kv > 0 ? k_rope : q;
  const void* vv = num_kv > 0 ? v : q;
  if (!encode_heads_map(&A.q, bf16, q, num_q, q_tok_stride, num_heads, q_head_stride, kQK, 64, kStageRows) ||
      !encode_heads_map(&A.k_nope, bf16, kn, kv_rows, k_tok_stride, num_heads, k_head_stride, kNope, 64, kKeys) ||
      !encode_heads_map(&A.k_rope, bf16, kr, kv_rows, k_rope_stride, 1, 0, kRope, 64, kKeys) ||
      !encode_heads_map(&A.v, bf16, vv, kv_rows, v_tok_stride, num_heads, v_head_stride, kV, 64, 64))
    return MTV_E_CUDA;
  A.out = out, A.lse = lse, A.part = static_cast<float*>(workspace), A.qo_indptr = qo_indptr, A.kv_indptr = kv_indptr;
  A.err = err, A.o_tok = out_tok_stride, A.o_head = out_head_stride, A.num_q = num_q, A.num_kv = num_kv;
  A.max_q = max_q, A.max_kv = max_kv, A.scale = scale, A.give_up = give_up, A.heads = num_heads, A.causal = causal;
  A.nsplit = splits.count, A.q_blocks = int(q_blocks), A.last = int(splits.last), A.part_rows = splits.rows;
  A.whole = unsigned(q_blocks * num_heads * bs - splits.last), A.by_block = splits.by_block;
  // Where blocks of 256 rows leave half of the SMs idle and keys are not split, blocks of 128 take half as much
  // in and out (one prompt, 64 heads of 256 tokens 8.2 -> 7.7 us, 16 heads of 900 16.2 -> 14.4)
  A.block_rows = kBlockRows;
  if (A.nsplit == 1 && max_q > kStageRows && 2 * q_blocks * num_heads * bs <= sm_count()) {
    A.block_rows = kStageRows, A.q_blocks = int((max_q + kStageRows - 1) / kStageRows);
    A.last = A.q_blocks * num_heads * bs, A.whole = 0;
  }
  A.q_by_head = q_head_stride != 0, A.k_by_head = k_head_stride != 0, A.v_by_head = v_head_stride != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? launch_prefill<__nv_bfloat16>(A, st) : launch_prefill<__half>(A, st);
  if (e != cudaSuccess) cudaGetLastError();  // or a later launch reports it
  return e == cudaSuccess ? MTV_OK : MTV_E_CUDA;
}
