// Tensor maps and TMA copies: the host-side encoder, and the device-side load
// and store of a tile.  The innermost coordinate of every copy is a multiple of
// 16 bytes (64 elements of 16 bits here).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mtv {

// The driver's encoder, looked up once a process; null where there is none.
inline decltype(&cuTensorMapEncodeTiled) tensor_map_encoder() {
  static const auto fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
  }();
  return fn;
}

// A [rows, heads, dim] tensor of 16-bit values, dense in dim, as a map over
// (dim, heads, rows) with boxes of box_dim x 1 x box_rows, 128-byte swizzled
// (box_dim 64).  A head stride of 0 (or one head) makes a map of one head: its
// copies pass head coordinate 0.  Values outside the tensor read as 0.
inline bool encode_heads_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t row_stride, int heads,
                             int64_t head_stride, int dim, int box_dim, int box_rows) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const bool one = heads == 1 || head_stride == 0;
  const cuuint64_t dims[3] = {cuuint64_t(dim), one ? 1u : cuuint64_t(heads), cuuint64_t(rows)};
  // the stride of an extent of one is never used, but has to be a multiple of 16 bytes
  const cuuint64_t strides[2] = {one ? 16u : cuuint64_t(head_stride) * 2, rows == 1 ? 16u : cuuint64_t(row_stride) * 2};
  const cuuint32_t box[3] = {cuuint32_t(box_dim), 1, cuuint32_t(box_rows)}, steps[3] = {1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
                dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for reads whose innermost extent may be cut into chunks of 64, so that
// one copy brings several: a map over (64, heads, rows, dim / 64) with boxes of 64 x
// 1 x box_rows x box_chunks.  With dim no multiple of 64 (`whole` false) it is (dim,
// heads, rows, 1) with boxes of one chunk, whose start is the first coordinate.
inline bool encode_chunked_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t row_stride, int heads,
                               int64_t head_stride, int dim, bool whole, int box_rows, int box_chunks) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const bool one = heads == 1 || head_stride == 0;
  const cuuint64_t dims[4] = {whole ? 64u : cuuint64_t(dim), one ? 1u : cuuint64_t(heads), cuuint64_t(rows),
                              whole ? cuuint64_t(dim / 64) : 1u};
  const cuuint64_t strides[3] = {one ? 16u : cuuint64_t(head_stride) * 2, rows == 1 ? 16u : cuuint64_t(row_stride) * 2, 128u};
  const cuuint32_t box[4] = {64, 1, cuuint32_t(box_rows), whole ? cuuint32_t(box_chunks) : 1u}, steps[4] = {1, 1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
                dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether encode_heads_map takes these strides (elements of 16 bits).
inline bool mappable_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s < (int64_t(1) << 38); }

namespace ptx {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// Into this CTA's memory, completing on a barrier of this or the other CTA of a pair (address from mapa).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c0, int c1, int c2, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c0), "r"(c1),
               "r"(c2), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's bulk groups still read shared memory.
template <int N> __device__ __forceinline__ void bulk_wait_group_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace ptx
}  // namespace mtv
