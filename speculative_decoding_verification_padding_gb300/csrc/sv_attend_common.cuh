// sv_attend_common.cuh — how the attention kernels see the paged cache: tensor
// maps of K and V, and the shared-memory image of a stage of four pages.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "sv_internal.cuh"

namespace sv {
namespace attn {

// Shared-memory image of one stage: for K then V, 4 pages x (D / 64) boxes of
// 16 rows x 128 bytes, as TMA writes them with the 128-byte swizzle (16-byte
// chunk c of row r of a box stored at chunk c ^ (r % 8)).
template <int D>
struct StageLayout {
  static constexpr int kHalves = D / 64;                 // boxes per page
  static constexpr int kBoxBytes = 16 * 128;
  static constexpr int kTensorBytes = 4 * kHalves * kBoxBytes;  // 64 tokens
  static constexpr int kStageBytes = 2 * kTensorBytes;
  // byte offset of (token t of the stage, 16-byte chunk c of the head dim)
  __device__ static __forceinline__ uint32_t off(int t, int c) {
    const int r = t & 15;
    return (uint32_t)((((t >> 4) * kHalves + (c >> 3)) * kBoxBytes) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  }
};

// cuTensorMapEncodeTiled from the driver, fetched through the runtime (no
// link against the driver library).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A cache viewed as rows of D bf16 (num_blocks * Hkv * 16 rows), boxes of
// 64 elements x 16 rows, 128-byte swizzle.
inline bool make_map(CUtensorMap* map, const void* base, int num_blocks, int Hkv, int D) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)num_blocks * Hkv * kBlockSize};
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, 16};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace sv
