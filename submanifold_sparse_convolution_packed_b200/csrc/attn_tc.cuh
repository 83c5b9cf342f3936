// Shared by the tensor-core attention kernels: packing of fp32 pairs,
// stores of whole rows, the TMA maps of [rows, heads, dim] tensors.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "kernels.h"
#include "tcgen05_attn.cuh"
#include "tokens.cuh"

namespace smc {
namespace attn {

constexpr int kRows = 128;                // rows of a resident tile
constexpr uint32_t kPanel = kRows * 128;  // 128 rows of 64 16-bit channels

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Stores 32 columns of a warp's 32 rows, one row per lane in o, through 2 KB of
// shared memory: a row's 64 bytes leave from four neighbouring lanes, where the
// lanes' own rows would leave 16 bytes at a time.  `at`: the place of the
// lane's row in `to` (elements), negative for none.  Warp-collective.
template <typename T>
__device__ __forceinline__ void store_rows(uint8_t* stage, const float (&o)[32], T* to, int64_t at, int c0, int dim) {
  const int lane = threadIdx.x & 31;
  uint4* s = reinterpret_cast<uint4*>(stage);
#pragma unroll
  for (int i = 0; i < 4; ++i)  // pieces swizzled so that eight rows meet eight banks groups
    s[lane * 4 + (i ^ ((lane >> 1) & 3))] =
        make_uint4(pack2<T>(o[8 * i], o[8 * i + 1]), pack2<T>(o[8 * i + 2], o[8 * i + 3]),
                   pack2<T>(o[8 * i + 4], o[8 * i + 5]), pack2<T>(o[8 * i + 6], o[8 * i + 7]));
  __syncwarp();
  const int piece = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2);
    const int64_t there = __shfl_sync(0xffffffffu, at, row);
    if (there >= 0 && c0 + 8 * piece < dim)
      *reinterpret_cast<uint4*>(to + there + c0 + 8 * piece) = s[row * 4 + (piece ^ ((row >> 1) & 3))];
  }
  __syncwarp();
}

// A [rows, heads, dim] tensor as boxes of 64 channels x `bh` heads x `br` rows.
inline bool make_map(CUtensorMap* map, const void* p, int dtype, int64_t rows, int heads, int dim, const int64_t st[2], int bh,
              int br) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(st[1]) * 2, static_cast<cuuint64_t>(st[0]) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(bh), static_cast<cuuint32_t>(br)};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUtensorMapDataType dt = dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode_fn()(map, dt, 3, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool map_fits(const void* p, const int64_t st[2]) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && st[0] > 0 && st[1] > 0 && st[0] % 8 == 0 && st[1] % 8 == 0 &&
         st[0] < (int64_t{1} << 38) && st[1] < (int64_t{1} << 38);
}

}  // namespace attn
}  // namespace smc
