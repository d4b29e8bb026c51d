// Tensor maps over the paged cache (host code), for the tiled copies of the
// attention kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "internal.h"

namespace flint {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

int attn_box(int block_size, int most) {
  int box = 1;
  while (box < most && block_size % (2 * box) == 0) box *= 2;
  return box;
}

bool attn_map(CUtensorMap* m, const AttnArgs& a, const uint16_t* base, int box) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {128, (cuuint64_t)a.nkv, (cuuint64_t)a.block_size, (cuuint64_t)a.num_blocks};
  // the stride of an extent of 1 is never used, but has to be a valid one
  const cuuint64_t strides[3] = {(cuuint64_t)(a.nkv > 1 ? a.s_head * 2 : 256),
                                 (cuuint64_t)(a.block_size > 1 ? a.s_slot * 2 : 256),
                                 (cuuint64_t)(a.num_blocks > 1 ? a.s_block * 2 : 256)};
  for (cuuint64_t s : strides)
    if (s == 0 || s >= (1ull << 40)) return false;
  const cuuint32_t bx[4] = {64, 1, (cuuint32_t)box, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_q_map(CUtensorMap* m, const AttnArgs& a, int heads, int tokens) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {128, (cuuint64_t)a.nq, (cuuint64_t)a.T};
  const cuuint64_t strides[2] = {256, (cuuint64_t)(a.T > 1 ? a.q_stride * 2 : 256)};
  if (strides[1] == 0 || strides[1] >= (1ull << 40)) return false;
  const cuuint32_t bx[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace flint
