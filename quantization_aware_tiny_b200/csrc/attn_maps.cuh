// Host side of the attention launches: tensor maps and the shared-memory limit.
#pragma once

#include <atomic>

#include "attn_sm100.cuh"
#include "gemm_sm100.cuh"

namespace qat {

// [token][head][dim] map of a bf16 tensor with rows ld elements apart: boxes of
// 64 dims of one head of `rows` tokens, 128-byte swizzle.  Dims behind a head's
// end and tokens behind the tensor's read as zero.
inline int make_head_map(CUtensorMap* m, const void* base, int hd, int heads, int64_t tokens,
                         int64_t ld, int rows) {
  EncodeFn enc = get_encode();
  if (!enc) return QAT_ERR_UNSUPPORTED;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? QAT_OK : QAT_ERR_ARG;
}

// Raises a kernel's dynamic shared-memory limit once per device.
inline int allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (device_flag_once(done, &dev)) return QAT_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return QAT_ERR_CUDA;
  device_flag_set(done, dev);
  return QAT_OK;
}

}  // namespace qat
