// AdamW: the table of tensors that the host lays out and the kernels read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

constexpr int DT_F32 = 2;  // beside DT_F16 and DT_BF16
constexpr int kAdamwChunkBlocks = 16;  // 256-element blocks of one workgroup

// the device table: `tensors` of these, then one AdamwChunk per workgroup
struct AdamwTensor {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* copy;
  int64_t n;
  int64_t first_block;  // blocks of the tensors before it
  int32_t copy_dtype;
  int32_t vec;          // every pointer takes four-element accesses
};
struct AdamwChunk {
  int32_t tensor;
  int32_t block;  // first of up to kAdamwChunkBlocks blocks in the tensor
};
struct AdamwScalars {
  float beta1, one_beta1, beta2, one_beta2, eps, decay, rate, root, grad_scale;
  uint32_t seed;
};

hipError_t launch_adamw(const void* table, int tensors, int chunks, int param_dtype, int grad_dtype, int bits,
                        const AdamwScalars& h, hipStream_t s);
hipError_t launch_adamw_moments(const void* table, int tensors, int chunks, float* m, float* v, hipStream_t s);

}  // namespace w4a16
