// AdamW: the table of tensors that the host lays out and the kernels read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

constexpr int DT_F32 = 2;  // beside DT_F16 and DT_BF16
// 256-element blocks of a wave (a workgroup has four): four, or one where the
// table has fewer than eight blocks for every wave of 256 CUs (a layer's
// adapters: 11.8 -> 5 us)
constexpr int64_t kAdamwSmallBlocks = 256 * 4 * 8;
inline int adamw_blocks_per_wave(int64_t blocks) { return blocks < kAdamwSmallBlocks ? 1 : 4; }

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
  int32_t block;  // first block in the tensor of up to 4 * blocks_per_wave
};
struct AdamwScalars {
  float beta1, one_beta1, beta2, one_beta2, eps, decay, rate, root, grad_scale;
  uint32_t seed;
};

hipError_t launch_adamw(const void* table, int tensors, int chunks, int blocks_per_wave, int param_dtype, int grad_dtype,
                        int bits, const AdamwScalars& h, hipStream_t s);
hipError_t launch_adamw_moments(const void* table, int tensors, int chunks, int blocks_per_wave, float* m, float* v,
                                hipStream_t s);

}  // namespace w4a16
