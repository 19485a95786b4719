// Device side of the 8-bit floating-point activations: a block's scale and its
// codes.
#pragma once

#include "w4a16_device.hpp"

namespace w4a16 {

typedef short short2_t __attribute__((ext_vector_type(2)));

// Exponent of the scale of a block whose largest finite magnitude has these
// bits (of the activation dtype): the smallest e for which it is at most
// 448 * 2^e (448 = 1.75 * 2^8, e4m3's largest), at least -126; 0 for zeros.
template <int DT>
__device__ __forceinline__ int block_exponent(uint32_t bits) {
  const uint32_t f = __builtin_bit_cast(uint32_t, act_to_f32<DT>((uint16_t)bits));
  const int e = (int)(f >> 23) - 127 - 8 + ((f & 0x007FFFFFu) > 0x00600000u);
  return f ? max(e, -126) : 0;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2_int(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// magnitude bits of both halves, zero where they are infinite or NaN
template <int DT>
__device__ __forceinline__ uint32_t finite_bits(uint32_t h) {
  constexpr uint32_t inf = DT == DT_F16 ? 0x7C00u : 0x7F80u;
  h &= 0x7FFFu;
  return h < inf ? h : 0u;
}

// Codes of the pair x / scale, scale a power of two (rounded once, to
// nearest-even; infinite and NaN values give e4m3's NaN).
template <int DT, bool HIGH>
__device__ __forceinline__ short2_t codes_of(short2_t old, uint32_t pair, float scale) {
  if constexpr (DT == DT_F16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(old, __builtin_bit_cast(half2_t, pair), scale, HIGH);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, __builtin_bit_cast(bf16x2_t, pair), scale, HIGH);
}

// Codes of a lane's eight values, sixteen lanes holding a block of 128, and the
// exponent of their scale.
template <int DT>
__device__ __forceinline__ u32x2 quantize_run(u32x4 v, int& e) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(finite_bits<DT>(v[i]), finite_bits<DT>(v[i] >> 16)));
#pragma unroll
  for (int o = 8; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  e = block_exponent<DT>(top);
  const float scale = exp2_int(e);
  short2_t lo = {0, 0}, hi = {0, 0};
  lo = codes_of<DT, false>(lo, v[0], scale);
  lo = codes_of<DT, true>(lo, v[1], scale);
  hi = codes_of<DT, false>(hi, v[2], scale);
  hi = codes_of<DT, true>(hi, v[3], scale);
  return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

}  // namespace w4a16
