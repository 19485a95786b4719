// The prefill GEMM's tiles with low-rank adapters beside the projection (the
// adapters' second product as more k of the tile's own, w4a16_lora.hpp).
#include "w4a16_gemm_tile.hpp"

namespace w4a16 {

namespace {

template <int DT, int GS, bool ASYM, int MB, int CB>
__global__ __launch_bounds__(kThreads) void gemm_lora_kernel(const GemmParams p, const LoraTerm lora) {
  gemm_tile<DT, GS, ASYM, MB, CB, false, true>(p, lora);
}

template <int DT, int GS, bool ASYM>
hipError_t launch_mb(const GemmParams& prm, const LoraTerm& lora, int mb, int cb, hipStream_t s) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(prm.units), dim3(kThreads), 0, s, prm, lora);
    return hipGetLastError();
  };
  switch (10 * mb + cb) {
    case 11: return go(gemm_lora_kernel<DT, GS, ASYM, 1, 1>);
    case 41: return go(gemm_lora_kernel<DT, GS, ASYM, 4, 1>);
    case 81: return go(gemm_lora_kernel<DT, GS, ASYM, 8, 1>);
    case 12: return go(gemm_lora_kernel<DT, GS, ASYM, 1, 2>);
    case 42: return go(gemm_lora_kernel<DT, GS, ASYM, 4, 2>);
    case 62: return go(gemm_lora_kernel<DT, GS, ASYM, 6, 2>);
    case 82: return go(gemm_lora_kernel<DT, GS, ASYM, 8, 2>);
    default: return hipErrorInvalidValue;
  }
}

template <int DT>
hipError_t launch_g(const GemmParams& prm, const LoraTerm& lora, int group, int mb, int cb, hipStream_t s) {
  const bool z = prm.zp != nullptr;
  switch (group) {
    case 32: return z ? launch_mb<DT, 32, true>(prm, lora, mb, cb, s) : launch_mb<DT, 32, false>(prm, lora, mb, cb, s);
    case 64: return z ? launch_mb<DT, 64, true>(prm, lora, mb, cb, s) : launch_mb<DT, 64, false>(prm, lora, mb, cb, s);
    case 128: return z ? launch_mb<DT, 128, true>(prm, lora, mb, cb, s) : launch_mb<DT, 128, false>(prm, lora, mb, cb, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gemm_lora_tiles(const GemmParams& prm, const LoraTerm& lora, int dtype, int group, int mb, int cb,
                                  hipStream_t s) {
  return dtype == DT_F16 ? launch_g<DT_F16>(prm, lora, group, mb, cb, s) : launch_g<DT_BF16>(prm, lora, group, mb, cb, s);
}

}  // namespace w4a16
