// Quantisation of activations to 8-bit floating point (OCP e4m3), and the
// slots of a routed batch in their experts' order.
#include <algorithm>

#include "w4a16_experts.h"
#include "w4a16_fp8.hpp"

namespace w4a16 {

namespace {

// A wave takes runs of 512 values of a row: eight a lane, so that sixteen lanes
// hold a block of 128 and the wave the four scales of a word.  ALIGNED: rows
// are whole 16-byte pieces; otherwise values are loaded one by one.
template <int DT, bool ALIGNED>
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ codes,
                                                       uint32_t* __restrict__ scales, int64_t runs, int runs_per_row,
                                                       int K, int columns) {
  const int lane = threadIdx.x & 63;
  const int64_t run = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (run >= runs) return;
  const int64_t m = run / runs_per_row;
  const int r = (int)(run - m * runs_per_row), k = 512 * r + 8 * lane;
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (ALIGNED) {
    if (k < K) v = *reinterpret_cast<const u32x4*>(x + m * K + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) v[i / 2] |= (uint32_t)x[m * K + k + i] << (16 * (i & 1));
  }
  int e;
  const u32x2 c = quantize_run<DT>(v, e);
  if (k < columns)
    *reinterpret_cast<u32x2*>(codes + m * columns + k) = c;
  const int e1 = __shfl(e, 16), e2 = __shfl(e, 32), e3 = __shfl(e, 48);
  if (lane == 0)
    scales[run] = (uint32_t)(e + 127) | (uint32_t)(e1 + 127) << 8 | (uint32_t)(e2 + 127) << 16 | (uint32_t)(e3 + 127) << 24;
}

// Workgroup e lists the slots of expert e (the last one those that name none),
// in slot order: its waves take parts of the slots one after another, count
// their own and those below e, and after one barrier write theirs behind the
// waves before them.  No atomics, so the order is always the same.
constexpr int kOrderWaves = 16;
__global__ __launch_bounds__(64 * kOrderWaves) void expert_order_kernel(const int32_t* __restrict__ ids,
                                                                        int32_t* __restrict__ start,
                                                                        int32_t* __restrict__ order, int slots, int E) {
  __shared__ int below[kOrderWaves], own[kOrderWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
  const int part = (slots + 64 * kOrderWaves - 1) / (64 * kOrderWaves) * 64;
  const int begin = min(slots, wave * part), end = min(slots, begin + part);
  int nb = 0, no = 0;
  for (int i = begin + lane; i - lane < end; i += 64) {
    int id = i < end ? ids[i] : INT32_MAX;
    if (i < end && (id < 0 || id >= E)) id = E;
    nb += __popcll(__ballot(id < e));
    no += __popcll(__ballot(id == e));
  }
  if (lane == 0) below[wave] = nb, own[wave] = no;
  __syncthreads();
  int at = 0, before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kOrderWaves; ++w) {
    at += below[w];
    before += w < wave ? own[w] : 0;
    all += own[w];
  }
  if (threadIdx.x == 0) {
    start[e] = at;
    if (e == E) start[E + 1] = at + all;
  }
  at += before;
  for (int i = begin + lane; i - lane < end; i += 64) {
    int id = i < end ? ids[i] : INT32_MAX;
    if (i < end && (id < 0 || id >= E)) id = E;
    const uint64_t mine = __ballot(id == e);
    if (id == e) order[at + __popcll(mine & ((1ull << lane) - 1))] = i;
    at += __popcll(mine);
  }
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, int dtype,
                               hipStream_t s) {
  const int64_t per_row = fp8_scales(K) / 4, runs = M * per_row, blocks = (runs + 3) / 4;
  const bool whole = K % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const uint16_t*>(x), codes,
                       reinterpret_cast<uint32_t*>(scales), runs, (int)per_row, (int)K, (int)fp8_columns(K));
  };
  if (dtype == DT_F16) whole ? go(quantize_kernel<DT_F16, true>) : go(quantize_kernel<DT_F16, false>);
  else whole ? go(quantize_kernel<DT_BF16, true>) : go(quantize_kernel<DT_BF16, false>);
  return hipGetLastError();
}

hipError_t launch_expert_order(const int32_t* ids, int32_t* start, int32_t* order, int slots, int E, hipStream_t s) {
  hipLaunchKernelGGL(expert_order_kernel, dim3((unsigned)E + 1), dim3(64 * kOrderWaves), 0, s, ids, start, order, slots, E);
  return hipGetLastError();
}

}  // namespace w4a16
