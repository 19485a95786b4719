// Quantisation of activations to 8-bit floating point (OCP e4m3), and the
// slots of a routed batch in their experts' order.
#include <algorithm>

#include "w4a16_experts.h"
#include "w4a16_fp8.hpp"

namespace w4a16 {

namespace {

// A wave takes a run of 512 values of a row: eight a lane, so that sixteen lanes
// hold a block of 128 and the wave the four scales of a word.  ALIGNED: rows
// are whole 16-byte pieces; otherwise values are loaded one by one.  A block's
// largest value goes over sixteen lanes, and a value's code is the matrix unit's own
// conversion with the scale's power of two, rounded once.  Bound by memory: 8192 x
// 14336 65 us, 5.4 TB/s; 67 x 2560 2.7 us, a launch.
struct QuantizeParams {
  const uint16_t* x;
  uint8_t* codes;
  uint32_t* scales;
  int64_t runs;
  int runs_per_row, K, columns;
};
template <int DT, bool ALIGNED>
__device__ __forceinline__ void quantize(const QuantizeParams& p, int64_t run) {
  const int lane = threadIdx.x & 63;
  if (run >= p.runs) return;
  const int64_t m = run / p.runs_per_row;
  const int r = (int)(run - m * p.runs_per_row), k = 512 * r + 8 * lane;
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (ALIGNED) {
    if (k < p.K) v = *reinterpret_cast<const u32x4*>(p.x + m * p.K + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < p.K) v[i / 2] |= (uint32_t)p.x[m * p.K + k + i] << (16 * (i & 1));
  }
  int e;
  const u32x2 c = quantize_run<DT>(v, e);
  if (k < p.columns)
    *reinterpret_cast<u32x2*>(p.codes + m * p.columns + k) = c;
  const int e1 = __shfl(e, 16), e2 = __shfl(e, 32), e3 = __shfl(e, 48);
  if (lane == 0)
    p.scales[run] = (uint32_t)(e + 127) | (uint32_t)(e1 + 127) << 8 | (uint32_t)(e2 + 127) << 16 | (uint32_t)(e3 + 127) << 24;
}

template <int DT, bool ALIGNED>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeParams p) {
  quantize<DT, ALIGNED>(p, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
}

// Workgroup e lists the slots of expert e (the last one those that name none),
// in slot order: its waves take parts of the slots one after another, count
// their own and those below e, and after one barrier write theirs behind the
// waves before them.  No atomics, so the order is always the same.  Bound by the
// latency of its loads, sixteen of which are under way at a time: 16384 slots of
// 64 experts 10 us together with 2048 rows' quantisation, 11.6 and 7.4 one after
// the other with one load at a time.
constexpr int kOrderWaves = 16, kOrderLoads = 16;
struct OrderParams {
  const int32_t* ids;
  int32_t *start, *order;
  int slots, E;
};
__device__ __forceinline__ void order_slots(const OrderParams& p, int e) {
  __shared__ int below[kOrderWaves], own[kOrderWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int part = (p.slots + 64 * kOrderWaves - 1) / (64 * kOrderWaves) * 64;
  const int begin = min(p.slots, wave * part), end = min(p.slots, begin + part);
  // f(slot, the expert that it names: E for none, more past the end)
  auto each = [&](auto&& f) {
    for (int at = begin; at < end; at += 64 * kOrderLoads) {
      int id[kOrderLoads];
#pragma unroll
      for (int j = 0; j < kOrderLoads; ++j) {
        const int i = at + 64 * j + lane;
        id[j] = p.ids[min(i, end - 1)];
      }
#pragma unroll
      for (int j = 0; j < kOrderLoads; ++j) {
        const int i = at + 64 * j + lane;
        const bool named = id[j] >= 0 && id[j] < p.E;
        f(i, i < end ? (named ? id[j] : p.E) : INT32_MAX);
      }
    }
  };
  int nb = 0, no = 0;
  each([&](int, int id) {
    nb += __popcll(__ballot(id < e));
    no += __popcll(__ballot(id == e));
  });
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
    p.start[e] = at;
    if (e == p.E) p.start[p.E + 1] = at + all;
  }
  at += before;
  each([&](int i, int id) {
    const uint64_t mine = __ballot(id == e);
    if (id == e) p.order[at + __popcll(mine & ((1ull << lane) - 1))] = i;
    at += __popcll(mine);
  });
}

__global__ __launch_bounds__(64 * kOrderWaves) void expert_order_kernel(OrderParams p) { order_slots(p, blockIdx.x); }

// both: neither waits for the other, and there is one launch less before the products
template <int DT, bool ALIGNED>
__global__ __launch_bounds__(64 * kOrderWaves) void quantize_and_order_kernel(QuantizeParams q, OrderParams o) {
  const int b = (int)blockIdx.x - (o.E + 1);
  if (b < 0) order_slots(o, blockIdx.x);
  else quantize<DT, ALIGNED>(q, (int64_t)b * kOrderWaves + (threadIdx.x >> 6));
}

QuantizeParams params_of(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K) {
  const int64_t per_row = fp8_scales(K) / 4;
  return {static_cast<const uint16_t*>(x), codes, reinterpret_cast<uint32_t*>(scales), M * per_row, (int)per_row, (int)K, (int)fp8_columns(K)};
}
// f(type, whether rows are whole 16-byte pieces)
template <typename F>
void by_form(const void* x, int64_t K, int dtype, F&& f) {
  using F16 = std::integral_constant<int, DT_F16>;
  using BF16 = std::integral_constant<int, DT_BF16>;
  const bool whole = K % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  if (dtype == DT_F16) whole ? f(F16{}, std::true_type{}) : f(F16{}, std::false_type{});
  else whole ? f(BF16{}, std::true_type{}) : f(BF16{}, std::false_type{});
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, int dtype,
                               hipStream_t s) {
  const QuantizeParams q = params_of(x, codes, scales, M, K);
  by_form(x, K, dtype, [&](auto dt, auto whole) {
    hipLaunchKernelGGL((quantize_kernel<decltype(dt)::value, decltype(whole)::value>), dim3((unsigned)((q.runs + 3) / 4)),
                       dim3(256), 0, s, q);
  });
  return hipGetLastError();
}

hipError_t launch_expert_order(const int32_t* ids, int32_t* start, int32_t* order, int slots, int E, hipStream_t s) {
  hipLaunchKernelGGL(expert_order_kernel, dim3((unsigned)E + 1), dim3(64 * kOrderWaves), 0, s, OrderParams{ids, start, order, slots, E});
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_and_order(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, int dtype,
                                         const int32_t* ids, int32_t* start, int32_t* order, int slots, int E, hipStream_t s) {
  const QuantizeParams q = params_of(x, codes, scales, M, K);
  const unsigned grid = (unsigned)(E + 1 + (q.runs + kOrderWaves - 1) / kOrderWaves);
  by_form(x, K, dtype, [&](auto dt, auto whole) {
    hipLaunchKernelGGL((quantize_and_order_kernel<decltype(dt)::value, decltype(whole)::value>), dim3(grid), dim3(64 * kOrderWaves), 0, s,
                       q, OrderParams{ids, start, order, slots, E});
  });
  return hipGetLastError();
}

}  // namespace w4a16
