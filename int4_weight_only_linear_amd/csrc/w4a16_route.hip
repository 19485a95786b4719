// Routing of tokens to experts and its gradient.
#include <algorithm>

#include "w4a16_device.hpp"
#include "w4a16_experts.h"

namespace w4a16 {

namespace {

enum { DT_F32 = 2 };

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return act_to_f32<DT>(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float v) {
  if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = f32_to_act<DT>(v);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// what this wave's lanes have stored in LDS is there for all of them
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

constexpr int kRouteWaves = 4;

// One wave a row, V experts a lane (expert 64 v + lane).
template <int DT, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  __shared__ double keys[kRouteWaves][64 * V];
  __shared__ double group_key[kRouteWaves][kMaxGroups];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (m >= a.M) return;  // (waves share nothing)
  const double none = -__builtin_inf();
  float l[V];
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    l[v] = e < a.E ? load_logit<DT>(a.logits, m * a.E + e) : -__builtin_inff();
    nan |= l[v] != l[v];
    if (l[v] != l[v]) l[v] = -__builtin_inff();
  }
  nan = __ballot(nan) != 0;
  double score[V], key[V];
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) score[v] = 1.0 / (1.0 + exp(-(double)l[v]));
  } else {
    float top = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, l[v]);
    top = wave_max(top);
    double sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // (equal to the largest: 1, also where that is infinite)
      score[v] = l[v] == -__builtin_inff() ? 0.0 : (l[v] == top ? 1.0 : exp((double)l[v] - (double)top));
      sum += score[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) score[v] = sum > 0 ? score[v] / sum : 0.0;
  }
  // scores grow with the logits: where nothing is added to them the logits rank the experts
  const bool by_logit = !a.bias && a.group_top == 1;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    key[v] = by_logit ? (double)l[v] : score[v] + (a.bias && e < a.E ? (double)a.bias[e] : 0.0);
    if (!(l[v] > -__builtin_inff()) || !(key[v] > none)) key[v] = none;
  }
  if (a.groups > 1) {
    const int per = a.E / a.groups;
#pragma unroll
    for (int v = 0; v < V; ++v) keys[wave][64 * v + lane] = key[v];
    wave_lds_fence();
    double mine = none;
    if (lane < a.groups) {
      double first = none, second = none;
      for (int i = 0; i < per; ++i) {
        const double k = keys[wave][lane * per + i];
        second = fmax(second, fmin(first, k));
        first = fmax(first, k);
      }
      mine = a.group_top == 2 && second > none ? first + second : first;
      group_key[wave][lane] = mine;
    }
    wave_lds_fence();
    int rank = 0;
    if (lane < a.groups)
      for (int g = 0; g < a.groups; ++g) {
        const double k = group_key[wave][g];
        rank += k > mine || (k == mine && g < lane);
      }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.topk_groups);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 64 * v + lane;
      if (e >= a.E || !((kept >> (e / per)) & 1)) key[v] = none;
    }
  }
  // the largest key, then the next: lane j keeps the j-th
  double weight = 0;
  int id = -1;
  for (int j = 0; j < a.topk; ++j) {
    double best = none, s = 0;
    int at = kMaxExperts;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] >= best && key[v] > none) best = key[v], at = 64 * v + lane, s = score[v];
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      const double other = __shfl_xor(best, o), so = __shfl_xor(s, o);
      const int oat = __shfl_xor(at, o);
      if (other > best || (other == best && oat < at)) best = other, at = oat, s = so;
    }
    if (at == kMaxExperts) break;  // none left
    if (lane == j) weight = s, id = at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == 64 * v + lane) key[v] = none;
  }
  if (a.renormalize) {
    const double sum = wave_sum(weight);
    weight = sum > 0 ? weight / sum : 0.0;
  }
  if (lane < a.topk) {
    a.weights[m * a.topk + lane] = nan ? __builtin_nanf("") : (float)(weight * (double)a.scale);
    a.ids[m * a.topk + lane] = id;
  }
}

// One wave a row, V experts a lane (expert 64 v + lane).
template <int DT, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_kernel(RouteBackwardArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (m >= a.M) return;
  float s[V], rest[V], ds[V];  // score, 1 - score, its gradient
  if (a.sigmoid) {
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 64 * v + lane;
      const float l = e < a.E ? load_logit<DT>(a.logits, m * a.E + e) : -__builtin_inff();
      // (of the two, the small one is formed without a difference)
      const float t = expf(-fabsf(l)), q = 1.f / (1.f + t);
      s[v] = l >= 0 ? q : t * q;
      rest[v] = l >= 0 ? t * q : q;
      nan |= l != l;
    }
    // a NaN makes its row NaN, as in the forward pass
    if (__ballot(nan)) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = __builtin_nanf("");
    }
  } else {
    float top = -__builtin_inff(), sum = 0;
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 64 * v + lane;
      s[v] = e < a.E ? load_logit<DT>(a.logits, m * a.E + e) : -__builtin_inff();
      nan |= s[v] != s[v];
      top = fmaxf(top, s[v]);
    }
    top = wave_max(top);
    nan = __ballot(nan) != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = s[v] == -__builtin_inff() ? 0.f : (s[v] == top ? 1.f : expf(s[v] - top));
      sum += s[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = nan ? __builtin_nanf("") : (sum > 0 ? s[v] / sum : 0.f);
  }
  // lane j: slot j's expert and gradient
  const int id = lane < a.topk ? a.ids[m * a.topk + lane] : -1;
  const bool named = id >= 0 && id < a.E;
  float g = named ? a.dweights[m * a.topk + lane] * a.scale : 0.f;
  if (a.renormalize) {
    float p = 0;
    for (int j = 0; j < a.topk; ++j) {
      const int e = __shfl(id, j);
      if (e < 0 || e >= a.E) continue;
      float at = 0;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e >> 6 == v) at = s[v];
      at = __shfl(at, e & 63);
      if (lane == j) p = at;
    }
    const float sum = wave_sum(p);
    const float inv = sum > 0 ? 1.f / sum : (sum == 0 ? 0.f : sum);
    const float c = wave_sum(p * inv * g);
    g = named ? (g - c) * inv : 0.f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) ds[v] = 0;
  for (int j = 0; j < a.topk; ++j) {
    const int e = __shfl(id, j);
    const float gj = __shfl(g, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == 64 * v + lane) ds[v] += gj;
  }
  float dot = 0;
  if (!a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) dot += s[v] * ds[v];
    dot = wave_sum(dot);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    if (e >= a.E) continue;
    store_logit<DT>(a.dlogits, m * a.E + e, a.sigmoid ? ds[v] * s[v] * rest[v] : s[v] * (ds[v] - dot));
  }
}

template <template <int, int> class Launch, typename Args>
hipError_t by_type_and_size(const Args& a, hipStream_t s) {
  auto size = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (a.E <= 64) return Launch<DT, 1>::run(a, s);
    if (a.E <= 128) return Launch<DT, 2>::run(a, s);
    if (a.E <= 256) return Launch<DT, 4>::run(a, s);
    if (a.E <= 512) return Launch<DT, 8>::run(a, s);
    return Launch<DT, 16>::run(a, s);
  };
  if (a.dtype == DT_F16) return size(std::integral_constant<int, DT_F16>{});
  if (a.dtype == DT_BF16) return size(std::integral_constant<int, DT_BF16>{});
  return size(std::integral_constant<int, DT_F32>{});
}

dim3 route_grid(int64_t M) { return dim3((unsigned)((M + kRouteWaves - 1) / kRouteWaves)); }

template <int DT, int V>
struct RouteLaunch {
  static hipError_t run(const RouteArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((route_kernel<DT, V>), route_grid(a.M), dim3(64 * kRouteWaves), 0, s, a);
    return hipGetLastError();
  }
};
template <int DT, int V>
struct RouteBackwardLaunch {
  static hipError_t run(const RouteBackwardArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((route_backward_kernel<DT, V>), route_grid(a.M), dim3(64 * kRouteWaves), 0, s, a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) { return by_type_and_size<RouteLaunch>(a, s); }
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s) {
  return by_type_and_size<RouteBackwardLaunch>(a, s);
}

}  // namespace w4a16
