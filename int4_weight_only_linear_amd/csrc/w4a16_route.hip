// Routing of tokens to experts and its gradient (include/w4a16.h, w4a16_route):
//   s = softmax(l) or sigmoid(l), key = s + bias, the largest keys of the groups kept,
//   w = s of those, over their sum where asked, times a scale.
// Every choice is that of keys in 64 bits; equal keys go to the lower expert.
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

// A row by one wave, keys in 64 bits, V experts a lane (expert 64 v + lane): what
// rows of more than 512 experts or 16 choices take, those whose groups are not a
// power of two of whole lanes in the sixteen-lane form, and single rows of equal
// keys.  Bound by the vector unit (160 experts: 1225 instructions a row): 16384 rows
// of 160 experts in 8 groups 41 us, of 60 in 4 27, of 1024 88; 32 choices of 256
// 171; with sixteen lanes a row 128 experts in 8 groups take 8.8, 256 14.5;
// keys [64 V] and group_key [kMaxGroups] are the wave's own LDS.
template <int DT, int V>
__device__ void route_row(const RouteArgs& a, int64_t m, double* keys, double* group_key) {
  const int lane = threadIdx.x & 63;
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
    for (int v = 0; v < V; ++v) keys[64 * v + lane] = key[v];
    wave_lds_fence();
    double mine = none;
    if (lane < a.groups) {
      double first = none, second = none;
      for (int i = 0; i < per; ++i) {
        const double k = keys[lane * per + i];
        second = fmax(second, fmin(first, k));
        first = fmax(first, k);
      }
      mine = a.group_top == 2 && second > none ? first + second : first;
      group_key[lane] = mine;
    }
    wave_lds_fence();
    int rank = 0;
    if (lane < a.groups)
      for (int g = 0; g < a.groups; ++g) {
        const double k = group_key[g];
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
    a.weights[m * a.topk + lane] = nan ? __builtin_nanf("") : (float)(weight * a.scale);
    a.ids[m * a.topk + lane] = id;
  }
}

// Any number of experts: one wave a row.
template <int DT, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  __shared__ double keys[kRouteWaves][64 * V];
  __shared__ double group_key[kRouteWaves][kMaxGroups];
  const int wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (m < a.M) route_row<DT, V>(a, m, keys[wave], group_key[wave]);  // (waves share nothing)
}

// ---- sixteen lanes a row, four rows a wave ----------------------------------------
// Lane c of a row holds its experts V c .. V c + V - 1.

// The lane's part of a row, minus infinity past the last expert.  All of its loads
// are issued at once (past the end: of the last one's place; behind a condition
// each would be waited for alone).  WHOLE: rows are whole 16-byte pieces.
template <int DT, int V, bool WHOLE>
__device__ __forceinline__ void load_part(const void* values, int64_t row, int c, int E, float (&l)[V]) {
  constexpr int PER = DT == DT_F32 ? 4 : 8;  // values of a piece
  constexpr float none = -__builtin_inff();
  if constexpr (WHOLE && V % PER == 0) {
    u32x4 w[V / PER];
#pragma unroll
    for (int q = 0; q < V / PER; ++q)
      w[q] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(values) + (row * E + min(V * c + PER * q, E - PER)) * (16 / PER));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t word = w[v / PER][v % PER * 4 / PER];  // (a bit cast of the element itself takes element 0)
      float x;
      if constexpr (DT == DT_F32) x = __builtin_bit_cast(float, word);
      else x = act_to_f32<DT>((uint16_t)(word >> (16 * (v & 1))));
      l[v] = V * c + v < E ? x : none;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = load_logit<DT>(values, row * E + min(V * c + v, E - 1));
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = V * c + v < E ? l[v] : none;
  }
}

// whether any lane of this lane's row says so
__device__ __forceinline__ bool row_any(bool b) { return (__ballot(b) >> (threadIdx.x & 48)) & 0xFFFF; }

// Moves between the sixteen lanes of a row, in the vector unit.
constexpr int dpp_rotate(int n) { return 0x120 + n; }
constexpr int kDppNext = 0xB1, kDppNextPair = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;
template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  if constexpr (sizeof(T) == 8) {
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 15, 15, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 15, 15, true);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 15, 15, true));
  }
}
// over the sixteen lanes of a row; every lane gets the same
template <typename T, typename F>
__device__ __forceinline__ T row_all(T v, F&& f) {
  v = f(v, dpp<dpp_rotate(8)>(v));
  v = f(v, dpp<dpp_rotate(4)>(v));
  v = f(v, dpp<dpp_rotate(2)>(v));
  return f(v, dpp<dpp_rotate(1)>(v));
}
__device__ __forceinline__ float row_max(float v) { return row_all(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float row_min(float v) { return row_all(v, [](float a, float b) { return fminf(a, b); }); }
__device__ __forceinline__ int row_max(int v) { return row_all(v, [](int a, int b) { return max(a, b); }); }
template <typename T>
__device__ __forceinline__ T row_sum(T v) { return row_all(v, [](T a, T b) { return a + b; }); }
// order kept, compared as an integer (no zero of either sign apart, no NaN), and back
__device__ __forceinline__ int ordered(float v) {
  const int b = __builtin_bit_cast(int, v + 0.f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_ordered(int b) { return __builtin_bit_cast(float, b ^ ((b >> 31) & 0x7FFFFFFF)); }
// a tree of V terms
template <int V, typename T>
__device__ __forceinline__ T part_sum(const T (&x)[V]) {
  T t[V];
#pragma unroll
  for (int v = 0; v < V; ++v) t[v] = x[v];
#pragma unroll
  for (int n = V / 2; n; n /= 2)
#pragma unroll
    for (int v = 0; v < n; ++v) t[v] += t[v + n];
  return t[0];
}
// a or b, both by value (a choice of elements would become an index into the array)
template <typename T>
__device__ __forceinline__ T pick(bool which, T a, T b) { return which ? a : b; }

// The two largest so far
template <typename T>
struct TwoLargest {
  T first = -__builtin_inf(), second = -__builtin_inf();
  __device__ __forceinline__ void add(T k) {
    second = max(second, min(first, k));
    first = max(first, k);
  }
  // over `lanes` neighbouring lanes
  __device__ __forceinline__ void join(int lanes) {
    auto with = [&](auto ctrl) {
      const T f = dpp<decltype(ctrl)::value>(first), s = dpp<decltype(ctrl)::value>(second);
      second = max(max(second, s), min(first, f));
      first = max(first, f);
    };
    if (lanes > 1) with(std::integral_constant<int, kDppNext>{});
    if (lanes > 2) with(std::integral_constant<int, kDppNextPair>{});
    if (lanes > 4) with(std::integral_constant<int, kDppMirror8>{});
    if (lanes > 8) with(std::integral_constant<int, kDppMirror16>{});
  }
  __device__ __forceinline__ T key(int top) const { return top == 2 && second > -__builtin_inf() ? first + second : first; }
};
// Lanes of a row whose key is before this lane's: larger, or equal and `at` lower.
// step 2, 4, ..: one lane of that many alone, the others hold the same.
template <typename T>
__device__ __forceinline__ int rank_of(T key, int at, int step) {
  int ahead = 0;
  static_for<1, 16>([&](auto R) {
    constexpr int r = decltype(R)::value;
    if (r & (step - 1)) return;
    const T other = dpp<dpp_rotate(r)>(key);
    const int oat = dpp<dpp_rotate(r)>(at);
    ahead += other > key || (other == key && oat < at);
  });
  return ahead;
}

// Batcher's network of odd and even merges for V values.
template <int V>
struct SortNetwork {
  int n = 0, low[200] = {}, high[200] = {};
  constexpr SortNetwork() {
    for (int p = 1; p < V; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < V; j += 2 * k)
          for (int i = j; i < j + k && i + k < V; ++i)
            if (i / (2 * p) == (i + k) / (2 * p)) low[n] = i, high[n] = i + k, ++n;
  }
};
// the largest first
template <int V>
__device__ __forceinline__ void sort_part(int (&x)[V]) {
  constexpr SortNetwork<V> net;
  static_for<0, net.n>([&](auto I) {
    constexpr SortNetwork<V> with;
    constexpr int lo = with.low[decltype(I)::value], hi = with.high[decltype(I)::value];
    const int a = x[lo], b = x[hi];
    x[lo] = max(a, b);
    x[hi] = min(a, b);
  });
}

// Keys are formed in 32 bits; what hangs on less than their error is decided by
// the 64-bit keys of the experts concerned, so that every choice is that of the
// 64-bit keys:
//  - groups: those of the experts that may be among a group's largest;
//  - experts: the choice goes on until the next key is clearly below (lane j holds
//    the j-th expert), and those found are ranked by their 64-bit keys, of which
//    the weights need the scores anyway;
//  - a row with more than sixteen in question (a row of equal scores): route_row.
// The error is below 2^-22 (1 + |key|).  Sigmoid, in units of 2^-23: with t the
// exponential, 1 / (1 + t) changes by t / (1 + t)^2 <= 1/4 of t's relative error, of
// one unit by the instruction, and by at most 0.23 of that of the exponent x (x t /
// (1 + t)^2 <= 0.23), of one unit by log2(e)'s rounding and the product's; half a
// unit by the sum's rounding and one by the reciprocal's: 1.98.  Softmax rounds both
// sides and the quotient, half a unit each.  The bias is added with 2^-24 |key|.
// A lane sorts its keys once, as integers whose lowest bits name the place (V units
// of 2^-23 |key| more), so that a round of the choice looks at sixteen first places
// (rounds that search all V and take one out: 2 us more at 16384 x 256).
// Bound by the vector unit: 16384 x 256 in fp32 with 8 groups 14.5 us, 1.2 TB/s, of
// which a launch is 2.4; a wave of four rows issues 1400 vector instructions, and
// those of a SIMD's four waves take 23000 of the 24200 cycles that they live.  4 rows
// take 3.7 us in the kernel.
template <int DT, int V, bool WHOLE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_quick_kernel(RouteArgs a) {
  constexpr int V64 = V > 4 ? V / 4 : 1;
  __shared__ double keys[kRouteWaves][64 * V64];
  __shared__ double group_key[kRouteWaves][kMaxGroups];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15;
  const int64_t m0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * 4;
  if (m0 >= a.M) return;  // (waves share nothing)
  const bool there = m0 + (lane >> 4) < a.M;
  const int64_t m = there ? m0 + (lane >> 4) : a.M - 1;
  constexpr float none = -__builtin_inff();
  constexpr float kNear = 0x1.1p-21f;  // two keys' errors, and that of their difference
  float l[V], key[V], b[V];
  load_part<DT, V, WHOLE>(a.logits, m, c, a.E, l);
  if (a.bias) load_part<DT_F32, V, WHOLE>(a.bias, 0, c, a.E, b);
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    nan |= l[v] != l[v];
    l[v] = l[v] == l[v] ? l[v] : none;
  }
  nan = row_any(nan);
  const bool by_logit = !a.bias && a.group_top == 1;
  float top = none;
  double sum = 1;
  auto exp_of = [&](float x) {  // (equal to the largest: 1, also where that is infinite)
    return x == none ? 0.0 : (x == top ? 1.0 : exp((double)x - (double)top));
  };
  auto score_of = [&](float x) { return a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : (sum > 0 ? exp_of(x) / sum : 0.0); };
  if (!a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
    top = row_max(top);
    double e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = exp_of(l[v]);
    sum = row_sum(part_sum<V>(e));
    const float whole = (float)sum;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = whole > 0 ? (float)e[v] / whole : 0.f;
  } else if (!by_logit) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[v] * -1.44269504f));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (by_logit) key[v] = l[v];
    else if (a.bias) key[v] += b[v];
    if (!(l[v] > none) || !(key[v] > none)) key[v] = none;
  }
  if (a.groups > 1) {
    const int lanes = a.E / a.groups / V;  // of a group: 1, 2, 4, 8 or 16
    TwoLargest<float> two;
#pragma unroll
    for (int v = 0; v < V; ++v) two.add(key[v]);
    two.join(lanes);
    const float mine = two.key(a.group_top);
    // (lanes past the last expert have no key and the highest places: behind)
    bool kept = rank_of(mine, c, lanes) < a.topk_groups;
    const float low = row_min(kept ? mine : __builtin_inff()), high = row_max(kept ? none : mine);
    // (the sum of two keys may be far smaller than they are)
    const float size = row_max(two.first > none ? fabsf(two.first) + (two.second > none ? fabsf(two.second) : 0.f) : 0.f);
    const bool close = !by_logit && high > none && !(low - high > 1.25f * kNear * (2 + size));
    if (__ballot(close)) {
      const float least = a.group_top == 2 ? two.second : two.first, from = least - kNear * (1 + fabsf(least));
      uint32_t concerned = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) concerned |= key[v] > none && !(key[v] < from) ? 1u << v : 0u;
      TwoLargest<double> exact;
      while (__ballot(concerned)) {
        const int at = concerned ? __builtin_ctz(concerned) : -1;
        concerned &= concerned - 1;
        float x = none;
#pragma unroll
        for (int v = 0; v < V; ++v) x = pick(v == at, l[v], x);
        if (at >= 0) exact.add(score_of(x) + (a.bias ? (double)a.bias[V * c + at] : 0.0));
      }
      exact.join(lanes);
      kept = rank_of(exact.key(a.group_top), c, lanes) < a.topk_groups;
    }
    if (!kept) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = none;
    }
  }
  // the largest key, then the next
  constexpr int empty = INT32_MIN;
  int left[V];
#pragma unroll
  for (int v = 0; v < V; ++v) left[v] = pick(key[v] > none, (ordered(key[v]) & -V) | (V - 1 - v), empty);
  sort_part<V>(left);
  // logits of 16 bits are whole in what is left of 32
  const bool whole_keys = by_logit && DT != DT_F32;
  int id = -1;
  float before = __builtin_inff();
  bool doubt = false, open = true;  // open: the j-th may be as large as the last one chosen
  for (int j = 0;; ++j) {
    const int head = left[0] & -V, most = row_max(head);  // (INT32_MIN stays itself)
    const float k = of_ordered(most);
    const float near = V * 0x1p-23f * fabsf(k) + 0x1p-120f + (by_logit ? 0.f : kNear * (1 + fabsf(k)));
    const bool close = !whole_keys && j > 0 && most != empty && !(before - k > near);
    if (j >= a.topk) {
      open &= close;
      if (j == 16 || !__ballot(open)) break;
    }
    doubt |= open && close;
    before = k;
    const uint32_t hits = (uint32_t)(__ballot(head == most) >> (lane & 48)) & 0xFFFF;
    const bool taken = c == __builtin_ctz(hits);  // the lowest lane: the lowest experts
    const int e = row_max(taken ? V * c + V - 1 - (left[0] & (V - 1)) : -1);
    if (c == j && open && most != empty) id = e;
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) left[v] = pick(taken, left[v + 1], left[v]);
    left[V - 1] = pick(taken, empty, left[V - 1]);
  }
  double weight = 0;
  int slot = c;
  if (id >= 0) weight = score_of(load_logit<DT>(a.logits, m * a.E + id));
  if (__ballot(doubt)) {
    double k = none;
    if (id >= 0) k = by_logit ? (double)load_logit<DT>(a.logits, m * a.E + id) : weight + (a.bias ? (double)a.bias[id] : 0.0);
    slot = rank_of(k, id >= 0 ? id : kMaxExperts + c, 1);
  }
  if (slot >= a.topk) weight = 0;
  if (a.renormalize) {
    const double total = row_sum(weight);
    weight = total > 0 ? weight / total : 0.0;
  }
  // (rows that are done again below are stored there alone: by other lanes of this wave, whose stores nothing would
  // order behind these)
  if (slot < a.topk && there && !open) {
    a.weights[m * a.topk + slot] = nan ? __builtin_nanf("") : (float)(weight * a.scale);
    a.ids[m * a.topk + slot] = id;
  }
  uint64_t again = __ballot(open && c == 0 && there);
  while (again) {
    const int r = __builtin_ctzll(again) >> 4;
    again &= again - 1;
    route_row<DT, V64>(a, m0 + r, keys[wave], group_key[wave]);
  }
}

// The gradient, sixteen lanes a row: lane j has slot j's gradient (and those of
// slots j + 16, ..), and every lane adds what meets its own experts.  Lanes take
// turns over a row's pieces, so that a row's loads and stores are whole lines (parts
// of 64 bytes a lane: 13.4 us at 16384 x 256).  Softmax without renormalisation (ROW)
// is formed over the whole row, in fp32; otherwise only chosen experts have
// gradients, from scores in 64 bits.  Renormalised, with the shares r_j = p_j / S and c the sum
// of r_j g_j, d l is r_j (g_j - c), times 1 - s_j for sigmoid (softmax's sum of
// s_k d s_k is c - c); all p_j of a row may lie below fp32's range and their shares
// be ordinary numbers.  A kernel for each of the two, since one with both held the
// registers of both (16384 rows of 1024 experts, sigmoid: 38.5 us, 34.0 apart).  Memory and the slots' chain bound it: 16384 x 256 in fp32 10.2 us, 3.4 TB/s.
template <int DT, int V, bool WHOLE, bool ROW>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_kernel(RouteBackwardArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, base = lane & 48;
  const int64_t row = ((int64_t)blockIdx.x * kRouteWaves + wave) * 4 + (lane >> 4);
  if (row - (lane >> 4) >= a.M) return;
  const int64_t m = min(row, a.M - 1);
  constexpr int PER = DT == DT_F32 ? 4 : 8, P = WHOLE && V % PER == 0 ? PER : 1;  // experts of a piece
  auto place = [](int v) { return v / P * 16 * P + v % P; };  // the lane's v-th expert is place(v) + P c
  float s[V], ds[V];
  u32x4 w[V / P];
#pragma unroll
  for (int i = 0; i < V / P; ++i) {
    const int64_t at = m * a.E + min(place(P * i) + P * c, a.E - P);
    if constexpr (P > 1) w[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.logits) + at * (16 / PER));
    else s[i] = load_logit<DT>(a.logits, at);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (P > 1) {
      const uint32_t word = w[v / PER][v % PER * 4 / PER];
      if constexpr (DT == DT_F32) s[v] = __builtin_bit_cast(float, word);
      else s[v] = act_to_f32<DT>((uint16_t)(word >> (16 * (v & 1))));
    }
    if (place(v) + P * c >= a.E) s[v] = -__builtin_inff();
  }
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) nan |= s[v] != s[v], ds[v] = 0.f;
  nan = row_any(nan);
  float top = -__builtin_inff(), total = 1.f;
  if (ROW || !a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, s[v]);
    top = row_max(top);
  }
  if constexpr (ROW) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = s[v] == -__builtin_inff() ? 0.f : (s[v] == top ? 1.f : expf(s[v] - top));
    total = row_sum(part_sum<V>(s));
    // (the reciprocal and what it lacks: a score is rounded once)
    const float inv = total > 0.f ? 1.f / total : 0.f, lack = __builtin_fmaf(-total, inv, 1.f) * inv;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = __builtin_fmaf(s[v], inv, s[v] * lack);
  }
  // Sixteen slots at a time, lane c the c-th of them: with shares once for the scores' sum and the mean of the
  // gradients, then for the gradients (the first sixteen are kept for that where there are no others).
  const int rounds = (a.topk + 15) / 16;
  int id = -1;
  float g = 0.f;
  double p = 0, rest = 1, sum = 0, mean = 0;
  const bool shares = !ROW && a.renormalize;
  for (int r = shares ? 0 : rounds; r < 2 * rounds; ++r) {
    const int j0 = 16 * (r < rounds ? r : r - rounds), j = j0 + c;
    if (r < rounds || rounds > 1 || !shares) {
      id = j < a.topk ? a.ids[m * a.topk + j] : -1;
      if (id < 0 || id >= a.E) id = -1;
      g = p = 0;
      if (id >= 0) {
        g = (float)((double)a.dweights[m * a.topk + j] * a.scale);
        if constexpr (!ROW) {
          const float l = load_logit<DT>(a.logits, m * a.E + id);
          const double t = exp(a.sigmoid ? -(double)l : (double)l - (double)top);
          if (a.sigmoid) {
            p = 1.0 / (1.0 + t);
            rest = t == __builtin_inf() ? 1.0 : t * p;  // 1 - p, without a difference
          } else {
            p = l == -__builtin_inff() ? 0.0 : (l == top ? 1.0 : t);
          }
          if (!shares) g = (float)((double)g * p * rest);
          p *= 0x1p60;  // (1 / sum is finite, also of subnormal scores)
        }
      }
    }
    if (r < rounds) {
      sum += p;
      mean += id >= 0 ? p * (double)g : 0.0;
      if (r + 1 < rounds) continue;
      sum = row_sum(sum);
      mean = row_sum(mean);
      const double inv = 1.0 / sum;
      mean = sum > 0 ? mean * inv : 0.0;
      sum = sum > 0 ? inv : 0.0;  // (from here on its reciprocal)
      // (0, or NaN where a gradient is not finite: softmax hands it to the whole row)
      const float others = a.sigmoid ? 0.f : (float)(mean - mean);
#pragma unroll
      for (int v = 0; v < V; ++v) ds[v] = others;
      continue;
    }
    if (shares) g = sum > 0 ? (float)(p * sum * ((double)g - mean) * rest) : 0.f;
    const int n = min(16, a.topk - j0);
    for (int k = 0; k < n; ++k) {
      const int e = __shfl(id, base + k) - P * c;
      const float gk = __shfl(g, base + k);
#pragma unroll
      for (int v = 0; v < V; ++v) ds[v] += e == place(v) ? gk : 0.f;
    }
  }
  float dot = 0.f;
  if constexpr (ROW) {
    float t[V];
#pragma unroll
    for (int v = 0; v < V; ++v) t[v] = s[v] * ds[v];
    dot = row_sum(part_sum<V>(t));
  }
  float dl[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dl[v] = nan ? __builtin_nanf("") : (ROW ? s[v] * (ds[v] - dot) : ds[v]);
  if (row >= a.M) return;
#pragma unroll
  for (int i = 0; i < V / P; ++i) {
    const int e = place(P * i) + P * c;
    if (e >= a.E) continue;
    if constexpr (P > 1) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if constexpr (DT == DT_F32) w[i][h] = __builtin_bit_cast(uint32_t, dl[P * i + h]);
        else w[i][h] = f32x2_to_act_pair<DT>(dl[P * i + 2 * h], dl[P * i + 2 * h + 1]);
      }
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.dlogits) + (m * a.E + e) * (16 / PER)) = w[i];
    } else {
      store_logit<DT>(a.dlogits, m * a.E + e, dl[i]);
    }
  }
}

dim3 rows_grid(int64_t M, int rows) { return dim3((unsigned)((M + rows - 1) / rows)); }

// f(type, experts a lane) for a type and at least E / lanes experts a lane
template <typename F>
void by_type(int dtype, F&& f) {
  if (dtype == DT_F16) f(std::integral_constant<int, DT_F16>{});
  else if (dtype == DT_BF16) f(std::integral_constant<int, DT_BF16>{});
  else f(std::integral_constant<int, DT_F32>{});
}
template <typename F>
void by_size(int E, int lanes, F&& f) {
  const int v = (E + lanes - 1) / lanes;
  if (v <= 1) f(std::integral_constant<int, 1>{});
  else if (v <= 2) f(std::integral_constant<int, 2>{});
  else if (v <= 4) f(std::integral_constant<int, 4>{});
  else if (v <= 8) f(std::integral_constant<int, 8>{});
  else if (v <= 16) f(std::integral_constant<int, 16>{});
  else if (v <= 32) f(std::integral_constant<int, 32>{});
  else f(std::integral_constant<int, 64>{});
}
int part_of(int E) {  // experts a lane of sixteen
  int v = 1;
  while (16 * v < E) v *= 2;
  return v;
}
// rows of whole 16-byte pieces
bool whole_rows(const void* p, const void* q, int E, int dtype) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q);
  return at % 16 == 0 && (size_t)E * (dtype == DT_F32 ? 4 : 2) % 16 == 0;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  // sixteen lanes a row for up to 512 experts and 16 of them chosen, where a group is a power of two of lanes
  const int v = part_of(a.E), per = a.E / a.groups;
  const bool quick = a.E <= 512 && a.topk <= 16 && (a.groups == 1 || (per % v == 0 && (per / v & (per / v - 1)) == 0 && per / v <= 16));
  const bool whole = whole_rows(a.logits, a.bias, a.E, a.dtype);
  by_type(a.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (quick)
      by_size(a.E, 16, [&](auto n) {
        constexpr int V = decltype(n)::value;
        if constexpr (V <= 32) {
          const dim3 grid = rows_grid(a.M, 4 * kRouteWaves);
          if (whole) hipLaunchKernelGGL((route_quick_kernel<DT, V, true>), grid, dim3(64 * kRouteWaves), 0, s, a);
          else hipLaunchKernelGGL((route_quick_kernel<DT, V, false>), grid, dim3(64 * kRouteWaves), 0, s, a);
        }
      });
    else
      by_size(a.E, 64, [&](auto n) {
        constexpr int V = decltype(n)::value;
        if constexpr (V <= 16)
          hipLaunchKernelGGL((route_kernel<DT, V>), rows_grid(a.M, kRouteWaves), dim3(64 * kRouteWaves), 0, s, a);
      });
  });
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s) {
  const bool whole = whole_rows(a.logits, a.dlogits, a.E, a.dtype);
  by_type(a.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_size(a.E, 16, [&](auto n) {
      constexpr int V = decltype(n)::value;
      const dim3 grid = rows_grid(a.M, 4 * kRouteWaves);
      auto go = [&](auto row) {
        constexpr bool ROW = decltype(row)::value;
        if (whole) hipLaunchKernelGGL((route_backward_kernel<DT, V, true, ROW>), grid, dim3(64 * kRouteWaves), 0, s, a);
        else hipLaunchKernelGGL((route_backward_kernel<DT, V, false, ROW>), grid, dim3(64 * kRouteWaves), 0, s, a);
      };
      if (!a.sigmoid && !a.renormalize) go(std::true_type{});
      else go(std::false_type{});
    });
  });
  return hipGetLastError();
}

}  // namespace w4a16
