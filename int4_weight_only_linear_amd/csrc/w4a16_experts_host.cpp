// Host side of the experts' operators (include/w4a16.h): argument checks,
// workspaces and launches of routing, 8-bit quantisation and 8-bit products.
#include "w4a16_experts.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "w4a16_host.hpp"
#include "w4a16_internal.h"

namespace {

using w4a16::act_bytes;
using w4a16::aligned;
using w4a16::DeviceInfo;
using w4a16::device_info;
using w4a16::fail;
using w4a16::fp8_columns;
using w4a16::fp8_scales;
using w4a16::ok;
using w4a16::overlap;
using w4a16::round256;

// a launch has fewer than 2^32 threads
constexpr int64_t kMaxRouteTokens = int64_t(1) << 25;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxValues = int64_t(1) << 34;  // of a tensor to quantise

w4a16_status launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
}

size_t float_bytes(int32_t dtype) { return dtype == W4A16_F32 ? 4 : 2; }

w4a16_status check_route(const char* what, int64_t M, int64_t E, int64_t topk, int32_t dtype, int32_t score, double scale) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16 && dtype != W4A16_F32)
    return fail(W4A16_ERR_INVALID_ARG, "%s: logits must be fp16, bf16 or fp32, got %d", what, (int)dtype);
  if (score != W4A16_SCORE_SOFTMAX && score != W4A16_SCORE_SIGMOID)
    return fail(W4A16_ERR_INVALID_ARG, "%s: unknown score %d", what, (int)score);
  if (M < 0 || E < 1 || topk < 1 || topk > E)
    return fail(W4A16_ERR_INVALID_ARG, "%s: need M >= 0 and 1 <= topk <= E (M=%lld E=%lld topk=%lld)", what, (long long)M,
                (long long)E, (long long)topk);
  if (E > w4a16::kMaxExperts || topk > w4a16::kMaxTopk || M > kMaxRouteTokens)
    return fail(W4A16_ERR_UNSUPPORTED, "%s: at most %d experts, topk %d and %lld tokens (M=%lld E=%lld topk=%lld)", what,
                w4a16::kMaxExperts, w4a16::kMaxTopk, (long long)kMaxRouteTokens, (long long)M, (long long)E, (long long)topk);
  if (!std::isfinite(scale)) return fail(W4A16_ERR_INVALID_ARG, "%s: the scale must be finite", what);
  return ok();
}

// the sizes of an 8-bit product of `rows` rows
w4a16_status check_fp8_sizes(const char* what, int64_t rows, int64_t N, int64_t K, int32_t x_dtype, int32_t scale_dtype,
                             int32_t dtype, int32_t transpose) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "%s: outputs must be fp16 (0) or bf16 (1), got %d", what, (int)dtype);
  if (x_dtype != W4A16_E4M3 && x_dtype != dtype)
    return fail(W4A16_ERR_INVALID_ARG, "%s: x must be of the output's type or e4m3 codes, got %d", what, (int)x_dtype);
  if (scale_dtype != W4A16_F32 && scale_dtype != W4A16_E8M0)
    return fail(W4A16_ERR_INVALID_ARG, "%s: the weights' scales must be fp32 or e8m0, got %d", what, (int)scale_dtype);
  if (rows < 0 || N < 1 || K < 1)
    return fail(W4A16_ERR_INVALID_ARG, "%s: need M >= 0, N >= 1 and K >= 1 (N=%lld K=%lld)", what, (long long)N, (long long)K);
  if ((transpose ? N : K) % 16)
    return fail(W4A16_ERR_UNSUPPORTED, "%s: a row of the weights must hold a multiple of 16 codes, got %lld", what,
                (long long)(transpose ? N : K));
  // codes of x and of one layer's (expert's) weights are addressed with 32-bit offsets
  if (rows > kMaxRows || N > w4a16::kMaxK || K > w4a16::kMaxK || rows * fp8_columns(K) > 0xFFFFFFFFll || N * K > 0xFFFFFFFFll)
    return fail(W4A16_ERR_UNSUPPORTED, "%s: too large: M * K and N * K must be below 4 Gi (M=%lld N=%lld K=%lld)", what, (long long)rows,
                (long long)N, (long long)K);
  return ok();
}

struct Buffer {
  const void* p;
  size_t bytes;
};
template <int A, int B>
bool any_overlap(const Buffer (&a)[A], const Buffer (&b)[B]) {
  for (const Buffer& x : a)
    for (const Buffer& y : b)
      if (overlap(x.p, x.bytes, y.p, y.bytes)) return true;
  return false;
}

// A product's tiles, and its workspace: behind the region that every entry point
// leaves zero, the quantised x, the experts' order, and the K ranges' sums.
struct Fp8Plan {
  bool decode;
  w4a16::Fp8Tiles tiles;
  size_t codes, scales, start, order, part, bytes;
};
Fp8Plan plan_fp8(int64_t rows, int64_t slots, int64_t E, int64_t N, int64_t K, int32_t x_dtype, bool transpose, bool experts,
                 int cus) {
  Fp8Plan p{};
  p.decode = w4a16::fp8_decodes(slots, N, K, (int)E, experts, transpose);
  if (!p.decode) p.tiles = w4a16::plan_fp8_tiles(slots, N, K, (int)E, experts, cus);
  size_t at = w4a16::kCounterBytes;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += round256(n);
    return was;
  };
  const bool quantize = x_dtype != W4A16_E4M3;
  p.codes = take(quantize ? (size_t)(rows * fp8_columns(K)) : 0);
  p.scales = take(quantize ? (size_t)(rows * fp8_scales(K)) : 0);
  p.start = take(experts && !p.decode ? (size_t)(E + 2) * 4 : 0);
  p.order = take(experts && !p.decode ? (size_t)slots * 4 : 0);
  p.part = take(w4a16::fp8_partial_bytes(p.tiles, slots, N));
  p.bytes = at == w4a16::kCounterBytes ? 0 : at;
  return p;
}

w4a16_status check_workspace(const char* what, const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (workspace == nullptr || bytes < need))
    return fail(W4A16_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu%s", what, need, bytes,
                workspace ? "" : " (NULL)");
  if (need > 0 && !aligned(workspace, 256)) return fail(W4A16_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return ok();
}

// both products; ids NULL: one layer (topk 1, E 1)
w4a16_status fp8_product(const char* what, const void* x, const uint8_t* x_scales, const void* w, const void* w_scales,
                         const void* bias, const int32_t* ids, const float* slot_weights, void* y, int64_t M, int64_t topk,
                         int64_t E, int64_t N, int64_t K, int32_t x_dtype, int32_t scale_dtype, int32_t dtype,
                         int32_t transpose, bool per_slot, bool experts, void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t slots = M * topk, rows = per_slot ? slots : M;
  w4a16_status st = check_fp8_sizes(what, rows, N, K, x_dtype, scale_dtype, dtype, transpose);
  if (st != W4A16_OK) return st;
  if (M == 0) return ok();
  const bool codes = x_dtype == W4A16_E4M3;
  if (!x || !w || !w_scales || !y || (experts && !ids) || (codes && !x_scales))
    return fail(W4A16_ERR_INVALID_ARG, "%s: x, w, their scales%s and y must not be NULL", what, experts ? ", topk_ids" : "");
  if (!codes && x_scales) return fail(W4A16_ERR_INVALID_ARG, "%s: x_scales go with e4m3 codes", what);
  if (!aligned(w, 16) || (codes && !aligned(x, 16)))
    return fail(W4A16_ERR_ALIGNMENT, "%s: w and codes must be 16-byte aligned", what);
  if (!aligned(x, 2) || !aligned(y, 2) || (bias && !aligned(bias, 2)))
    return fail(W4A16_ERR_ALIGNMENT, "%s: x, bias and y must be 2-byte aligned", what);
  if ((scale_dtype == W4A16_F32 && !aligned(w_scales, 4)) || (x_scales && !aligned(x_scales, 4)) || (ids && !aligned(ids, 4)) ||
      (slot_weights && !aligned(slot_weights, 4)))
    return fail(W4A16_ERR_ALIGNMENT, "%s: scales, topk_ids and topk_weights must be 4-byte aligned", what);
  const int64_t blocks = ((N + 127) / 128) * ((K + 127) / 128);
  const Buffer in[] = {{x, codes ? (size_t)(rows * fp8_columns(K)) : act_bytes(rows * K)},
                       {x_scales, (size_t)(rows * fp8_scales(K))},
                       {w, (size_t)(E * N * K)},
                       {w_scales, (size_t)(E * blocks) * (scale_dtype == W4A16_F32 ? 4 : 1)},
                       {bias, act_bytes(E * N)},
                       {ids, (size_t)slots * 4},
                       {slot_weights, (size_t)slots * 4}};
  const Buffer out[] = {{y, act_bytes(slots * N)}};
  if (any_overlap(out, in)) return fail(W4A16_ERR_INVALID_ARG, "%s: y must not overlap any input", what);
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const Fp8Plan p = plan_fp8(rows, slots, E, N, K, x_dtype, transpose != 0, experts, dev->cu_count);
  if ((int64_t)p.tiles.tiles_m * p.tiles.tiles_n * p.tiles.splits > w4a16::kMaxFp8Tiles)
    return fail(W4A16_ERR_UNSUPPORTED, "%s: too large (M=%lld N=%lld)", what, (long long)slots, (long long)N);
  st = check_workspace(what, workspace, workspace_bytes, p.bytes);
  if (st != W4A16_OK) return st;
  const Buffer ws[] = {{workspace, p.bytes}};
  if (any_overlap(ws, in) || any_overlap(ws, out))
    return fail(W4A16_ERR_INVALID_ARG, "%s: the workspace must not overlap an input or an output", what);
  if (w4a16::tuning().log) {
    char plan[64] = "decode";
    if (!p.decode) std::snprintf(plan, sizeof(plan), "tile=%dx128 splits=%d steps=%d", p.tiles.bm, p.tiles.splits, p.tiles.steps);
    std::fprintf(stderr, "[w4a16] %s slots=%lld E=%lld N=%lld K=%lld %s%s%s %s\n", what, (long long)slots, (long long)E,
                 (long long)N, (long long)K, dtype == W4A16_F16 ? "f16" : "bf16", scale_dtype == W4A16_E8M0 ? " e8m0" : "",
                 transpose ? " transposed" : "", plan);
  }
  char* const base = static_cast<char*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  w4a16::Fp8Args a{};
  a.x = static_cast<const uint8_t*>(x);
  a.xs = x_scales;
  // (rows of K % 16 == 0 values: aligned where the first one is)
  const bool in_place = p.decode && !codes && aligned(x, 16) && w4a16::fp8_decode_quantizes(slots, K);
  const bool sorts = experts && !p.decode;
  int32_t* const start = reinterpret_cast<int32_t*>(base + p.start);
  int32_t* const order = reinterpret_cast<int32_t*>(base + p.order);
  if (!codes && !in_place) {
    uint8_t* const q = reinterpret_cast<uint8_t*>(base + p.codes);
    uint8_t* const qs = reinterpret_cast<uint8_t*>(base + p.scales);
    const hipError_t e = sorts ? w4a16::launch_fp8_quantize_and_order(x, q, qs, rows, K, dtype, ids, start, order, (int)slots, (int)E, s)
                               : w4a16::launch_fp8_quantize(x, q, qs, rows, K, dtype, s);
    if (e != hipSuccess) return launched(e);
    a.x = q;
    a.xs = qs;
  } else if (sorts) {
    const hipError_t e = w4a16::launch_expert_order(ids, start, order, (int)slots, (int)E, s);
    if (e != hipSuccess) return launched(e);
  }
  a.w = static_cast<const uint8_t*>(w);
  a.ws = w_scales;
  a.bias = bias;
  a.y = y;
  a.M = slots;
  a.N = N;
  a.K = K;
  a.dtype = dtype;
  a.e8m0 = scale_dtype == W4A16_E8M0;
  a.transpose = transpose != 0;
  a.slot_weights = slot_weights;
  a.E = (int)E;
  a.topk = per_slot ? 1 : (int)topk;
  if (p.decode)
    return launched(w4a16::launch_fp8_decode(a, in_place ? x : a.x, in_place ? dtype : (int)W4A16_E4M3, ids, s));
  if (sorts) {
    a.start = start;
    a.order = order;
  }
  a.part = reinterpret_cast<float*>(base + p.part);
  return launched(w4a16::launch_fp8_gemm(a, p.tiles, s));
}

}  // namespace

extern "C" {

w4a16_status w4a16_route(const void* logits, const float* bias, float* weights, int32_t* ids, int64_t M, int64_t E,
                         int64_t topk, int64_t groups, int64_t topk_groups, int64_t group_top, int32_t dtype, int32_t score,
                         int32_t renormalize, double scale, void* stream) {
  w4a16_status st = check_route("route", M, E, topk, dtype, score, scale);
  if (st != W4A16_OK) return st;
  if (groups < 1 || groups > w4a16::kMaxGroups || E % groups || topk_groups < 1 || topk_groups > groups)
    return fail(W4A16_ERR_INVALID_ARG, "route: need 1 <= topk_groups <= groups <= %d and E a multiple of groups (E=%lld groups=%lld topk_groups=%lld)",
                w4a16::kMaxGroups, (long long)E, (long long)groups, (long long)topk_groups);
  if ((group_top != 1 && group_top != 2) || group_top > E / groups)
    return fail(W4A16_ERR_INVALID_ARG, "route: a group is ranked by its largest or its two largest scores, got group_top=%lld", (long long)group_top);
  if (topk > topk_groups * (E / groups))
    return fail(W4A16_ERR_INVALID_ARG, "route: topk=%lld experts out of %lld groups of %lld", (long long)topk, (long long)topk_groups,
                (long long)(E / groups));
  if (M == 0) return ok();
  if (!logits || !weights || !ids) return fail(W4A16_ERR_INVALID_ARG, "route: logits, weights and ids must not be NULL");
  if (!aligned(logits, float_bytes(dtype)) || (bias && !aligned(bias, 4)) || !aligned(weights, 4) || !aligned(ids, 4))
    return fail(W4A16_ERR_ALIGNMENT, "route: a pointer is not aligned to its elements");
  const Buffer in[] = {{logits, (size_t)(M * E) * float_bytes(dtype)}, {bias, (size_t)E * 4}};
  const Buffer out[] = {{weights, (size_t)(M * topk) * 4}, {ids, (size_t)(M * topk) * 4}};
  if (any_overlap(out, in) || overlap(out[0].p, out[0].bytes, out[1].p, out[1].bytes))
    return fail(W4A16_ERR_INVALID_ARG, "route: weights and ids must not overlap an input or each other");
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const w4a16::RouteArgs a{logits, bias, weights, ids, M, (int)E, (int)topk, (int)groups, (int)topk_groups,
                           groups > 1 ? (int)group_top : 1, dtype, score == W4A16_SCORE_SIGMOID, renormalize != 0, scale};
  return launched(w4a16::launch_route(a, static_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_route_backward(const float* dweights, const void* logits, const int32_t* ids, void* dlogits, int64_t M,
                                  int64_t E, int64_t topk, int32_t dtype, int32_t score, int32_t renormalize, double scale,
                                  void* stream) {
  w4a16_status st = check_route("route_backward", M, E, topk, dtype, score, scale);
  if (st != W4A16_OK) return st;
  if (M == 0) return ok();
  if (!dweights || !logits || !ids || !dlogits)
    return fail(W4A16_ERR_INVALID_ARG, "route_backward: dweights, logits, ids and dlogits must not be NULL");
  if (!aligned(logits, float_bytes(dtype)) || !aligned(dlogits, float_bytes(dtype)) || !aligned(dweights, 4) || !aligned(ids, 4))
    return fail(W4A16_ERR_ALIGNMENT, "route_backward: a pointer is not aligned to its elements");
  const size_t lbytes = (size_t)(M * E) * float_bytes(dtype);
  const Buffer in[] = {{logits, lbytes}, {dweights, (size_t)(M * topk) * 4}, {ids, (size_t)(M * topk) * 4}};
  const Buffer out[] = {{dlogits, lbytes}};
  if (any_overlap(out, in)) return fail(W4A16_ERR_INVALID_ARG, "route_backward: dlogits must not overlap an input");
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const w4a16::RouteBackwardArgs a{dweights, logits, ids, dlogits, M, (int)E, (int)topk, dtype, score == W4A16_SCORE_SIGMOID,
                                   renormalize != 0, scale};
  return launched(w4a16::launch_route_backward(a, static_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_minifloat_quantize(const void* x, void* codes, uint8_t* scales, int64_t M, int64_t K, int32_t dtype, void* stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "minifloat_quantize: x must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (M < 0 || K < 1) return fail(W4A16_ERR_INVALID_ARG, "minifloat_quantize: need M >= 0 and K >= 1 (M=%lld K=%lld)", (long long)M, (long long)K);
  if (M > kMaxRows || K > w4a16::kMaxK || M * fp8_scales(K) > kMaxValues / 128)
    return fail(W4A16_ERR_UNSUPPORTED, "minifloat_quantize: too large (M=%lld K=%lld)", (long long)M, (long long)K);
  if (M == 0) return ok();
  if (!x || !codes || !scales) return fail(W4A16_ERR_INVALID_ARG, "minifloat_quantize: x, codes and scales must not be NULL");
  if (!aligned(x, 2) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(W4A16_ERR_ALIGNMENT, "minifloat_quantize: x must be 2-byte, codes 16-byte and scales 4-byte aligned");
  const Buffer in[] = {{x, act_bytes(M * K)}};
  const Buffer out[] = {{codes, (size_t)(M * fp8_columns(K))}, {scales, (size_t)(M * fp8_scales(K))}};
  if (any_overlap(out, in) || overlap(out[0].p, out[0].bytes, out[1].p, out[1].bytes))
    return fail(W4A16_ERR_INVALID_ARG, "minifloat_quantize: codes and scales must not overlap x or each other");
  const DeviceInfo* dev = nullptr;
  w4a16_status st = device_info(&dev);
  if (st != W4A16_OK) return st;
  return launched(w4a16::launch_fp8_quantize(x, static_cast<uint8_t*>(codes), scales, M, K, dtype, static_cast<hipStream_t>(stream)));
}

size_t w4a16_minifloat_linear_workspace_size(int64_t M, int64_t N, int64_t K, int32_t x_dtype, int32_t transpose) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxRows || N > w4a16::kMaxK || K > w4a16::kMaxK) return 0;
  return plan_fp8(M, M, 1, N, K, x_dtype, transpose != 0, false, w4a16::planning_cus()).bytes;
}

w4a16_status w4a16_minifloat_linear(const void* x, const uint8_t* x_scales, const void* w, const void* w_scales, const void* bias,
                              void* y, int64_t M, int64_t N, int64_t K, int32_t x_dtype, int32_t scale_dtype, int32_t dtype,
                              int32_t transpose, void* workspace, size_t workspace_bytes, void* stream) {
  return fp8_product("minifloat_linear", x, x_scales, w, w_scales, bias, nullptr, nullptr, y, M, 1, 1, N, K, x_dtype, scale_dtype, dtype,
                     transpose, false, false, workspace, workspace_bytes, stream);
}

size_t w4a16_minifloat_moe_workspace_size(int64_t M, int64_t topk, int64_t E, int64_t N, int64_t K, int32_t x_dtype,
                                    int32_t transpose, int32_t x_per_slot) {
  if (M <= 0 || topk <= 0 || E <= 0 || N <= 0 || K <= 0 || M > kMaxRows || topk > kMaxRows / M || E > w4a16::kMaxExperts ||
      N > w4a16::kMaxK || K > w4a16::kMaxK)
    return 0;
  return plan_fp8(x_per_slot ? M * topk : M, M * topk, E, N, K, x_dtype, transpose != 0, true, w4a16::planning_cus()).bytes;
}

w4a16_status w4a16_minifloat_moe_linear(const void* x, const uint8_t* x_scales, const void* w, const void* w_scales,
                                  const void* bias, const int32_t* topk_ids, const float* topk_weights, void* y, int64_t M,
                                  int64_t topk, int64_t E, int64_t N, int64_t K, int32_t x_dtype, int32_t scale_dtype,
                                  int32_t dtype, int32_t transpose, int32_t x_per_slot, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (M < 0 || topk < 1 || E < 1)
    return fail(W4A16_ERR_INVALID_ARG, "minifloat_moe_linear: need M >= 0, topk >= 1 and E >= 1 (M=%lld topk=%lld E=%lld)", (long long)M,
                (long long)topk, (long long)E);
  if (E > w4a16::kMaxExperts || M > kMaxRows || (M > 0 && topk > kMaxRows / M))
    return fail(W4A16_ERR_UNSUPPORTED, "minifloat_moe_linear: at most %d experts and %lld slots (M=%lld topk=%lld E=%lld)",
                w4a16::kMaxExperts, (long long)kMaxRows, (long long)M, (long long)topk, (long long)E);
  return fp8_product("minifloat_moe_linear", x, x_scales, w, w_scales, bias, topk_ids, topk_weights, y, M, topk, E, N, K, x_dtype,
                     scale_dtype, dtype, transpose, x_per_slot != 0, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
