// Internal interface of the experts' operators: routing of tokens to experts,
// quantisation to 8-bit floating point, and products of 8-bit weights with a
// scale for each block of 128 x 128.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

// ---- routing ------------------------------------------------------------------
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;

struct RouteArgs {
  const void* logits;  // [M, E]
  const float* bias;   // [E] or NULL
  float* weights;      // [M, topk]
  int32_t* ids;        // [M, topk]
  int64_t M;
  int E, topk, groups, topk_groups, group_top;
  int dtype, sigmoid, renormalize;
  double scale;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct RouteBackwardArgs {
  const float* dweights;  // [M, topk]
  const void* logits;     // [M, E]
  const int32_t* ids;     // [M, topk]
  void* dlogits;          // [M, E]
  int64_t M;
  int E, topk;
  int dtype, sigmoid, renormalize;
  double scale;
};
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s);

// ---- quantisation ---------------------------------------------------------------
constexpr int kFp8Block = 128;
// columns of a row of codes, and scales of a row
inline int64_t fp8_columns(int64_t K) { return (K + kFp8Block - 1) / kFp8Block * kFp8Block; }
inline int64_t fp8_scales(int64_t K) { return (K + 4 * kFp8Block - 1) / (4 * kFp8Block) * 4; }
hipError_t launch_fp8_quantize(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, int dtype,
                               hipStream_t s);

// ---- the slots in their experts' order --------------------------------------------
// start[e]: how many slots name experts below e, start[E] all that name one
// (the others follow), start[E + 1] all; order: the slots, expert by expert, in
// slot order.
hipError_t launch_expert_order(const int32_t* ids, int32_t* start, int32_t* order, int slots, int E, hipStream_t s);
// both of them
hipError_t launch_fp8_quantize_and_order(const void* x, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, int dtype,
                                         const int32_t* ids, int32_t* start, int32_t* order, int slots, int E, hipStream_t s);

// ---- products -----------------------------------------------------------------
struct Fp8Args {
  const uint8_t* x;        // codes [rows, fp8_columns(K)]
  const uint8_t* xs;       // scales [rows, fp8_scales(K)]
  const uint8_t* w;        // [E][N, K], or [E][K, N] where transposed
  const void* ws;          // [E][ceil(N / 128), ceil(K / 128)], or transposed
  const void* bias;        // [E][N] or NULL
  void* y;                 // [M, N]
  int64_t M, N, K;         // M: tokens, or slots
  int dtype;               // of y and bias
  bool e8m0, transpose;
  // experts (NULL start: one layer)
  const float* slot_weights = nullptr;
  const int32_t* start = nullptr;  // the order's
  const int32_t* order = nullptr;
  int E = 1, topk = 1;             // x row of slot s: s / topk, or s (topk 1)
  float* part = nullptr;           // fp8_partial_bytes
};
// tiles of bm tokens (experts: slots) x 128 features, and K ranges of `steps` blocks
struct Fp8Tiles {
  int bm, tiles_m, tiles_n, splits, steps;
};
constexpr int64_t kMaxFp8Tiles = int64_t(1) << 22;  // of a launch: its threads stay below 2^32
Fp8Tiles plan_fp8_tiles(int64_t M, int64_t N, int64_t K, int E, bool experts, int cus);
size_t fp8_partial_bytes(const Fp8Tiles& t, int64_t M, int64_t N);
hipError_t launch_fp8_gemm(const Fp8Args& a, const Fp8Tiles& t, hipStream_t s);

// Few tokens (experts: few slots for each): whether they are decoded, by one
// launch that takes the slots' ids without an order and either x as it is
// (x_dtype DT_F16 or DT_BF16, 16-byte aligned, where fp8_decode_quantizes says
// so: two workgroups' tokens fit a CU's LDS) or codes (any other).
bool fp8_decodes(int64_t M, int64_t N, int64_t K, int E, bool experts, bool transpose);
bool fp8_decode_quantizes(int64_t M, int64_t K);
hipError_t launch_fp8_decode(const Fp8Args& a, const void* x, int x_dtype, const int32_t* ids, hipStream_t s);

}  // namespace w4a16
