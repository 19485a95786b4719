// Gradients of the projection with low-rank adapters: what the host lays out
// and the kernels share.
#pragma once

#include "w4a16_internal.h"

namespace w4a16 {

// Tokens in the order of their adapters: seg[s] .. seg[s + 1] are the places
// in perm of the tokens of adapter s, in token order.
struct PrepArgs {
  const int32_t* ids;
  int32_t* perm;        // [M]
  int32_t* seg;         // [S + 1]
  const uint16_t* la;   // [S][R][K]
  const uint16_t* lb;   // [S][N][R]
  uint16_t* la_t;       // [S][K][R]
  uint16_t* lb_t;       // [S][R][np], zero past N
  const uint16_t* dy;   // [M][N]
  uint16_t* dy_pad;     // [M][np], zero past N; NULL: dy's rows are used as they are
  uint32_t* zero;       // zero_words words set to zero
  int zero_words;
  int M, N, K, S, R, np;
};
hipError_t launch_prep(const PrepArgs& a, hipStream_t s);

// out_s[c, r] = sum over the tokens m of adapter s of v[m, c] * alpha_s * w[m, r]
struct OuterProblem {
  const uint16_t* v;  // [M][ld]
  const float* w;     // [M][R]
  uint16_t* out;      // [S][R][C] (by_rank) or [S][C][R]
  int ld, C, by_rank;
};
struct OuterArgs {
  OuterProblem p[2];
  const int32_t* perm;
  const int32_t* seg;
  const float* alpha;  // [S] or NULL
  float* partial;
  uint32_t* counters;  // outer_counters(...) zeros
  int M, S, R, dtype;
};
struct OuterPlan {
  int tokens;        // of one workgroup, a multiple of 128
  int splits;        // token ranges at most
  int rc, rgroups;   // 16-rank blocks of a workgroup, groups of them
  int tiles[2];      // 128-column tiles of the two problems
};
OuterPlan plan_outer(int64_t M, int64_t C0, int64_t C1, int S, int R, int cu_count);
size_t outer_partial_bytes(const OuterPlan& p, int64_t M);
size_t outer_counter_bytes(const OuterPlan& p, int S);
hipError_t launch_outer(const OuterArgs& a, const OuterPlan& p, hipStream_t s);

// dx[m, k] = sum over n of dy[m, n] * W[n, k] (+ the adapters' term)
struct DxArgs {
  const uint16_t* dy;  // [M][ldy], ldy a multiple of 8
  const int32_t* wq;
  const void* scales;
  const int32_t* zp;
  void* dx;            // [M][K]
  const void* zeros;   // 16 zero bytes on the device
  float* partial;
  int64_t M, N, K;
  int ldy, group, dtype, sG, gmul;
};
struct DxPlan {
  int mw;              // 32-token blocks of a wave: a tile is 64 mw tokens x 256 k
  int splits;          // ranges of n
  int steps_per_split; // of 64 n
  int tiles_k, tiles;
};
DxPlan plan_dx(int64_t M, int64_t N, int64_t K, int cu_count);
size_t dx_partial_bytes(const DxPlan& p, int64_t M, int64_t K);
hipError_t launch_dx(const DxArgs& a, const DxPlan& p, const LoraTerm& lora, hipStream_t s);
// y = sum of the splits' fp32 partials [split][M][np] in split order, + bias, one rounding
hipError_t launch_splitk_reduce(int dtype, const float* partial, const uint16_t* bias, uint16_t* y, int M, int N, int np,
                                int splits, hipStream_t s);

}  // namespace w4a16
