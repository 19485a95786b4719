// Gradients of the projection with low-rank adapters: what the host lays out
// and the kernels share.
#pragma once

#include "w4a16_internal.h"

namespace w4a16 {

// Tokens in the order of their adapters: the places start[s] ..
// start[s] + count[s] of `order` hold the tokens of adapter s, in token order.
// start[s] = round32(tokens of smaller adapters) + 32 s, a multiple of 32 that
// every adapter's workgroup can form by itself; places between are -1.
inline int64_t order_places(int64_t M, int64_t S) { return (M + 31) / 32 * 32 + 32 * S; }
// What dx_kernel reads beside the packed words.  Constants of every row and
// group, by group and row, in the form its conversions take (zero past N):
// fp16, per pair of rows, both scales and both -(1024 + z) as fp16 (8 bytes);
// bf16, per row, s 2^9 and -z s as fp32 (8 bytes).  And where N is no multiple
// of 64, the weights' last N % 64 rows as 64 (zero past N) in complete tiles.
struct DxPrep {
  const uint32_t* wq = nullptr;
  const uint16_t* scales = nullptr;
  const uint32_t* zp = nullptr;   // NULL: symmetric
  void* constants = nullptr;      // [G][np]; NULL: no dx wanted
  uint32_t* wq_tail = nullptr;    // [4][16 * K / 8]; NULL: no tail
  int G = 0, dtype = 0;           // scales per row
};
inline size_t dx_constant_bytes(int64_t np, int64_t G, int dtype) { return (size_t)np * (size_t)G * (dtype == 0 ? 4 : 8); }
struct PrepArgs {
  const int32_t* ids;
  int32_t* order;       // [order_places(M, S)]
  int32_t* start;       // [S]
  int32_t* count;       // [S]
  const uint16_t* la;   // [S][R][K]
  const uint16_t* lb;   // [S][N][R]
  uint16_t* la_t;       // [S][K][R]
  uint16_t* lb_t;       // [S][R][np], zero past N
  const uint16_t* dy;   // [M][N]
  uint16_t* dy_pad;     // [M][np], zero past N; NULL: dy's rows are used as they are
  uint32_t* zero;       // zero_words words set to zero
  int zero_words;
  int M, N, K, S, R, np, places;
  DxPrep dx;
};
hipError_t launch_prep(const PrepArgs& a, hipStream_t s);

// where rank r's shift stands among those of 32 places
__host__ __device__ inline int shift_at(int r) { return r / 64 * 64 + r % 16 * 4 + r % 64 / 16; }
inline int64_t shift_row(int64_t R) { return (R + 63) / 64 * 64; }

// alpha * g (the sum of its K ranges) and alpha * u as MFMA operands, value and
// remainder in the activation dtype (split_hi_lo): both by rank and place, and
// alpha * g by token.  With fp16 times a power of two (op_shift): of a token in
// g, of a rank over 32 places (one adapter's, and a step of outer_kernel) in op.
struct OperandArgs {
  const float* part;    // [splits][M][R]
  const float* u;       // [M][R]
  const int32_t* ids;
  const int32_t* order;
  const float* alpha;   // [S] or NULL
  uint16_t* g;          // [M][2][R]
  uint16_t* op[2];      // of g and of u: [2][R][places]
  int32_t* g_shift;     // [M], fp16 only
  int8_t* op_shift[2];  // [places / 32][R to 64]: shifts / 16, four ranks 16 apart together (shift_at); fp16 only
  int M, S, R, splits, places, dtype;
};
hipError_t launch_operands(const OperandArgs& a, hipStream_t s);

// out_s[c, r] = sum over the tokens m of adapter s of v[m, c] * w[m, r]
struct OuterProblem {
  const uint16_t* v;   // [M][ld]
  const uint16_t* op;  // [2][R][places]
  const int8_t* shift; // OperandArgs' op_shift
  uint16_t* out;       // [S][R][C] (by_rank) or [S][C][R]
  int ld, C, by_rank;
};
struct OuterArgs {
  OuterProblem p[2];
  const int32_t* order;
  const int32_t* start;
  const int32_t* count;
  float* partial;
  uint32_t* counters;  // outer_counter_bytes(...) of zeros
  int M, S, R, places, dtype;
};
struct OuterPlan {
  int tokens;        // of one workgroup, a multiple of 256
  int splits;        // token ranges at most
  int rc, rgroups;   // 16-rank blocks of a workgroup, groups of them
  int tiles[2];      // column tiles of the two problems
};
OuterPlan plan_outer(int64_t M, int64_t C0, int64_t C1, int S, int R, int cu_count);
size_t outer_partial_bytes(const OuterPlan& p, int64_t places);
size_t outer_counter_bytes(const OuterPlan& p, int S);
hipError_t launch_outer(const OuterArgs& a, const OuterPlan& p, hipStream_t s);

// dx[m, k] = sum over n of dy[m, n] * W[n, k] (+ the adapters' term)
struct DxArgs {
  const uint16_t* dy;  // [M][ldy], ldy a multiple of 64, zero past N
  const int32_t* wq;
  const uint32_t* wq_tail;  // DxPrep's
  const void* constants;
  void* dx;            // [M][K]
  float* partial;
  int64_t M, N, K;
  int ldy, group, dtype;  // group: k of one scale (K for per-channel scales)
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
