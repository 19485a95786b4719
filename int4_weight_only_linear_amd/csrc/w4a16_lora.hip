// The low-rank adapters' first product: u[m, r] = sum_k x[m, k] * A_a[r, k],
// a = ids[m], in fp32 (the second product is added by the projection's own
// kernels, w4a16_lora.hpp).
#include <algorithm>

#include "w4a16_lora.hpp"

namespace w4a16 {

namespace {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// waves of a workgroup, and 32-k chunks a wave loads before it multiplies
// (about 100 registers of loads in flight)
constexpr int shrink_waves(int tt, int rc) { return tt + rc > 4 ? 8 : 16; }
constexpr int shrink_depth(int tt, int rc) { return tt + rc > 8 ? 1 : (tt + rc > 4 ? 2 : 4); }

// A workgroup owns a tile of 16 TT tokens, 16 RC ranks and one K range, and of
// the adapters that the tile's tokens name, in the order of their first token,
// every `turns`-th: an adapter's rows are read once per tile, several adapters
// of a tile side by side.  Each XCD takes a run of work units, tile by tile of
// one K range, so that the tiles find the range of an adapter's rows in their
// L2; turns come last, since with one adapter only the first has work.
// The waves take the range's chunks in turn.  The tokens are the MFMA's A
// rows, the adapter's ranks its B columns, both loaded straight from their
// rows (16 bytes a lane); the waves are added through LDS in wave order, and
// the rows of the adapter's own tokens stored: u[split][M][R].  Tokens without
// an adapter get zeros.
//
// Bound by x, which is read once, and by a start of 4-8 us (the ids, then the
// rows that they name, then the waves' sums): one token of 4096 values 4.9 us,
// sixteen of sixteen adapters 6.1, 67 of 16 adapters (2560 values) 8; 1920 x
// 28672 with 64 ranks 45 us, 135 MB from memory (8 us and 3.7 TB/s; deeper
// loads, more waves or ranges change nothing), 1920 x 14336 26 us.
template <int DT, int TT, int RC>
__global__ __launch_bounds__(64 * shrink_waves(TT, RC)) void shrink_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ down, const int32_t* __restrict__ ids,
    float* __restrict__ u, uint16_t* __restrict__ op, const float* __restrict__ alpha, int M, int K, int S, int R, int chunks_per_split, int turns) {
  constexpr int WAVES = shrink_waves(TT, RC), DEPTH = shrink_depth(TT, RC), BM = 16 * TT, BR = 16 * RC;
  __shared__ __attribute__((aligned(16))) float red[WAVES * 256 * RC];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, row4 = lane >> 4;
  // unit = ((turn * rank groups + rank group) * splits + split) * tiles + tile
  const int tiles = (M + BM - 1) / BM, rgroups = (R + BR - 1) / BR;
  const int per_turn = gridDim.x / turns;  // units of a turn: rank groups x splits x tiles
  const int turn = blockIdx.x / per_turn;
  int unit = xcd_unit(blockIdx.x - turn * per_turn, per_turn);
  const int tile = unit % tiles;
  unit /= tiles;
  const int splits = per_turn / (tiles * rgroups), split = unit % splits;
  const int m0 = tile * BM, r0 = unit / splits * BR;
  float* const out = u + (size_t)split * M * R;

  const bool token = lane < BM && m0 + lane < M;
  const int mine = token ? ids[m0 + lane] : -1;
  const bool named = mine >= 0 && mine < S;
  if (turn == 0) {
    uint64_t none = __ballot(token && !named);
    for (; none; none &= none - 1) {
      const int m = m0 + __builtin_ctzll(none);
      for (int r = r0 + tid; r < min(R, r0 + BR); r += blockDim.x) out[(size_t)m * R + r] = 0.f;
    }
  }
  const uint16_t* xrow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xrow[t] = x + (size_t)min(m0 + 16 * t + col, M - 1) * K;
  const int c_begin = split * chunks_per_split;
  const int c_end = min((K + 31) >> 5, c_begin + chunks_per_split);

  uint64_t todo = __ballot(named);
  for (int n = 0; todo; ++n) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
    const uint64_t own = __ballot(named && mine == a);
    todo &= ~own;
    if (n % turns != turn) continue;
    const uint16_t* arow[RC];
    f32x4 acc[TT][RC];
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) {
      arow[rc] = down + ((size_t)a * R + min(r0 + 16 * rc + col, R - 1)) * K;
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t][rc] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int c0 = c_begin + wave * DEPTH; c0 < c_end; c0 += WAVES * DEPTH) {
      u32x4 xv[DEPTH][TT], av[DEPTH][RC];
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) {
        // K is a multiple of 8: past it (a last chunk's upper lanes, a depth
        // past the range) both operands are zero
        const int k = 32 * (c0 + i) + 8 * row4;
        const bool in = k < K;
        const int kc = in ? k : K - 8;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          xv[i][t] = *reinterpret_cast<const u32x4*>(xrow[t] + kc);
          if (!in) xv[i][t] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int rc = 0; rc < RC; ++rc) {
          av[i][rc] = *reinterpret_cast<const u32x4*>(arow[rc] + kc);
          if (!in) av[i][rc] = u32x4{0u, 0u, 0u, 0u};
        }
      }
#pragma unroll
      for (int i = 0; i < DEPTH; ++i)
        if (c0 + i < c_end) {
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int rc = 0; rc < RC; ++rc) acc[t][rc] = mfma16x16x32<DT>(xv[i][t], av[i][rc], acc[t][rc]);
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t || n) __syncthreads();  // the previous block's sums are read
#pragma unroll
      for (int rc = 0; rc < RC; ++rc)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[wave * (16 * BR) + (4 * row4 + e) * BR + 16 * rc + col] = acc[t][rc][e];
      __syncthreads();
      for (int i = tid; i < 16 * BR; i += blockDim.x) {
        const int m = 16 * t + i / BR, r = r0 + i % BR;
        if (r < R && (own >> m) & 1) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < WAVES; ++w) v += red[w * (16 * BR) + i];
          out[(size_t)(m0 + m) * R + r] = v;
          if constexpr (DT == DT_BF16) {
            if (op) {  // (one K range)
              uint16_t* const d = op + (size_t)(m0 + m) * 2 * R + r;
              split_hi_lo<DT>(alpha ? v * alpha[a] : v, d[0], d[R]);
            }
          }
        }
      }
    }
  }
}

// u = the K ranges' sums in range order, and alpha * u as operands (each where
// wanted); n = M R.  Four ranks a lane, a token 2^lanes_log2 lanes, which find
// its largest value together.  (A launch of its own: 2.3-4 us for 67 tokens of 32
// ranks, 5.2 for 1920 of 64.)
template <int DT>
__global__ __launch_bounds__(256) void shrink_reduce_kernel(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                            const float* __restrict__ alpha, float* u, uint16_t* __restrict__ op,
                                                            int32_t* __restrict__ shift, int64_t n, int lanes_log2, int splits,
                                                            int S, int R) {
  const int64_t lane = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, m = lane >> lanes_log2;
  const int r = 4 * (int)(lane & ((1 << lanes_log2) - 1));
  const int64_t i = m * R + r;
  if (m * R >= n) return;  // (a token's lanes together)
  const bool in = r < R;
  // (alpha's two loads on their way beside the sums')
  const int a = op ? ids[m] : -1;
  const float k = alpha && a >= 0 && a < S ? alpha[a] : 1.f;
  const float* const src = part + (in ? i : m * R);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 4) {  // four at a time, so that their loads overlap
    f32x4 p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = *reinterpret_cast<const f32x4*>(src + min(s0 + k, splits - 1) * n);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 + k < splits) v += p[k];
  }
  if (u && in) *reinterpret_cast<f32x4*>(u + i) = v;
  if (!op) return;
  if (!in) v = f32x4{0.f, 0.f, 0.f, 0.f};
  v *= k;
  if constexpr (DT == DT_F16) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, magnitude_bits(v[e]));
    for (int b = 0; b < lanes_log2; ++b) top = max(top, (uint32_t)__shfl_xor((int)top, 1 << b));
    const int sh = op_shift(top);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e], sh);
    if (r == 0) shift[m] = sh;
  }
  if (!in) return;
  u16x4 h, l;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint16_t hi, lo;
    split_hi_lo<DT>(v[e], hi, lo);
    h[e] = hi, l[e] = lo;
  }
  uint16_t* const d = op + (size_t)m * 2 * R + r;
  *reinterpret_cast<u16x4*>(d) = h;
  *reinterpret_cast<u16x4*>(d + R) = l;
}

template <int DT, int TT, int RC>
hipError_t launch_t(const ShrinkArgs& a, const ShrinkPlan& p, float* out, hipStream_t s) {
  const int64_t tiles = (a.M + 16 * TT - 1) / (16 * TT);
  const int turns = std::min(a.S, TT == 1 ? 16 : 8);  // (adapters of a tile: at most its tokens)
  const int64_t units = tiles * p.splits * ((a.R + 16 * RC - 1) / (16 * RC)) * turns;
  if (units > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)units);
  hipLaunchKernelGGL((shrink_kernel<DT, TT, RC>), grid, dim3(64 * shrink_waves(TT, RC)), 0, s,
                     static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.down), a.ids, out,
                     p.splits == 1 && DT == DT_BF16 ? a.op : nullptr, a.alpha, (int)a.M, (int)a.K, a.S, a.R, p.chunks_per_split, turns);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const ShrinkArgs& a, const ShrinkPlan& p, float* out, hipStream_t s) {
  switch (10 * p.tt + p.rc) {
    case 11: return launch_t<DT, 1, 1>(a, p, out, s);
    case 41: return launch_t<DT, 4, 1>(a, p, out, s);
    case 42: return launch_t<DT, 4, 2>(a, p, out, s);
    case 44: return launch_t<DT, 4, 4>(a, p, out, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

ShrinkPlan plan_shrink(int64_t M, int64_t K, int R, int cu_count, bool few) {
  ShrinkPlan p;
  const int chunks = (int)((K + 31) / 32);
  // 16-token tiles up to 256 tokens: more workgroups for little x (64-token
  // tiles read an adapter's rows a fourth as often, from L2 either way)
  p.tt = M <= 256 ? 1 : 4;
  const int blocks_r = (R + 15) / 16;
  p.rc = p.tt == 1 ? 1 : (blocks_r > 2 ? 4 : blocks_r);
  const int64_t groups = (M + 16 * p.tt - 1) / (16 * p.tt) * ((blocks_r + p.rc - 1) / p.rc);
  // ranges of 1024 k (half: the shrink 5-15 % faster, the sum over ranges
  // slower by more); `few`: at most four, which a decode epilogue reads at once
  int splits = (int)std::min<int64_t>((K + 1023) / 1024, std::max<int64_t>(1, 2 * cu_count / groups));
  splits = std::min(splits, few ? 4 : kMaxShrinkSplits);
  p.chunks_per_split = (chunks + splits - 1) / splits;
  p.splits = (chunks + p.chunks_per_split - 1) / p.chunks_per_split;
  return p;
}

hipError_t launch_shrink(const ShrinkArgs& a, const ShrinkPlan& p, hipStream_t s) {
  float* const out = p.splits > 1 && a.u ? a.part : (a.u ? a.u : a.part);
  const hipError_t e = a.dtype == DT_F16 ? launch_dt<DT_F16>(a, p, out, s) : launch_dt<DT_BF16>(a, p, out, s);
  // one K range: u is there, and bf16's operands; fp16's need a token's largest
  // value, which several workgroups hold (1920 tokens, 1024 x 4096: 34 -> 37 us)
  const bool u_done = p.splits == 1, op_done = u_done && a.dtype == DT_BF16;
  if (e != hipSuccess || !((a.u && !u_done) || (a.op && !op_done))) return e;
  const int64_t n = a.M * a.R;
  int lanes_log2 = 1;
  while ((4 << lanes_log2) < a.R) ++lanes_log2;
  auto kern = a.dtype == DT_F16 ? shrink_reduce_kernel<DT_F16> : shrink_reduce_kernel<DT_BF16>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(((a.M << lanes_log2) + 255) / 256)), dim3(256), 0, s, out, a.ids, a.alpha,
                     u_done ? nullptr : a.u, a.op, a.shift, n, lanes_log2, p.splits, a.S, a.R);
  return hipGetLastError();
}

}  // namespace w4a16
