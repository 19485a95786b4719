// Gradients of the low-rank adapters: the tokens in the order of their
// adapters, the factors transposed, and the two sums over tokens
//   dA_s[r, k] = sum_m g[m, r] x[m, k],  dB_s[n, r] = alpha_s sum_m dy[m, n] u[m, r]
// (g = alpha_s dy . B_s comes from shrink_kernel over the transposed B, the
// input gradient from w4a16_dx.hip).
#include <algorithm>

#include "w4a16_lora.hpp"
#include "w4a16_lora_bwd.hpp"

namespace w4a16 {

namespace {

constexpr int kTile = 64;  // rows / columns of a transposed tile (the rank side holds up to 128)

// One launch: the workgroups take one job each, by index --
//   S        the tokens of one adapter, in order: each scans all ids, counting
//            those of smaller adapters (its segment's start) and ranking its own
//   S tiles  lb[s][n..][:] and la[s][:][k..] transposed through LDS
//   rows     dy with its rows padded to np, where N is no multiple of 8
//   1        the words that later kernels find zero
__global__ __launch_bounds__(256) void prep_kernel(const PrepArgs a, int tiles_n, int tiles_k, int pad_blocks) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[kMaxRank * (kTile + 2)];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int job = blockIdx.x;
  if (job < a.S) {
    int* const counts = reinterpret_cast<int*>(lds);  // [4] below, [4] own, per wave
    const int s = job;
    int below = 0;
    for (int m0 = 0; m0 < a.M; m0 += 256) {
      const int m = m0 + tid, id = m < a.M ? a.ids[m] : -1;
      below += __popcll(__ballot(id >= 0 && id < s));
    }
    if (lane == 0) counts[wave] = below;
    __syncthreads();
    int at = counts[0] + counts[1] + counts[2] + counts[3];
    if (tid == 0) a.seg[s] = at;
    for (int m0 = 0; m0 < a.M; m0 += 256) {
      const int m = m0 + tid;
      const bool own = m < a.M && a.ids[m] == s;
      const uint64_t mask = __ballot(own);
      __syncthreads();
      if (lane == 0) counts[4 + wave] = __popcll(mask);
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < 4; ++w) {
        before += w < wave ? counts[4 + w] : 0;
        all += counts[4 + w];
      }
      if (own) a.perm[at + before + __popcll(mask & ((1ull << lane) - 1))] = m;
      at += all;
    }
    if (s == a.S - 1 && tid == 0) a.seg[a.S] = at;
    return;
  }
  job -= a.S;
  if (job < a.S * tiles_n) {
    // lb[s][n0 + i][r] -> lb_t[s][r][n0 + i]
    const int s = job / tiles_n, n0 = (job - s * tiles_n) * kTile;
    const int rows = min(kTile, a.N - n0);
    const uint16_t* src = a.lb + ((size_t)s * a.N + n0) * a.R;
    for (int i = tid; i < kTile * a.R; i += 256) {
      const int n = i / a.R, r = i - n * a.R;
      lds[r * (kTile + 2) + n] = n < rows ? src[i] : 0;
    }
    __syncthreads();
    uint16_t* dst = a.lb_t + (size_t)s * a.R * a.np + n0;
    for (int i = tid; i < a.R * kTile; i += 256) {
      const int r = i / kTile, n = i - r * kTile;
      if (n0 + n < a.np) dst[(size_t)r * a.np + n] = lds[r * (kTile + 2) + n];
    }
    return;
  }
  job -= a.S * tiles_n;
  if (job < a.S * tiles_k) {
    // la[s][r][k0 + i] -> la_t[s][k0 + i][r]
    const int s = job / tiles_k, k0 = (job - s * tiles_k) * kTile;
    const int cols = min(kTile, a.K - k0);
    const uint16_t* src = a.la + (size_t)s * a.R * a.K + k0;
    for (int i = tid; i < a.R * kTile; i += 256) {
      const int r = i / kTile, k = i - r * kTile;
      if (k < cols) lds[r * (kTile + 2) + k] = src[(size_t)r * a.K + k];
    }
    __syncthreads();
    uint16_t* dst = a.la_t + ((size_t)s * a.K + k0) * a.R;
    for (int i = tid; i < cols * a.R; i += 256) {
      const int k = i / a.R, r = i - k * a.R;
      dst[i] = lds[r * (kTile + 2) + k];
    }
    return;
  }
  job -= a.S * tiles_k;
  if (job < pad_blocks) {
    const int64_t total = (int64_t)a.M * a.np;
    for (int64_t i = (int64_t)job * 256 + tid; i < total; i += (int64_t)pad_blocks * 256) {
      const int64_t m = i / a.np;
      const int n = (int)(i - m * a.np);
      a.dy_pad[i] = n < a.N ? a.dy[m * a.N + n] : (uint16_t)0;
    }
    return;
  }
  for (int i = tid; i < a.zero_words; i += 256) a.zero[i] = 0u;
}

// A workgroup owns 128 columns of one problem, 16 RC ranks, one adapter and a
// range of its tokens; its four waves take steps of 32 tokens in turn.  The
// tokens are the MFMA's reduction (16x16x32): a lane loads 8 columns of 8
// tokens (16 bytes each) and pairs the tokens' halves with v_perm into the A
// operands of its 8 columns; the B operand is its rank's 8 tokens of w as
// value + remainder (split_hi_lo), so nothing is rounded but the result.
// The waves are added through LDS in wave order; where an adapter has more
// tokens than one workgroup takes, the ranges' fp32 sums go through the
// workspace and the last to arrive adds them in range order.
template <int DT, int RC>
__global__ __launch_bounds__(256) void outer_kernel(const OuterArgs a, const OuterPlan pl) {
  constexpr int BR = 16 * RC, LD = 128 + 4;
  __shared__ __attribute__((aligned(16))) float sum[BR * LD];
  __shared__ uint32_t last_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, q = lane >> 4;
  const bool second = (int)blockIdx.x >= pl.tiles[0];
  const OuterProblem& p = second ? a.p[1] : a.p[0];
  const int tile = blockIdx.x - (second ? pl.tiles[0] : 0);
  const int s = blockIdx.y;
  const int split = blockIdx.z / pl.rgroups, rg = blockIdx.z - split * pl.rgroups;
  const int start = a.seg[s], count = a.seg[s + 1] - start;
  const int ranges = max(1, (count + pl.tokens - 1) / pl.tokens);
  if (split >= ranges) return;
  const int t_begin = start + split * pl.tokens, t_end = start + min(count, (split + 1) * pl.tokens);
  const int c0 = tile * 128, r0 = rg * BR;
  const float alpha = a.alpha ? a.alpha[s] : 1.f;

  f32x4 acc[8][RC];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) acc[t][rc] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint16_t* vcol = p.v + min(c0 + 8 * col, p.ld - 8);
  for (int t0 = t_begin + 32 * wave; t0 < t_end; t0 += 128) {
    u32x4 v[8];
    float w[RC][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = t0 + 8 * q + e;
      const bool in = i < t_end;
      const int m = a.perm[in ? i : t_end - 1];
      v[e] = *reinterpret_cast<const u32x4*>(vcol + (size_t)m * p.ld);
      if (!in) v[e] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int rc = 0; rc < RC; ++rc) {
        const int r = r0 + 16 * rc + col;
        w[rc][e] = in && r < a.R ? p.w[(size_t)m * a.R + r] * alpha : 0.f;
      }
    }
    u32x4 hi[RC], lo[RC];
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) split_hi_lo<DT>(w[rc], hi[rc], lo[rc]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
      const u32x4 f = {__builtin_amdgcn_perm(v[1][t >> 1], v[0][t >> 1], sel),
                       __builtin_amdgcn_perm(v[3][t >> 1], v[2][t >> 1], sel),
                       __builtin_amdgcn_perm(v[5][t >> 1], v[4][t >> 1], sel),
                       __builtin_amdgcn_perm(v[7][t >> 1], v[6][t >> 1], sel)};
#pragma unroll
      for (int rc = 0; rc < RC; ++rc) {
        acc[t][rc] = mfma16x16x32<DT>(f, hi[rc], acc[t][rc]);
        acc[t][rc] = mfma16x16x32<DT>(f, lo[rc], acc[t][rc]);
      }
    }
  }
  // acc[t][rc][e]: column 8 (4 q + e) + t, rank 16 rc + col
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int rc = 0; rc < RC; ++rc)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* d = sum + (16 * rc + col) * LD + 8 * (4 * q + e) + t;
            *d = w == 0 ? acc[t][rc][e] : *d + acc[t][rc][e];
          }
    }
    __syncthreads();
  }
  if (ranges > 1) {
    // slots of an adapter with several ranges: from 2 floor(start / tokens),
    // which no other such adapter reaches (ceil(c / t) <= 2 floor(c / t), c > t)
    const size_t tiles = (size_t)(pl.tiles[0] + pl.tiles[1]) * pl.rgroups;
    const size_t place = (size_t)blockIdx.x * pl.rgroups + rg;
    const size_t slot = 2 * (size_t)(start / pl.tokens);
    float* const mine = a.partial + ((slot + split) * tiles + place) * (BR * 128);
    for (int i = tid; i < BR * 128; i += 256) store_coherent(mine + i, sum[(i >> 7) * LD + (i & 127)]);
    wait_vm_all();  // every store of this thread has completed before the arrival
    __syncthreads();
    uint32_t* const counter = a.counters + (size_t)s * tiles + place;
    if (tid == 0) last_flag = arrive(counter) == (uint32_t)(ranges - 1);
    __syncthreads();
    if (!last_flag) return;
    for (int i = tid; i < BR * 128; i += 256) {
      float v = 0.f;
      for (int sp = 0; sp < ranges; ++sp) v += load_coherent(a.partial + ((slot + sp) * tiles + place) * (BR * 128) + i);
      sum[(i >> 7) * LD + (i & 127)] = v;
    }
    __syncthreads();
  }
  if (p.by_rank) {
    for (int i = tid; i < BR * 128; i += 256) {
      const int r = i >> 7, c = i & 127;
      if (r0 + r < a.R && c0 + c < p.C)
        p.out[((size_t)s * a.R + r0 + r) * p.C + c0 + c] = f32_to_act<DT>(sum[r * LD + c]);
    }
  } else {
    for (int i = tid; i < BR * 128; i += 256) {
      const int c = i / BR, r = i - c * BR;
      if (r0 + r < a.R && c0 + c < p.C)
        p.out[((size_t)s * p.C + c0 + c) * a.R + r0 + r] = f32_to_act<DT>(sum[r * LD + c]);
    }
  }
}

}  // namespace

hipError_t launch_prep(const PrepArgs& a, hipStream_t s) {
  const int tiles_n = (a.np + kTile - 1) / kTile, tiles_k = (a.K + kTile - 1) / kTile;
  const int pad_blocks = a.dy_pad ? (int)std::min<int64_t>(2048, ((int64_t)a.M * a.np + 255) / 256) : 0;
  const int64_t jobs = (int64_t)a.S * (1 + tiles_n + tiles_k) + pad_blocks + 1;
  if (jobs > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(prep_kernel, dim3((unsigned)jobs), dim3(256), 0, s, a, tiles_n, tiles_k, pad_blocks);
  return hipGetLastError();
}

OuterPlan plan_outer(int64_t M, int64_t C0, int64_t C1, int S, int R, int cu_count) {
  OuterPlan p;
  const int blocks = (R + 15) / 16;
  p.rc = blocks > 2 ? 4 : blocks;
  p.rgroups = (blocks + p.rc - 1) / p.rc;
  p.tiles[0] = (int)((C0 + 127) / 128);
  p.tiles[1] = (int)((C1 + 127) / 128);
  // about two workgroups per CU when one adapter has all tokens
  const int64_t want = std::max<int64_t>(1, 2 * cu_count / ((int64_t)(p.tiles[0] + p.tiles[1]) * p.rgroups));
  p.tokens = (int)std::max<int64_t>(128, (M / want + 127) / 128 * 128);
  p.splits = (int)((M + p.tokens - 1) / p.tokens);
  return p;
}
size_t outer_partial_bytes(const OuterPlan& p, int64_t M) {
  if (p.splits <= 1) return 0;
  return (size_t)(2 * (M / p.tokens) + 2 + p.splits) * (size_t)(p.tiles[0] + p.tiles[1]) * p.rgroups * (16 * p.rc * 128) * sizeof(float);
}
size_t outer_counter_bytes(const OuterPlan& p, int S) {
  return (size_t)S * (size_t)(p.tiles[0] + p.tiles[1]) * p.rgroups * sizeof(uint32_t);
}

hipError_t launch_outer(const OuterArgs& a, const OuterPlan& p, hipStream_t s) {
  if (a.S > 65535 || (int64_t)p.splits * p.rgroups > 65535) return hipErrorInvalidValue;
  const dim3 grid(p.tiles[0] + p.tiles[1], a.S, p.splits * p.rgroups);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, a, p);
    return hipGetLastError();
  };
  if (a.dtype == DT_F16)
    return p.rc == 1 ? go(outer_kernel<DT_F16, 1>) : p.rc == 2 ? go(outer_kernel<DT_F16, 2>) : go(outer_kernel<DT_F16, 4>);
  return p.rc == 1 ? go(outer_kernel<DT_BF16, 1>) : p.rc == 2 ? go(outer_kernel<DT_BF16, 2>) : go(outer_kernel<DT_BF16, 4>);
}

}  // namespace w4a16
