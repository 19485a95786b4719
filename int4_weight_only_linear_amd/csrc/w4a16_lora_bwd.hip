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
//   rows     dy with its rows padded to np, where N is no multiple of 64
//   tail     the weights' last rows as a whole step, where N is no multiple of 64
//   consts   the rows' constants by group, as dx_kernel takes them (DxPrep)
//   1        the words that later kernels find zero
// Bound by memory latency: 3.6 us for 128 tokens and 4096 x 4096, 6.8 us for 1920
// and 4096 x 28672.
__global__ __launch_bounds__(256) void prep_kernel(const PrepArgs a, int tiles_n, int tiles_k, int pad_blocks, int tail_blocks,
                                                   int const_blocks) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[kMaxRank * (kTile + 2)];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int job = blockIdx.x;
  if (job < a.S) {
    // batches of 8 x 256 ids, a batch's loads all issued at once (one load and
    // two barriers per 256 ids made this the launch's critical path)
    constexpr int B = 8;
    int* const counts = reinterpret_cast<int*>(lds);  // [B][4] own per wave, [4] below
    const int s = job;
    int id[B];
    auto load = [&](int m0) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int m = m0 + 256 * i + tid;
        id[i] = m < a.M ? a.ids[m] : -1;
      }
    };
    int below = 0;
    for (int m0 = 0; m0 < a.M; m0 += 256 * B) {
      load(m0);
#pragma unroll
      for (int i = 0; i < B; ++i) below += __popcll(__ballot(id[i] >= 0 && id[i] < s));
    }
    if (lane == 0) counts[4 * B + wave] = below;
    __syncthreads();
    const int before_all = counts[4 * B] + counts[4 * B + 1] + counts[4 * B + 2] + counts[4 * B + 3];
    const int first = (before_all + 31) / 32 * 32 + 32 * s;
    int at = first;
    for (int m0 = 0; m0 < a.M; m0 += 256 * B) {
      if (a.M > 256 * B) load(m0);  // (a single batch is still here)
      uint64_t mask[B];
#pragma unroll
      for (int i = 0; i < B; ++i) mask[i] = __ballot(id[i] == s);
      __syncthreads();
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < B; ++i) counts[4 * i + wave] = __popcll(mask[i]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < B; ++i) {
        int before = at;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int n = counts[4 * i + w];
          before += w < wave ? n : 0;
          at += n;
        }
        if (id[i] == s) a.order[before + __popcll(mask[i] & ((1ull << lane) - 1))] = m0 + 256 * i + tid;
      }
    }
    // nothing up to where the next adapter begins (the last: to the end; the
    // first: from the beginning, which is its own)
    const int next = s == a.S - 1 ? a.places : (before_all + (at - first) + 31) / 32 * 32 + 32 * (s + 1);
    for (int i = at + tid; i < next; i += 256) a.order[i] = -1;
    if (tid == 0) {
      a.start[s] = first;
      a.count[s] = at - first;
    }
    return;
  }
  job -= a.S;
  if (job < a.S * tiles_n) {
    // lb[s][n0 + i][r] -> lb_t[s][r][n0 + i]
    const int s = job / tiles_n, n0 = (job - s * tiles_n) * kTile, R8 = a.R >> 3;
    const uint16_t* src = a.lb + ((size_t)s * a.N + n0) * a.R;
#pragma unroll 4
    for (int i = tid; i < kTile * R8; i += 256) {
      const int n = i / R8, r = 8 * (i - n * R8);
      const u32x4 w = n0 + n < a.N ? *reinterpret_cast<const u32x4*>(src + 8 * i) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) lds[(r + e) * (kTile + 2) + n] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
    __syncthreads();
    uint16_t* dst = a.lb_t + (size_t)s * a.R * a.np + n0;
    for (int i = tid; i < a.R * (kTile / 8); i += 256) {  // (np is a multiple of the tile)
      const int r = i / (kTile / 8), n = 8 * (i % (kTile / 8));
      const uint32_t* l = reinterpret_cast<const uint32_t*>(lds + r * (kTile + 2) + n);
      *reinterpret_cast<u32x4*>(dst + (size_t)r * a.np + n) = u32x4{l[0], l[1], l[2], l[3]};
    }
    return;
  }
  job -= a.S * tiles_n;
  if (job < a.S * tiles_k) {
    // la[s][r][k0 + i] -> la_t[s][k0 + i][r]
    const int s = job / tiles_k, k0 = (job - s * tiles_k) * kTile, R8 = a.R >> 3;
    const uint16_t* src = a.la + (size_t)s * a.R * a.K + k0;
#pragma unroll 4
    for (int i = tid; i < a.R * (kTile / 8); i += 256) {
      const int r = i / (kTile / 8), k = 8 * (i % (kTile / 8));
      if (k0 + k >= a.K) continue;  // K is a multiple of 8
      const u32x4 w = *reinterpret_cast<const u32x4*>(src + (size_t)r * a.K + k);
      uint32_t* l = reinterpret_cast<uint32_t*>(lds + r * (kTile + 2) + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) l[e] = w[e];
    }
    __syncthreads();
    uint16_t* dst = a.la_t + ((size_t)s * a.K + k0) * a.R;
    for (int i = tid; i < min(kTile, a.K - k0) * R8; i += 256) {
      const int k = i / R8, r = 8 * (i - k * R8);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)lds[(r + 2 * e) * (kTile + 2) + k] | ((uint32_t)lds[(r + 2 * e + 1) * (kTile + 2) + k] << 16);
      *reinterpret_cast<u32x4*>(dst + 8 * i) = u32x4{w[0], w[1], w[2], w[3]};
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
  job -= pad_blocks;
  if (job < tail_blocks) {
    const int J = a.K >> 3, n0 = a.N / 64 * 64, runs = J >> 4, tail = J & 15;
    for (int i = job * 256 + tid; i < 64 * J; i += tail_blocks * 256) {
      const int t = i / (16 * J), off = i - t * 16 * J, first = n0 + 16 * t;
      uint32_t w = 0u;
      if (first + 16 <= a.N) {
        w = a.dx.wq[(size_t)first * J + off];
      } else {
        // row and word of the row at this place of a complete tile
        const bool run = off < 256 * runs;
        const int piece = (off & 255) >> 2, rest = off - 256 * runs;
        const int row = run ? piece & 15 : rest / max(tail, 1);
        const int word = run ? (off >> 8) * 16 + 4 * (piece >> 4) + (off & 3) : 16 * runs + rest - row * tail;
        if (first + row < a.N) w = a.dx.wq[(size_t)(first + row) * J + word];
      }
      a.dx.wq_tail[i] = w;
    }
    return;
  }
  job -= tail_blocks;
  if (job < const_blocks) {
    // 16 rows x 32 groups through LDS: scale bits and zero point of each
    uint32_t* const sz = reinterpret_cast<uint32_t*>(lds);  // [16][33]
    const int G = a.dx.G, gb = (G + 31) / 32, n0 = job / gb * 16, g0 = (job - job / gb * gb) * 32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = (tid >> 5) + 8 * j, n = min(n0 + row, a.N - 1), g = min(g0 + (tid & 31), G - 1);
      const uint32_t sc = a.dx.scales[(size_t)n * G + g];
      const uint32_t z = a.dx.zp ? (a.dx.zp[(size_t)(n >> 3) * G + g] >> (4 * (n & 7))) & 15u : 8u;
      sz[row * 33 + (tid & 31)] = n0 + row < a.N ? sc | (z << 16) : 0u;
    }
    __syncthreads();
    const int g = tid >> 3, q = tid & 7;  // group, pair of rows
    if (g0 + g >= G) return;
    const uint32_t a0 = sz[2 * q * 33 + g], a1 = sz[(2 * q + 1) * 33 + g];
    const size_t at = (size_t)(g0 + g) * a.np / 2 + n0 / 2 + q;
    if (a.dx.dtype == DT_F16) {
      constexpr uint32_t NEG = Magic<DT_F16>::neg;
      static_cast<u32x2*>(a.dx.constants)[at] = u32x2{(a0 & 0xFFFFu) | (a1 << 16), (NEG | (a0 >> 16)) | ((NEG | (a1 >> 16)) << 16)};
    } else {
      const GroupConst<DT_BF16> c0 = group_const<DT_BF16, true>((uint16_t)a0, a0 >> 16);
      const GroupConst<DT_BF16> c1 = group_const<DT_BF16, true>((uint16_t)a1, a1 >> 16);
      static_cast<f32x4*>(a.dx.constants)[at] = f32x4{c0.s_f32, c0.c_f32, c1.s_f32, c1.c_f32};
    }
    return;
  }
  for (int i = tid; i < a.zero_words; i += 256) a.zero[i] = 0u;
}

// Workgroups below row_blocks sum g's K ranges token by token (eight ranks a
// lane, a token 2^lanes_log2 lanes, which find its largest value together); the
// others take 64 places of one problem each and transpose its rows through LDS
// into operands.
// Bound by the sum over g's K ranges, read twice: 3.1 us for 128 tokens of 16
// ranks, 12 us for 1920 of 64 (16 ranges).
// (the sum over K ranges, four at a time so that their loads overlap)
__device__ __forceinline__ f32x4 sum_ranges(const float* src, int64_t plane, int splits) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 4) {
    f32x4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const f32x4*>(src + min(s0 + i, splits - 1) * plane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s0 + i < splits) v += p[i];
  }
  return v;
}

template <int DT>
__global__ __launch_bounds__(256) void operand_kernel(const OperandArgs a, int row_blocks, int place_blocks, int lanes_log2) {
  __shared__ float lds[kMaxRank * (kTile + 1)];
  const int tid = threadIdx.x;
  const int64_t n = (int64_t)a.M * a.R;
  if ((int)blockIdx.x < row_blocks) {
    // eight ranks of a token (none is read of a token without an adapter)
    const int64_t at = (int64_t)blockIdx.x * 256 + tid, m = at >> lanes_log2;
    const int r = 8 * (int)(at & ((1 << lanes_log2) - 1));
    if (m >= a.M) return;  // (a token's lanes together)
    const int s = a.ids[m];
    if (s < 0 || s >= a.S) return;
    const float alpha = a.alpha ? a.alpha[s] : 1.f;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < a.R) {
      const float* src = a.part + m * a.R + r;
      const f32x4 g[2] = {sum_ranges(src, n, a.splits), sum_ranges(src + 4, n, a.splits)};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = g[e >> 2][e & 3] * alpha;
    }
    if constexpr (DT == DT_F16) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(v[e]));
      for (int b = 0; b < lanes_log2; ++b) top = max(top, (uint32_t)__shfl_xor((int)top, 1 << b));
      const int sh = op_shift(top);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], sh);
      if (r == 0) a.g_shift[m] = sh;
    }
    if (r >= a.R) return;
    u32x4 hi, lo;
    split_hi_lo<DT>(v, hi, lo);
    uint16_t* const d = a.g + 2 * m * a.R + r;
    *reinterpret_cast<u32x4*>(d) = hi;
    *reinterpret_cast<u32x4*>(d + a.R) = lo;
    return;
  }
  const int job = blockIdx.x - row_blocks;
  const bool second = job >= place_blocks;
  const int p0 = (job - (second ? place_blocks : 0)) * kTile;
  for (int i = tid; i < kTile * (a.R / 4); i += 256) {
    const int pl = i / (a.R / 4), r = 4 * (i - pl * (a.R / 4));
    const int m = p0 + pl < a.places ? a.order[p0 + pl] : -1;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (m >= 0) {
      const float alpha = a.alpha ? a.alpha[a.ids[m]] : 1.f;
      v = second ? *reinterpret_cast<const f32x4*>(a.u + (size_t)m * a.R + r)
                 : sum_ranges(a.part + (size_t)m * a.R + r, n, a.splits);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= alpha;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) lds[(r + e) * (kTile + 1) + pl] = v[e];
  }
  __syncthreads();
  uint16_t* const out = second ? a.op[1] : a.op[0];
  const int ranks = DT == DT_F16 ? (a.R + 63) / 64 * 64 : a.R;  // (shifts of ranks past R: zero)
  for (int i = tid; i < ranks * (kTile / 8); i += 256) {
    const int r = i / (kTile / 8), pl = 8 * (i - r * (kTile / 8));
    if (p0 + pl >= a.places) continue;  // places is a multiple of 32
    int8_t* const shift = (second ? a.op_shift[1] : a.op_shift[0]) + (size_t)((p0 + pl) / 32) * ((a.R + 63) / 64 * 64) + shift_at(r);
    if (DT == DT_F16 && r >= a.R) {
      *shift = 0;
      continue;
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = lds[r * (kTile + 1) + pl + e];
    if constexpr (DT == DT_F16) {
      // 32 places are four lanes, which take this turn together
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(v[e]));
      top = max(top, (uint32_t)__shfl_xor((int)top, 1));
      top = max(top, (uint32_t)__shfl_xor((int)top, 2));
      const int sh = op_shift(top);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], sh);
      if ((i & 3) == 0) *shift = (int8_t)(sh / 16);
    }
    u32x4 hi, lo;
    split_hi_lo<DT>(v, hi, lo);
    uint16_t* const d = out + (size_t)r * a.places + p0 + pl;
    *reinterpret_cast<u32x4*>(d) = hi;
    *reinterpret_cast<u32x4*>(d + (size_t)a.R * a.places) = lo;
  }
}

// columns per lane: with 64 ranks, four (eight would spill the accumulators);
// then two waves side by side share a step's operands, which they find in L1
constexpr int outer_cpl(int rc) { return rc == 4 ? 4 : 8; }
constexpr int outer_cw(int rc) { return rc == 4 ? 2 : 1; }
constexpr int outer_cols(int rc) { return 16 * outer_cpl(rc) * outer_cw(rc); }

// A workgroup owns 128 columns of one problem, 16 RC ranks, one adapter and a
// range of its tokens; its eight waves, CW beside each other, take steps of 32
// places in turn.  The
// tokens are the MFMA's reduction (16x16x32): a lane loads CPL columns of 8
// tokens (a step later in flight) and pairs the tokens' halves with v_perm
// into the A operands of its columns; the B operands, value and
// remainder of w, come ready by rank and place.  Nothing is rounded but the
// result.  The waves are added through LDS buffers in two passes, always in
// the same order; where an adapter has more tokens than one workgroup
// takes, the ranges' fp32 sums go through the workspace and the last to arrive
// adds them in range order.
//
// Bound by the rows of x and dy, and by the operands that every 128 columns
// read again: 1920 tokens of one adapter, 64 ranks, 4096 and 28672 columns: 44 us
// for 126 MB (66 with one wave for 64 columns and tokens read one step ahead);
// 1921 tokens of three, 16 ranks, 4096 and 6144 columns: 10.9 us; 128 tokens 4.9.
template <int DT, int RC>
__global__ __launch_bounds__(512) void outer_kernel(const OuterArgs a, const OuterPlan pl) {
  constexpr int CPL = outer_cpl(RC), CW = outer_cw(RC), BC = outer_cols(RC), BR = 16 * RC, LD = BC + 4;
  constexpr int TW = 8 / CW, STRIDE = 32 * TW, BUFS = TW / 2;
  typedef uint32_t cols_t __attribute__((ext_vector_type(CPL / 2)));
  __shared__ __attribute__((aligned(16))) float sum[BUFS * BR * LD];
  __shared__ uint32_t last_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave8 = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wave8 / CW, cw = wave8 % CW;  // turn among the steps, place among the columns
  const int col = lane & 15, q = lane >> 4;
  const bool second = (int)blockIdx.x >= pl.tiles[0];
  const OuterProblem& p = second ? a.p[1] : a.p[0];
  const int tile = blockIdx.x - (second ? pl.tiles[0] : 0);
  const int s = blockIdx.y;
  const int split = blockIdx.z / pl.rgroups, rg = blockIdx.z - split * pl.rgroups;
  const int start = a.start[s], count = a.count[s];
  const int ranges = max(1, (count + pl.tokens - 1) / pl.tokens);
  if (split >= ranges) return;
  const int t_begin = start + split * pl.tokens, t_end = start + min(count, (split + 1) * pl.tokens);
  const int c0 = tile * BC, r0 = rg * BR;

  f32x4 acc[CPL][RC];
#pragma unroll
  for (int t = 0; t < CPL; ++t)
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) acc[t][rc] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint16_t* vcol = p.v + min(c0 + 16 * CPL * cw + CPL * col, p.ld - CPL);
  const size_t lo_at = (size_t)a.R * a.places;
  // fp16: the sums of a lane's ranks (a byte each) at the shifts of the last
  // step's operands
  constexpr bool SHIFTED = DT == DT_F16;
  const int8_t* const shifts = p.shift + r0 / 64 * 64;
  const uint32_t shift_step = (uint32_t)((a.R + 63) / 64 * 64);  // bytes of 32 places (all of them below 4 GiB)
  uint32_t shift = 0;
  auto rescale = [&](uint32_t to) {
    if (__builtin_expect(__ballot(to != shift) == 0, 1)) return;
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) {
      // (r0 is a multiple of 16 RC, so a group of ranks lies inside 64)
      const int by = 16 * ((int8_t)(to >> (8 * rc)) - (int8_t)(shift >> (8 * rc)));
#pragma unroll
      for (int t = 0; t < CPL; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][rc][e] = __builtin_ldexpf(acc[t][rc][e], by);
        __builtin_amdgcn_sched_barrier(0);  // (few registers beside the accumulators)
      }
    }
    shift = to;
  };

  // The tokens of a step's places are read two steps ahead and its rows one:
  // the rows' addresses never wait.  (Places past the tokens hold -1.)
  struct Step {
    cols_t v[8];
    u32x4 hi[RC], lo[RC];
    uint32_t shift;
  };
  const int t_last = start + (count + 31) / 32 * 32 - 32;  // the adapter's last step
  auto load_tokens = [&](int t0, int (&m)[8]) {
    const int at = min(t0, t_last) + 8 * q;
    const int4 m0 = *reinterpret_cast<const int4*>(a.order + at), m1 = *reinterpret_cast<const int4*>(a.order + at + 4);
    m[0] = m0.x, m[1] = m0.y, m[2] = m0.z, m[3] = m0.w, m[4] = m1.x, m[5] = m1.y, m[6] = m1.z, m[7] = m1.w;
  };
  auto load = [&](int t0, const int (&m)[8], Step& st) {
    const int at = min(t0, t_last) + 8 * q;
#pragma unroll
    for (int e = 0; e < 8; ++e) st.v[e] = *reinterpret_cast<const cols_t*>(vcol + (size_t)max(m[e], 0) * p.ld);
    int c = col;
    asm("" : "+v"(c));  // the ranks' rows are formed here (kept over the loop they would spill)
#pragma unroll
    for (int rc = 0; rc < RC; ++rc) {
      const uint16_t* row = p.op + (size_t)min(r0 + 16 * rc + c, a.R - 1) * a.places + at;
      st.hi[rc] = *reinterpret_cast<const u32x4*>(row);
      st.lo[rc] = *reinterpret_cast<const u32x4*>(row + lo_at);
    }
    if constexpr (SHIFTED)
      st.shift = *reinterpret_cast<const uint32_t*>(shifts + ((uint32_t)(min(t0, t_last) / 32) * shift_step + 4u * (uint32_t)col));
  };
  auto multiply = [&](Step& st, int t0) {
    if (t0 + 32 > t_end) {  // wave-uniform: only an adapter's last step holds empty places
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t0 + 8 * q + e >= t_end) st.v[e] = cols_t{};
    }
    if constexpr (SHIFTED) rescale(st.shift);
#pragma unroll
    for (int t = 0; t < CPL; ++t) {
      const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
      const u32x4 f = {__builtin_amdgcn_perm(st.v[1][t >> 1], st.v[0][t >> 1], sel),
                       __builtin_amdgcn_perm(st.v[3][t >> 1], st.v[2][t >> 1], sel),
                       __builtin_amdgcn_perm(st.v[5][t >> 1], st.v[4][t >> 1], sel),
                       __builtin_amdgcn_perm(st.v[7][t >> 1], st.v[6][t >> 1], sel)};
#pragma unroll
      for (int rc = 0; rc < RC; ++rc) {
        acc[t][rc] = mfma16x16x32<DT>(f, st.hi[rc], acc[t][rc]);
        acc[t][rc] = mfma16x16x32<DT>(f, st.lo[rc], acc[t][rc]);
      }
    }
  };
  int t0 = t_begin + 32 * wave;
  if (t0 < t_end) {
    Step x, y;
    int mx[8], my[8];
    load_tokens(t0, mx);
    load_tokens(t0 + STRIDE, my);
    load(t0, mx, x);
    for (;;) {
      load(t0 + STRIDE, my, y);
      load_tokens(t0 + 2 * STRIDE, mx);
      multiply(x, t0);
      t0 += STRIDE;
      if (t0 >= t_end) break;
      load(t0 + STRIDE, mx, x);
      load_tokens(t0 + 2 * STRIDE, my);
      multiply(y, t0);
      t0 += STRIDE;
      if (t0 >= t_end) break;
    }
  }
  if constexpr (SHIFTED) rescale(0u);
  // acc[t][rc][e]: column CPL (4 q + e) + t, rank 16 rc + col
  auto put = [&](bool add) {
    float* const buf = sum + (wave % BUFS) * (BR * LD) + 16 * CPL * cw;
#pragma unroll
    for (int rc = 0; rc < RC; ++rc)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int half = 0; half < CPL / 4; ++half) {
          f32x4* d = reinterpret_cast<f32x4*>(buf + (16 * rc + col) * LD + CPL * (4 * q + e) + 4 * half);
          f32x4 v = {acc[4 * half][rc][e], acc[4 * half + 1][rc][e], acc[4 * half + 2][rc][e], acc[4 * half + 3][rc][e]};
          if (add) v = *d + v;
          *d = v;
        }
  };
  if (wave < BUFS) put(false);
  __syncthreads();
  if (wave >= BUFS) put(true);
  __syncthreads();
  auto total = [&](int r, int c) {
    const float* d = sum + r * LD + c;
    if constexpr (BUFS == 2) return d[0] + d[BR * LD];
    return (d[0] + d[BR * LD]) + (d[(BUFS - 2) * BR * LD] + d[(BUFS - 1) * BR * LD]);
  };
  if (ranges > 1) {
    // slots of an adapter with several ranges: from 2 floor(start / tokens),
    // which no other such adapter reaches (ceil(c / t) <= 2 floor(c / t) where
    // c > t, and starts are at least their adapters' tokens apart)
    const size_t tiles = (size_t)(pl.tiles[0] + pl.tiles[1]) * pl.rgroups;
    const size_t place = (size_t)blockIdx.x * pl.rgroups + rg;
    const size_t slot = 2 * (size_t)(start / pl.tokens);
    float* const mine = a.partial + ((slot + split) * tiles + place) * (BR * BC);
    for (int i = tid; i < BR * BC; i += 512) store_coherent(mine + i, total(i / BC, i % BC));
    wait_vm_all();  // every store of this thread has completed before the arrival
    __syncthreads();
    uint32_t* const counter = a.counters + (size_t)s * tiles + place;
    if (tid == 0) last_flag = arrive(counter) == (uint32_t)(ranges - 1);
    __syncthreads();
    if (!last_flag) return;
    for (int i = tid; i < BR * BC; i += 512) {
      float v = 0.f;
      for (int sp = 0; sp < ranges; ++sp) v += load_coherent(a.partial + ((slot + sp) * tiles + place) * (BR * BC) + i);
      float* d = sum + (i / BC) * LD + i % BC;
      d[0] = v;
#pragma unroll
      for (int k = 1; k < BUFS; ++k) d[k * BR * LD] = 0.f;
    }
    __syncthreads();
  }
  if (p.by_rank) {
    for (int i = tid; i < BR * (BC / 8); i += 512) {
      const int r = i / (BC / 8), c = 8 * (i % (BC / 8));
      if (r0 + r >= a.R || c0 + c >= p.C) continue;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32x2_to_act_pair<DT>(total(r, c + 2 * e), total(r, c + 2 * e + 1));
      // C is K here, a multiple of 32
      *reinterpret_cast<u32x4*>(p.out + ((size_t)s * a.R + r0 + r) * p.C + c0 + c) = u32x4{w[0], w[1], w[2], w[3]};
    }
  } else {
    for (int i = tid; i < BC * (BR / 8); i += 512) {
      const int r = 8 * (i / BC), c = i % BC;
      if (r0 + r >= a.R || c0 + c >= p.C) continue;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32x2_to_act_pair<DT>(total(r + 2 * e, c), total(r + 2 * e + 1, c));
      *reinterpret_cast<u32x4*>(p.out + ((size_t)s * p.C + c0 + c) * a.R + r0 + r) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

}  // namespace

hipError_t launch_prep(const PrepArgs& a, hipStream_t s) {
  const int tiles_n = (a.np + kTile - 1) / kTile, tiles_k = (a.K + kTile - 1) / kTile;
  const int pad_blocks = a.dy_pad ? (int)std::min<int64_t>(2048, ((int64_t)a.M * a.np + 255) / 256) : 0;
  const int tail_blocks = a.dx.wq_tail ? (8 * a.K + 1023) / 1024 : 0;  // four words a thread
  const int const_blocks = a.dx.constants ? a.np / 16 * ((a.dx.G + 31) / 32) : 0;
  const int64_t jobs = (int64_t)a.S * (1 + tiles_n + tiles_k) + pad_blocks + tail_blocks + const_blocks + 1;
  if (jobs > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(prep_kernel, dim3((unsigned)jobs), dim3(256), 0, s, a, tiles_n, tiles_k, pad_blocks, tail_blocks, const_blocks);
  return hipGetLastError();
}

hipError_t launch_operands(const OperandArgs& a, hipStream_t s) {
  int lanes_log2 = 0;
  while ((8 << lanes_log2) < a.R) ++lanes_log2;
  const int row_blocks = (int)((((int64_t)a.M << lanes_log2) + 255) / 256), place_blocks = (a.places + kTile - 1) / kTile;
  auto kern = a.dtype == DT_F16 ? operand_kernel<DT_F16> : operand_kernel<DT_BF16>;
  hipLaunchKernelGGL(kern, dim3(row_blocks + 2 * place_blocks), dim3(256), 0, s, a, row_blocks, place_blocks, lanes_log2);
  return hipGetLastError();
}

OuterPlan plan_outer(int64_t M, int64_t C0, int64_t C1, int S, int R, int cu_count) {
  OuterPlan p;
  const int blocks = (R + 15) / 16;
  p.rc = blocks > 2 ? 4 : blocks;
  p.rgroups = (blocks + p.rc - 1) / p.rc;
  const int cols = outer_cols(p.rc);
  p.tiles[0] = (int)((C0 + cols - 1) / cols);
  p.tiles[1] = (int)((C1 + cols - 1) / cols);
  // about one workgroup per CU when one adapter has all tokens (a range costs
  // its sums' round trip through memory)
  const int64_t want = std::max<int64_t>(1, cu_count / ((int64_t)(p.tiles[0] + p.tiles[1]) * p.rgroups));
  p.tokens = (int)std::max<int64_t>(256, (M / want + 255) / 256 * 256);
  p.splits = (int)((M + p.tokens - 1) / p.tokens);
  return p;
}
size_t outer_partial_bytes(const OuterPlan& p, int64_t places) {
  if (p.splits <= 1) return 0;
  // starts lie below order_places(M, S): 32 per adapter past the tokens, and an
  // adapter of several ranges has more than `tokens` >= 256 of them
  return (size_t)(2 * (places / p.tokens) + 2 + p.splits) * (size_t)(p.tiles[0] + p.tiles[1]) * p.rgroups * (16 * p.rc * outer_cols(p.rc)) * sizeof(float);
}
size_t outer_counter_bytes(const OuterPlan& p, int S) {
  return (size_t)S * (size_t)(p.tiles[0] + p.tiles[1]) * p.rgroups * sizeof(uint32_t);
}

hipError_t launch_outer(const OuterArgs& a, const OuterPlan& p, hipStream_t s) {
  if (a.S > 65535 || (int64_t)p.splits * p.rgroups > 65535) return hipErrorInvalidValue;
  const dim3 grid(p.tiles[0] + p.tiles[1], a.S, p.splits * p.rgroups);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(512), 0, s, a, p);
    return hipGetLastError();
  };
  if (a.dtype == DT_F16)
    return p.rc == 1 ? go(outer_kernel<DT_F16, 1>) : p.rc == 2 ? go(outer_kernel<DT_F16, 2>) : go(outer_kernel<DT_F16, 4>);
  return p.rc == 1 ? go(outer_kernel<DT_BF16, 1>) : p.rc == 2 ? go(outer_kernel<DT_BF16, 2>) : go(outer_kernel<DT_BF16, 4>);
}

}  // namespace w4a16
