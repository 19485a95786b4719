// Low-rank adapters beside the shared projection (device side, gfx950 only).
//
// Token m names an adapter a = ids[m]; its output row gains
//   alpha_a * sum_r u[m, r] * up_a[n, r],   u[m, r] = sum_k x[m, k] * A_a[r, k]
// u is formed first, in fp32, by shrink_kernel (w4a16_lora.hip); the
// projection's kernels then add the sum to their fp32 accumulators before
// their one rounding.  up is the stack [S][N][R], R a multiple of 8, so 16
// bytes are eight ranks of one row.
#pragma once

#include "w4a16_device.hpp"
#include "w4a16_internal.h"

namespace w4a16 {

// the adapter of token m, or -1 (no adapter, or no such token)
__device__ __forceinline__ int lora_id(const LoraTerm& t, int M, int m) {
  const int a = m < M ? t.ids[m] : -1;
  return a >= 0 && a < t.S ? a : -1;
}

__device__ __forceinline__ float lora_alpha(const LoraTerm& t, int a) { return t.alpha ? t.alpha[a] : 1.f; }

// The decode kernels' term, in fp32 throughout.  Token m belongs to the wave
// m % waves, which adds the term of the tile's 16 rows n0.. to its own sums
// before the waves are added (add(m, row, value), lanes 0..15): no further
// barrier, and every wave's loads are under way at once.  A lane takes every
// fourth run of eight ranks of one row; the K ranges of u are read four at a
// time, so that their loads overlap.
template <int DT, typename Add>
__device__ __forceinline__ void lora_wave_add(const LoraTerm& t, int M, int N, int n0, int wave, int waves, int lane,
                                              Add&& add) {
  const int n = min(n0 + (lane & 15), N - 1);
  const size_t plane = (size_t)M * t.R;
  for (int m = wave; m < M; m += waves) {
    const int a = __builtin_amdgcn_readfirstlane(lora_id(t, M, m));
    if (a < 0) continue;
    const uint16_t* up = static_cast<const uint16_t*>(t.up) + ((size_t)a * N + n) * t.R;
    const float alpha = lora_alpha(t, a);
    float s = 0.f;
    for (int r = 8 * (lane >> 4); r < t.R; r += 32) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(up + r);
      float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int s0 = 0; s0 < t.usplits; s0 += 4) {
        f32x4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* src = t.u + (size_t)min(s0 + i, t.usplits - 1) * plane + (size_t)m * t.R + r;
          v[i][0] = *reinterpret_cast<const f32x4*>(src);
          v[i][1] = *reinterpret_cast<const f32x4*>(src + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (s0 + i < t.usplits) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] += v[i][e >> 2][e & 3];
          }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        s = __builtin_fmaf(u[e], act_to_f32<DT>((uint16_t)(w[e >> 1] >> (16 * (e & 1)))), s);
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) add(m, lane, s * alpha);
  }
}

// Eight fp32 values as two MFMA operands whose sum is the value to about 16
// (bf16) or 22 (fp16) significant bits: v rounded, and what that left.  One
// operand alone would add a rounding of u as large as the output's own.
template <int DT>
__device__ __forceinline__ void split_hi_lo(const float (&v)[8], u32x4& hi, u32x4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = f32x2_to_act_pair<DT>(v[2 * i], v[2 * i + 1]);
    l[i] = f32x2_to_act_pair<DT>(v[2 * i] - act_to_f32<DT>((uint16_t)h[i]),
                                 v[2 * i + 1] - act_to_f32<DT>((uint16_t)(h[i] >> 16)));
  }
  hi = u32x4{h[0], h[1], h[2], h[3]};
  lo = u32x4{l[0], l[1], l[2], l[3]};
}
template <int DT>
__device__ __forceinline__ void split_hi_lo(float v, uint16_t& hi, uint16_t& lo) {
  hi = (uint16_t)f32x2_to_act_pair<DT>(v, 0.f);
  lo = (uint16_t)f32x2_to_act_pair<DT>(v - act_to_f32<DT>(hi), 0.f);
}

// The GEMM tile's adapter term, as more k of its product: for every adapter
// that a token of the tile names (in the order of their first tokens),
// ceil(R / 16) k-subs whose A operand is the wave's rows of up_a and whose B
// operand is alpha * u of the adapter's own tokens, zero for the others; token
// blocks without such a token are left out.  The K ranges of a split tile take
// the adapters in turns, and the operands of the next two k-subs are loaded
// while two are multiplied: a tile of many adapters is otherwise a chain of
// memory round trips (16 adapters of rank 32 among 67 tokens, 19456 x 2560:
// 28 us of 48, now 11 of 31).  The large tiles, whose accumulators leave
// few registers and whose tokens are mostly of one request, take one k-sub at
// a time.
//   acc[rb][cb]: tokens m0 + 32 rb + (lane & 31), features nw0 + 32 cb + ...
typedef uint16_t uint16x2_t __attribute__((ext_vector_type(2)));
template <int DT, int MB, int CB>
__device__ __forceinline__ void lora_steps(const LoraTerm& t, int M, int N, int m0, int nw0, int lane, int turn, int turns,
                                           f32x16 (&acc)[MB][CB]) {
  constexpr bool DEEP = MB * CB <= 8;  // registers for operands in flight beside the accumulators
  constexpr int KS = DEEP ? 2 : 1;      // k-subs of an item
  const int j = lane & 31, h = lane >> 5;
  int id[MB];
  uint64_t todo[MB];
#pragma unroll
  for (int rb = 0; rb < MB; ++rb) {
    id[rb] = lora_id(t, M, m0 + 32 * rb + j);
    todo[rb] = __ballot(id[rb] >= 0);
  }
  const uint16_t* up = static_cast<const uint16_t*>(t.up) + 8 * h;
  uint32_t row[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) row[cb] = (uint32_t)min(nw0 + 32 * cb + j, N - 1);
  int count = 0;  // adapters of the tile seen so far

  struct Item {
    int a, r0;           // adapter (-1: no more), first rank (of both halves)
    uint64_t own[MB];    // lanes whose token is the adapter's
    u32x4 w[KS][CB];
    u32x4 u[KS][MB][2];  // alpha * u: value and remainder
  };
  // the item after `it`: the next ranks of its adapter, or the next adapter
  auto next = [&](const Item& it) {
    Item n;
    n.a = it.a;
    n.r0 = it.r0 + 16 * KS;
#pragma unroll
    for (int rb = 0; rb < MB; ++rb) n.own[rb] = it.own[rb];
    if (n.r0 >= t.R) {
      n.r0 = 0;
      do {
        n.a = -1;
#pragma unroll
        for (int rb = MB - 1; rb >= 0; --rb)
          if (todo[rb]) n.a = __builtin_amdgcn_readlane(id[rb], __builtin_ctzll(todo[rb]));
        if (n.a < 0) return n;
#pragma unroll
        for (int rb = 0; rb < MB; ++rb) {
          n.own[rb] = __ballot(id[rb] == n.a);
          todo[rb] &= ~n.own[rb];
        }
      } while (count++ % turns != turn);
    }
    // (R is a multiple of 8: a last k-sub may lie past it, wholly or its upper half)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int r = n.r0 + 16 * ks;
      const bool in = r + 8 * h < t.R;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        n.w[ks][cb] = in ? *reinterpret_cast<const u32x4*>(up + ((size_t)n.a * N + row[cb]) * t.R + r) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int rb = 0; rb < MB; ++rb)
        if (n.own[rb]) {
          const bool own = in && ((n.own[rb] >> lane) & 1);
          const uint16_t* src = t.op + (size_t)(m0 + 32 * rb + j) * 2 * t.R + r + 8 * h;
          n.u[ks][rb][0] = own ? *reinterpret_cast<const u32x4*>(src) : u32x4{0u, 0u, 0u, 0u};
          n.u[ks][rb][1] = own ? *reinterpret_cast<const u32x4*>(src + t.R) : u32x4{0u, 0u, 0u, 0u};
        }
    }
    return n;
  };
  // Other adapters' tokens of a block take part with zeros, which an infinite
  // or NaN factor would turn into NaN.  Where an item holds one, it is taken
  // out of the product and made of finite numbers that overflow for the
  // adapter's own tokens: + and - max * 2^127, in bf16 whose products pass
  // fp32's range; zeros stay zeros.  (Selecting sums by token instead keeps
  // them in vector registers: up to 1150 spilled.  The test costs 8 operations
  // a fragment, nothing where all tokens are the adapter's.)
  auto multiply = [&](const Item& it) {
    uint64_t others = 0;
#pragma unroll
    for (int rb = 0; rb < MB; ++rb)
      if (it.own[rb]) others |= __ballot(m0 + 32 * rb + j < M) & ~it.own[rb];
    bool broken = false;
    constexpr uint32_t INF = DT == DT_F16 ? 0x7C00 : 0x7F80;
    if (others) {
      uint16x2_t top = {0, 0};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t word = it.w[ks][cb][e] & 0x7FFF7FFFu;
            top = __builtin_elementwise_max(top, __builtin_bit_cast(uint16x2_t, word));
          }
      broken = __ballot(top[0] >= (uint16_t)INF || top[1] >= (uint16_t)INF) != 0;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (it.r0 + 16 * ks >= t.R) continue;
#pragma unroll
      for (int rb = 0; rb < MB; ++rb)
        if (it.own[rb]) {
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            u32x4 w = it.w[ks][cb];
            if (broken) {
              u32x4 bad;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t word = w[e];
                const uint32_t mask = ((((word & 0x7FFF7FFFu) + (0x80008000u - 0x10001u * INF)) & 0x80008000u) >> 15) * 0xFFFFu;
                w[e] = word & ~mask;
                bad[e] = mask & 0x7F7F7F7Fu;
              }
              const bool own = (it.own[rb] >> lane) & 1;
              const uint32_t big = own ? 0x7F007F00u : 0u, low = own ? 0xFF00FF00u : 0u;
              acc[rb][cb] = mfma32x32x16<DT_BF16>(bad, u32x4{big, big, big, big}, acc[rb][cb]);
              acc[rb][cb] = mfma32x32x16<DT_BF16>(bad, u32x4{low, low, low, low}, acc[rb][cb]);
            }
            acc[rb][cb] = mfma32x32x16<DT>(w, it.u[ks][rb][0], acc[rb][cb]);
            acc[rb][cb] = mfma32x32x16<DT>(w, it.u[ks][rb][1], acc[rb][cb]);
          }
        }
    }
  };
  Item none{};
  none.r0 = t.R;
  Item p = next(none);
  if constexpr (!DEEP) {
    for (; p.a >= 0; p = next(p)) multiply(p);
    return;
  }
  while (p.a >= 0) {
    const Item q = next(p);
    multiply(p);
    if (q.a < 0) break;
    p = next(q);
    multiply(q);
  }
}

}  // namespace w4a16
