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
// before the waves are added: no further barrier, and every wave's loads are
// under way at once.  add(m, value) is called by all lanes with the term of
// row lane & 15, so that the lanes that hold token m's sums add it in their
// registers (in LDS they would have to wait for other lanes' stores).  A lane
// takes every fourth run of eight ranks of one row; the K ranges of u are read
// four at a time, so that their loads overlap.
// Bound by that one chain of loads: 3 us of 15.3 with 16 tokens of 16 adapters,
// ranks of 16, 4096 x 6144 (12.3 without adapters; spread over the projection's
// K ranges as well 15.1).
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
    add(m, s * alpha);
  }
}

// Eight fp32 values as two MFMA operands whose sum is the value to about 16
// (bf16) or 22 (fp16) significant bits: v rounded, and what that left.  One
// operand alone would add a rounding of u as large as the output's own.
// fp16's remainder ends at 2^-24, so a row of values is first moved to where
// that is far below them (op_shift).
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

// The power of two that a row of fp16 operands is multiplied by, from its
// largest magnitude: the multiple of 16 that takes it into [2^-2, 2^14), so that
// the row is held to 2^-23 of its largest value whatever its size (without it
// values of 1e-6 keep five bits, and 65504 is the largest).  The accumulators
// that such operands are added to are moved by the same power before, and back
// afterwards: exact, and not needed for rows already in that range, which most
// are (steps of 16 also keep the rows of a sum at few different shifts).
// Values below 2^-66 are as good as zero to fp16 outputs: at most 64.  Zeros,
// infinities and NaN are left as they are.  (Calls of 1920 tokens, 4096 x 28672,
// with it: forward 442 -> 448 us, 459 where rows are moved; the input gradient
// 413 -> 417, 425.)
__device__ __forceinline__ int op_shift(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);  // of a magnitude
  return top_bits == 0 || e == 255 ? 0 : min(64, -16 * ((e - 125) >> 4));
}
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

typedef __attribute__((address_space(3))) unsigned char lds_bytes;
typedef __attribute__((address_space(3))) u32x4 lds_piece;
typedef uint16_t uint16x2_t __attribute__((ext_vector_type(2)));

// A tile's rows of t.op into LDS: 256 bytes a token, values from hi(token) and
// remainders from lo(token), eight ranks (piece p) at p ^ (token & 15), so that
// the operand reads of 16 tokens touch 16 different banks of 16 bytes.  Rows of
// tokens without an adapter hold anything (lora_steps reads none of them).
// Begins and ends with a barrier.
template <typename Hi, typename Lo>
__device__ __forceinline__ void lora_stage(const LoraTerm& t, int M, int m0, int tokens, int tid, int threads, Hi&& hi,
                                           Lo&& lo) {
  constexpr int B = 8;  // pieces in flight per thread
  const int pieces = t.R >> 3, total = tokens * 2 * pieces;
  __syncthreads();  // the buffers are free
  for (int i0 = tid; i0 < total; i0 += threads * B) {
    u32x4 v[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = min(i0 + b * threads, total - 1), m = i / (2 * pieces), p = i - m * 2 * pieces;
      v[b] = *reinterpret_cast<const u32x4*>(t.op + (size_t)min(m0 + m, M - 1) * 2 * t.R + 8 * p);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = min(i0 + b * threads, total - 1), m = i / (2 * pieces), p = i - m * 2 * pieces;
      *(lds_piece*)((p < pieces ? hi(m) : lo(m)) + 16 * ((p < pieces ? p : p - pieces) ^ (m & 15))) = v[b];
    }
  }
  __syncthreads();
}

// The GEMM tile's adapter term, as more k of its product: for every adapter
// that a token of the tile names (in the order of their first tokens),
// ceil(R / 16) k-subs whose A operand is the wave's rows of up_a and whose B
// operand is alpha * u of the adapter's own tokens (from LDS), zero for the
// others; token blocks without such a token are left out.  The K ranges of a
// split tile take the adapters in turns.  A tile of many adapters is a chain
// of items (KS k-subs of one adapter), so the rows of the next two are on
// their way while one is multiplied.  Bound by the adapters' rows, read after
// the weights, and by a wave's instructions: 67 tokens of 16 adapters, ranks of
// 32, 2560 x 19456, fp16: 20.8 us without adapters, 22 with one per K range,
// 29 with all (48 before operands were split once, staged and prefetched);
// 1476 tokens of ten adapters mixed, ranks of 128, 256 x 5584: 112 -> 91 us
// by the LDS and the prefetch (15 without adapters).  1920 tokens of one
// adapter, ranks of 64, 14336 x 4096: 213 us, 208 without; of six, ranks of 16,
// 4096 x 28672: 419 us, 391 without.
//   acc[rb][cb]: tokens m0 + 32 rb + (lane & 31), features nw0 + 32 cb + ...
//   hi, lo: rows of token m0 (lora_stage)
template <int DT, int MB, int CB>
__device__ __forceinline__ void lora_steps(const LoraTerm& t, int M, int N, int m0, int nw0, int lane, int turn, int turns,
                                           const lds_bytes* hi, const lds_bytes* lo, f32x16 (&acc)[MB][CB]) {
  constexpr int KS = MB * CB <= 8 ? 2 : 1;  // registers beside the accumulators
  const int j = lane & 31, h = lane >> 5;
  int id[MB];
  uint64_t todo[MB];
  // fp16: each token's (lane's) sums are moved to the scale of its operands
  auto shift_of = [&](int rb) { return t.shift[min(m0 + 32 * rb + j, M - 1)]; };
  bool scaled = false;
  {
    int shift[MB];
#pragma unroll
    for (int rb = 0; rb < MB; ++rb) {
      id[rb] = lora_id(t, M, m0 + 32 * rb + j);
      shift[rb] = DT == DT_F16 ? shift_of(rb) : 0;
    }
#pragma unroll
    for (int rb = 0; rb < MB; ++rb) {
      todo[rb] = __ballot(id[rb] >= 0);
      scaled |= id[rb] >= 0 && shift[rb] != 0;
    }
    scaled = __ballot(scaled) != 0;
  }
  const uint16_t* const up = static_cast<const uint16_t*>(t.up);
  uint32_t row[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) row[cb] = (uint32_t)min(nw0 + 32 * cb + j, N - 1);
  auto rescale = [&](int sign) {
#pragma unroll
    for (int rb = 0; rb < MB; ++rb) {
      const int sh = id[rb] >= 0 ? sign * shift_of(rb) : 0;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[rb][cb][e] = __builtin_ldexpf(acc[rb][cb][e], sh);
        __builtin_amdgcn_sched_barrier(0);  // (few registers beside the accumulators)
      }
    }
  };
  if (__builtin_expect(scaled, 0)) rescale(1);
  int count = 0;  // adapters of the tile seen so far

  struct Item {
    int a, r0;  // adapter (-1: no more), first rank (of both halves)
    u32x4 w[KS][CB];
  };
  // The item after ranks r0 of adapter a: its next ranks, or the next adapter.
  // The loads stand behind no branch (valid addresses throughout, zeros put in
  // by multiply): behind one their number is unknown, and every wait would be
  // for all of them.
  auto next = [&](int a, int r0, Item& n) {
    r0 += 16 * KS;
    if (a < 0 || r0 >= t.R) {
      r0 = 0;
      do {
        a = -1;
#pragma unroll
        for (int rb = MB - 1; rb >= 0; --rb)
          if (todo[rb]) a = __builtin_amdgcn_readlane(id[rb], __builtin_ctzll(todo[rb]));
        if (a < 0) break;
#pragma unroll
        for (int rb = 0; rb < MB; ++rb) todo[rb] &= ~__ballot(id[rb] == a);
      } while (count++ % turns != turn);
    }
    n.a = a;
    n.r0 = r0;
    const uint16_t* const rows = up + (size_t)max(a, 0) * N * t.R;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int r = min(r0 + 16 * ks + 8 * h, t.R - 8);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) n.w[ks][cb] = *reinterpret_cast<const u32x4*>(rows + (size_t)row[cb] * t.R + r);
    }
  };
  // Other adapters' tokens of a block take part with zeros, which an infinite
  // or NaN factor would turn into NaN.  Where an item holds one, it is taken
  // out of the product and made of finite numbers that overflow for the
  // adapter's own tokens: + and - max * 2^127, in bf16 whose products pass
  // fp32's range; zeros stay zeros.  (Selecting sums by token instead keeps
  // them in vector registers: up to 1150 spilled.  The test costs 8 operations
  // a fragment.)
  auto multiply = [&](const Item& it) {
    constexpr uint32_t INF = DT == DT_F16 ? 0x7C00 : 0x7F80;
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
    const bool broken = __ballot(top[0] >= (uint16_t)INF || top[1] >= (uint16_t)INF) != 0;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // R is a multiple of 8: a last k-sub may lie past it, wholly or its upper half
      if (it.r0 + 16 * ks >= t.R) continue;
      const int piece = (it.r0 >> 3) + 2 * ks + h;
      const bool in = 8 * piece < t.R;
      u32x4 w[CB], bad[CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        w[cb] = in ? it.w[ks][cb] : u32x4{0u, 0u, 0u, 0u};
        if (broken) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t word = w[cb][e];
            const uint32_t mask = ((((word & 0x7FFF7FFFu) + (0x80008000u - 0x10001u * INF)) & 0x80008000u) >> 15) * 0xFFFFu;
            w[cb][e] = word & ~mask;
            bad[cb][e] = mask & 0x7F7F7F7Fu;
          }
        }
      }
#pragma unroll
      for (int rb = 0; rb < MB; ++rb) {
        const bool own = id[rb] == it.a;
        if (__ballot(own) == 0) continue;
        const int at = (32 * rb + j) * 256 + 16 * (piece ^ (j & 15));
        u32x4 x = *(const lds_piece*)(hi + at), y = *(const lds_piece*)(lo + at);
        if (!(own && in)) x = y = u32x4{0u, 0u, 0u, 0u};
        if (broken) {
          const uint32_t big = own ? 0x7F007F00u : 0u, low = own ? 0xFF00FF00u : 0u;
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            acc[rb][cb] = mfma32x32x16<DT_BF16>(bad[cb], u32x4{big, big, big, big}, acc[rb][cb]);
            acc[rb][cb] = mfma32x32x16<DT_BF16>(bad[cb], u32x4{low, low, low, low}, acc[rb][cb]);
          }
        }
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          acc[rb][cb] = mfma32x32x16<DT>(w[cb], x, acc[rb][cb]);
          acc[rb][cb] = mfma32x32x16<DT>(w[cb], y, acc[rb][cb]);
        }
      }
    }
  };
  Item p, q, r;
  next(-1, 0, p);
  next(p.a, p.r0, q);
  while (p.a >= 0) {
    next(q.a, q.r0, r);
    multiply(p);
    if (q.a < 0) break;
    next(r.a, r.r0, p);
    multiply(q);
    if (r.a < 0) break;
    next(p.a, p.r0, q);
    multiply(r);
  }
  if (__builtin_expect(scaled, 0)) rescale(-1);
}

}  // namespace w4a16
