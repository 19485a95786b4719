// Products of 8-bit weights for few tokens: one layer's decode, and the decode
// of routed experts.
#include <algorithm>

#include "w4a16_experts.h"
#include "w4a16_fp8.hpp"

namespace w4a16 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

enum { DT_CODES = 2 };

struct DecodeParams {
  const void* x;       // codes, or activations that the kernel quantises
  const uint8_t* xs;
  const uint8_t* w;
  const void* ws;
  const uint16_t* bias;
  uint16_t* y;
  const int32_t* ids;  // experts: [slots], or NULL (one layer)
  const float* slot_weights;
  int M, N, K, E, topk;
  int blocks, xsrow, wsrow;
  int64_t wexpert, wsexpert;
  bool f16;
};

// Sixteen rows of A times sixteen columns of B over 128 k (see mfma_fp8 of the
// tiles): lane l holds row (column) l % 16, and D[4 (l / 16) + r][l % 16].
__device__ __forceinline__ f32x4 mfma16(i32x8 a, i32x8 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

// A workgroup owns sixteen features and up to sixteen tokens; its waves take the
// blocks of 128 k in turn, load weights and tokens straight into the operands
// (lane l: row l % 16, k 16 (l / 16) .. of either half of the block), quantise
// the tokens there, and are added through LDS in wave order.
// Experts: workgroup (slot, features) does the products of its slot's expert for
// that slot and the next ones of the same expert, sixteen together, where an
// even sixteen of them come before it, and nothing otherwise; so an expert's
// weights are read once for sixteen of its slots, without a list made before.
template <int DT, bool E8M0>
__global__ __launch_bounds__(1024) void fp8_decode_kernel(DecodeParams p) {
  extern __shared__ __attribute__((aligned(16))) float red[];
  constexpr int DEPTH = DT == DT_CODES ? 4 : 2;  // blocks loaded before they are multiplied
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int tiles = (p.N + 15) >> 4;
  const int n0 = (p.ids ? (int)(blockIdx.x % tiles) : (int)blockIdx.x) * 16;

  int expert = 0, slot = col, count = p.M;
  if (p.ids) {
    const int s = blockIdx.x / tiles;
    expert = p.ids[s];
    if (expert < 0 || expert >= p.E) {  // no expert: zeros
      if (threadIdx.x < 16 && n0 + threadIdx.x < p.N) p.y[(size_t)s * p.N + n0 + threadIdx.x] = 0;
      return;
    }
    // lane j < 16: the j-th slot of this expert from s on
    int before = 0;
    count = 0;
    slot = s;
    for (int base = 0; base < p.M; base += 64) {
      const int i = base + lane;
      const uint64_t own = __ballot(i < p.M && p.ids[min(i, p.M - 1)] == expert);
      const uint64_t below = s <= base ? 0 : (s - base >= 64 ? ~0ull : (1ull << (s - base)) - 1);
      before += __popcll(own & below);
      uint64_t here = own & ~below;
      if (base + 64 > s && (before & 15)) break;  // (another workgroup's)
      while (here && count < 16) {
        if (lane % 16 == count) slot = base + __builtin_ctzll(here);
        here &= here - 1;
        ++count;
      }
      if (count == 16) break;
    }
    if (before & 15) return;
  }
  const bool live = col < count;
  const int64_t row = live ? (p.ids ? slot / p.topk : slot) : 0;
  const uint8_t* const wrow = p.w + expert * p.wexpert + (int64_t)min(n0 + col, p.N - 1) * p.K;
  const int64_t ws0 = expert * p.wsexpert + (int64_t)(n0 >> 7) * p.wsrow;

  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b0 = wave; b0 < p.blocks; b0 += waves * DEPTH) {
    u32x4 wv[DEPTH][2], xv[DEPTH][DT == DT_CODES ? 2 : 4];
    int xsb[DEPTH];
    float wsf[DEPTH];
    int wsb[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int b = min(b0 + waves * d, p.blocks - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // past the last k: bytes of the same row, which meet zero codes
        const int k = 128 * b + 64 * h + 16 * quad;
        wv[d][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow + min(k, p.K - 16)));
        if constexpr (DT == DT_CODES) {
          xv[d][h] = u32x4{0u, 0u, 0u, 0u};
          if (live) xv[d][h] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p.x) + row * (128 * p.blocks) + k);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            xv[d][2 * h + q] = u32x4{0u, 0u, 0u, 0u};
            if (live && k < p.K)
              xv[d][2 * h + q] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + row * p.K + k + 8 * q);
          }
        }
      }
      if constexpr (DT == DT_CODES) xsb[d] = p.xs[row * p.xsrow + b];
      if constexpr (E8M0) wsb[d] = static_cast<const uint8_t*>(p.ws)[ws0 + b];
      else wsf[d] = static_cast<const float*>(p.ws)[ws0 + b];
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (b0 + waves * d >= p.blocks) break;
      i32x8 xo;
      if constexpr (DT == DT_CODES) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xo[i] = (int)xv[d][i / 4][i % 4];
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t v = xv[d][i / 4][i % 4];
          top = max(top, max(finite_bits<DT>(v), finite_bits<DT>(v >> 16)));
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const int e = block_exponent<DT>(top);
        const float scale = exp2_int(e);
        xsb[d] = e + 127;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          short2_t c = {0, 0};
          c = codes_of<DT, false>(c, xv[d][i / 2][2 * (i % 2)], scale);
          c = codes_of<DT, true>(c, xv[d][i / 2][2 * (i % 2) + 1], scale);
          xo[i] = __builtin_bit_cast(int, c);
        }
      }
      i32x8 wo;
#pragma unroll
      for (int i = 0; i < 8; ++i) wo[i] = (int)wv[d][i / 4][i % 4];
      if constexpr (E8M0) {
        acc = mfma16(wo, xo, acc, wsb[d], xsb[d]);
      } else {
        const f32x4 v = mfma16(wo, xo, f32x4{0.f, 0.f, 0.f, 0.f}, 127, xsb[d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(v[i], wsf[d], acc[i]);
      }
    }
  }
  // red[wave][token][feature]
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave * 256 + col * 16 + 4 * quad + i] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 256; i += blockDim.x) {
    const int t = i >> 4, n = n0 + (i & 15);
    // (whole waves: 256 values are four of them)
    const int s = p.ids ? __shfl(slot, t) : t;
    if (t >= count || n >= p.N) continue;
    float v = 0.f;
    for (int u = 0; u < waves; ++u) v += red[u * 256 + i];
    if (p.bias) {
      const uint16_t bits = p.bias[(size_t)expert * p.N + n];
      v += p.f16 ? act_to_f32<DT_F16>(bits) : act_to_f32<DT_BF16>(bits);
    }
    if (p.slot_weights) v *= p.slot_weights[s];
    p.y[(size_t)s * p.N + n] = p.f16 ? f32_to_act<DT_F16>(v) : f32_to_act<DT_BF16>(v);
  }
}

template <int DT>
void launch_decode(const DecodeParams& p, bool e8m0, dim3 grid, int waves, hipStream_t s) {
  const size_t lds = (size_t)waves * 256 * sizeof(float);
  if (e8m0) hipLaunchKernelGGL((fp8_decode_kernel<DT, true>), grid, dim3(64 * waves), lds, s, p);
  else hipLaunchKernelGGL((fp8_decode_kernel<DT, false>), grid, dim3(64 * waves), lds, s, p);
}

}  // namespace

bool fp8_decodes(int64_t M, int64_t N, int64_t K, int E, bool experts, bool transpose) {
  if (transpose) return false;
  if (!experts) return M <= 16;
  return M <= 1024 && M <= 4 * (int64_t)E && M * ((N + 15) / 16) <= kMaxFp8Tiles;
}

hipError_t launch_fp8_decode(const Fp8Args& a, const void* x, int x_dtype, const int32_t* ids, hipStream_t s) {
  DecodeParams p{};
  p.x = x;
  p.xs = a.xs;
  p.w = a.w;
  p.ws = a.ws;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.y = static_cast<uint16_t*>(a.y);
  p.ids = ids;
  p.slot_weights = a.slot_weights;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)a.K;
  p.E = a.E;
  p.topk = a.topk;
  p.blocks = (int)(fp8_columns(a.K) / kFp8Block);
  p.xsrow = (int)fp8_scales(a.K);
  p.wsrow = p.blocks;
  p.wexpert = a.N * a.K;
  p.wsexpert = (a.N + kFp8Block - 1) / kFp8Block * p.blocks;
  p.f16 = a.dtype == DT_F16;
  const int waves = std::clamp((p.blocks + 1) / 2, 1, 16);
  const dim3 grid((unsigned)((a.N + 15) / 16 * (ids ? a.M : 1)));
  if (x_dtype == DT_F16) launch_decode<DT_F16>(p, a.e8m0, grid, waves, s);
  else if (x_dtype == DT_BF16) launch_decode<DT_BF16>(p, a.e8m0, grid, waves, s);
  else launch_decode<DT_CODES>(p, a.e8m0, grid, waves, s);
  return hipGetLastError();
}

}  // namespace w4a16
