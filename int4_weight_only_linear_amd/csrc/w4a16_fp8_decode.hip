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
  int tokens;          // whose codes LDS holds: min(16, M)
  int64_t wexpert, wsexpert;
  bool f16;
};

// Sixteen rows of A times sixteen columns of B over 128 k (see mfma_fp8 of the
// tiles): lane l holds row (column) l % 16, and D[4 (l / 16) + r][l % 16].
__device__ __forceinline__ f32x4 mfma16(i32x8 a, i32x8 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

// A workgroup owns 16 TN features and up to sixteen tokens.  Its waves take the
// blocks of 128 k in turn, weights straight into the operands (lane l: row
// l % 16, k 16 (l / 16) .. of either half of the block), DEPTH blocks ahead.
// Meanwhile, before the first product, they quantise the tokens into LDS (rows
// 16 bytes longer than their codes, so that sixteen rows' pieces of one k meet
// all banks); given codes are read where they are.  The waves' sums are added
// through LDS in wave order.
// Experts: workgroup (slot, features) does the products of its slot's expert for
// that slot and the next ones of the same expert, sixteen together, where an
// even sixteen of them come before it, and nothing otherwise; so an expert's
// weights are read once for sixteen of its slots, without a list made before.
// Bound by memory where the weights are many (8 tokens, 8 of 128 experts, 2048 x 1536, 35
// us, 4.7 TB/s), by the latency of a launch and two trips to memory where they are
// few (4096 x 4096, one token: 6.2 us in the kernel, 3.4 of them its bytes).  One
// launch: quantising first took 14.9 us for that token, 8.1 now.
template <int DT, bool E8M0, int TN>
__global__ __launch_bounds__(1024) void fp8_decode_kernel(DecodeParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  constexpr int DEPTH = 4, BN = 16 * TN;
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int tiles = (p.N + BN - 1) / BN;
  const int n0 = (p.ids ? (int)(blockIdx.x % tiles) : (int)blockIdx.x) * BN;

  int expert = 0, slot = col, count = p.M;
  if (p.ids) {
    const int s = blockIdx.x / tiles;
    expert = p.ids[s];
    if (expert < 0 || expert >= p.E) {  // no expert: zeros
      if (threadIdx.x < BN && n0 + threadIdx.x < p.N) p.y[(size_t)s * p.N + n0 + threadIdx.x] = 0;
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
  const uint8_t* const we = p.w + expert * p.wexpert;
  const int64_t ws0 = expert * p.wsexpert + (int64_t)(n0 >> 7) * p.wsrow;
  uint32_t wrow[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) wrow[t] = (uint32_t)min(n0 + 16 * t + col, p.N - 1) * (uint32_t)p.K;
  u32x4 wv[DEPTH][TN][2];
  uint32_t wsv[DEPTH];  // the blocks' scales, as they are
  auto load = [&](int b, u32x4 (&v)[TN][2], uint32_t& scale) {
    if constexpr (E8M0) scale = static_cast<const uint8_t*>(p.ws)[ws0 + b];
    else scale = static_cast<const uint32_t*>(p.ws)[ws0 + b];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // past the last k: bytes of the same row, which meet zero codes
      const uint32_t at = min(128 * b + 64 * h + 16 * quad, p.K - 16);
#pragma unroll
      for (int t = 0; t < TN; ++t) v[t][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(we + wrow[t] + at));
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (wave + waves * d < p.blocks) load(wave + waves * d, wv[d], wsv[d]);

  const bool live = col < count;
  const int stride = 128 * p.blocks + 16;
  unsigned char* const lds_scales = lds + p.tokens * stride;  // [tokens][blocks]
  if constexpr (DT != DT_CODES) {
    // runs of 512 values, eight a lane, as the quantisation kernel takes them
    const int per_row = (p.blocks + 3) >> 2;
    for (int run = wave; run < count * per_row; run += waves) {
      const int t = run / per_row, k = 512 * (run - t * per_row) + 8 * lane;
      const int64_t row = p.ids ? __builtin_amdgcn_readlane(slot, t) / p.topk : t;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (k < p.K) v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + row * p.K + k);
      int e;
      const u32x2 c = quantize_run<DT>(v, e);
      if (k < 128 * p.blocks) {
        *reinterpret_cast<u32x2*>(lds + t * stride + k) = c;
        if (col == 0) lds_scales[t * p.blocks + (k >> 7)] = (unsigned char)(e + 127);
      }
    }
    __syncthreads();
  }
  const int64_t row = DT == DT_CODES && live ? (p.ids ? slot / p.topk : slot) : 0;
  f32x4 acc[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b0 = wave; b0 < p.blocks; b0 += waves * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int b = b0 + waves * d;
      if (b >= p.blocks) break;
      u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = x0;
      int xsb = 127;
      if (live) {
        const unsigned char* const src = (DT == DT_CODES ? static_cast<const unsigned char*>(p.x) + row * (128 * p.blocks)
                                                         : lds + col * stride) + 128 * b + 16 * quad;
        x0 = *reinterpret_cast<const u32x4*>(src), x1 = *reinterpret_cast<const u32x4*>(src + 64);
        xsb = DT == DT_CODES ? p.xs[row * p.xsrow + b] : lds_scales[col * p.blocks + b];
      }
      const i32x8 xo = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
      float wsf = 1.f;
      int wsb = 127;
      if constexpr (E8M0) {
        wsb = (int)wsv[d];
      } else {
        // the scale's power of two goes to the matrix unit, so that a block's sum stays in range wherever its
        // product with the scale does (zero, infinite, NaN: 1/2; subnormal: 2^-126)
        const float whole = __builtin_bit_cast(float, wsv[d]);
        const int e = max(__builtin_amdgcn_frexp_expf(whole), -125);
        wsb = e + 126;
        wsf = __builtin_amdgcn_ldexpf(whole, 1 - e);
      }
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        i32x8 wo;
#pragma unroll
        for (int i = 0; i < 8; ++i) wo[i] = (int)wv[d][t][i / 4][i % 4];
        if constexpr (E8M0) {
          acc[t] = mfma16(wo, xo, acc[t], wsb, xsb);
        } else {
          const f32x4 v = mfma16(wo, xo, f32x4{0.f, 0.f, 0.f, 0.f}, wsb, xsb);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(v[i], wsf, acc[t][i]);
        }
      }
      if (b + waves * DEPTH < p.blocks) load(b + waves * DEPTH, wv[d], wsv[d]);
    }
  }
  float* const red = reinterpret_cast<float*>(lds);
  if constexpr (DT != DT_CODES) __syncthreads();  // (the codes have been read)
  // red[wave][token][feature]
#pragma unroll
  for (int t = 0; t < TN; ++t)
    *reinterpret_cast<f32x4*>(red + wave * 16 * BN + col * BN + 16 * t + 4 * quad) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * BN; i += blockDim.x) {
    const int t = i / BN, n = n0 + i % BN;
    // (whole waves: 16 BN values are a number of them)
    const int s = p.ids ? __shfl(slot, t) : t;
    if (t >= count || n >= p.N) continue;
    float v = 0.f;
    for (int u = 0; u < waves; ++u) v += red[u * 16 * BN + i];
    if (p.bias) {
      const uint16_t bits = p.bias[(size_t)expert * p.N + n];
      v += p.f16 ? act_to_f32<DT_F16>(bits) : act_to_f32<DT_BF16>(bits);
    }
    if (p.slot_weights) v *= p.slot_weights[s];
    p.y[(size_t)s * p.N + n] = p.f16 ? f32_to_act<DT_F16>(v) : f32_to_act<DT_BF16>(v);
  }
}

// codes of the tokens and their scales
size_t decode_lds(int64_t tokens, int64_t blocks) { return (size_t)(tokens * (129 * blocks + 16)); }

template <int DT, int TN>
void launch_decode(const DecodeParams& p, bool e8m0, int64_t slots, int waves, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * TN - 1) / (16 * TN) * slots)), block(64 * waves);
  const size_t lds = std::max((size_t)waves * 256 * TN * sizeof(float), DT == DT_CODES ? 0 : decode_lds(p.tokens, p.blocks));
  if (e8m0) hipLaunchKernelGGL((fp8_decode_kernel<DT, true, TN>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((fp8_decode_kernel<DT, false, TN>), grid, block, lds, s, p);
}

}  // namespace

// Where this kernel beats the tiles, us of both: 4096 x 4096 7.2 and 11.0 with one
// token, 10.7 and 11.5 with 8, 11.0 and 11.4 with 9 (left to the tiles); 4096 x
// 28672 27.6 and 29.4 with 2, 32.6 and 29.6 with 4; 14336 x 4096 21.9 and 23.6 with
// 8.  64 experts of 4096 x 2048, 8 a token: 106 and 116 with 16 tokens (2 slots an
// expert), 133 and 124 with 24.
bool fp8_decodes(int64_t M, int64_t N, int64_t K, int E, bool experts, bool transpose) {
  if (transpose) return false;
  if (!experts) return M <= 2 || (M <= 8 && N * K <= int64_t(1) << 26);
  return M <= 1024 && M <= 2 * (int64_t)E && M * ((N + 15) / 16) <= kMaxFp8Tiles;
}

// The codes of a workgroup's tokens leave room for a second workgroup on a CU;
// longer rows are quantised by a launch of their own.
bool fp8_decode_quantizes(int64_t M, int64_t K) {
  return decode_lds(std::min<int64_t>(16, M), fp8_columns(K) / kFp8Block) <= 80 * 1024;
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
  p.tokens = (int)std::min<int64_t>(16, a.M);
  p.wsrow = p.blocks;
  p.wexpert = a.N * a.K;
  p.wsexpert = (a.N + kFp8Block - 1) / kFp8Block * p.blocks;
  p.f16 = a.dtype == DT_F16;
  const int64_t slots = ids ? a.M : 1;
  // four blocks to a wave, all of them on their way at once; 32 features a workgroup where 16 would give
  // more than eight for each CU (64 experts of 4096 x 2048: 54.2 us with 32, 58.8 with 16 for 32 slots, 78.7 and
  // 92.9 for 64)
  const int waves = std::clamp((p.blocks + 3) / 4, 1, 16);
  const bool two = (a.N + 31) / 32 * slots >= 1024;
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (two && ids) launch_decode<DT, 2>(p, a.e8m0, slots, waves, s);
    else launch_decode<DT, 1>(p, a.e8m0, slots, waves, s);
  };
  if (x_dtype == DT_F16) go(std::integral_constant<int, DT_F16>{});
  else if (x_dtype == DT_BF16) go(std::integral_constant<int, DT_BF16>{});
  else go(std::integral_constant<int, DT_CODES>{});
  return hipGetLastError();
}

}  // namespace w4a16
