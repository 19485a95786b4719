// The projection's input gradient for gfx950: dx[m, k] = sum_n dy[m, n] W[n, k]
// with the packed 4-bit weights, so that nothing larger than a tile of W is
// ever dequantised (plus the adapters' term, as more n of the same product).
//
// The forward product reduces over k, along which the codes are packed; this
// one reduces over n, across rows.  An MFMA operand wants eight consecutive
// values of the reduction per lane, so the unit of dequantisation is a block
// of 8 rows x 8 k: eight words, one per row.  One v_perm pairs the halves of
// two rows' words, after which (word >> 4i) & 0x000F000F is the pair of rows
// at one k, and the forward's conversions give the two weights of an operand
// register; the block becomes eight 16-byte operands, one per k.
//
// A workgroup (4 waves) owns 64 MW tokens x 256 k and steps over 64 rows at a
// time: every thread dequantises one block into LDS, where the waves (each 32
// MW tokens x 128 k) read them as A operands; dy is staged as B operands by
// direct global->LDS loads.  Both are double buffered, the words of the step
// after next in registers, and one barrier ends a step.  Each weight is
// dequantised once per workgroup.
#include <algorithm>

#include "w4a16_lora.hpp"
#include "w4a16_lora_bwd.hpp"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;
constexpr int kBN = 64;    // rows of W per step
constexpr int kBKX = 256;  // k of a tile
constexpr int kWBytes = kBN * kBKX * 2;  // one buffer of dequantised weights

typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

struct DxParams {
  const uint16_t* dy;
  const uint32_t* wq;
  const uint16_t* scales;
  const uint32_t* zp;
  uint16_t* dx;
  const void* zeros;
  float* partial;
  int M, N, K, ldy;
  int sG, gmul;
  int wpr;      // words per weight row
  int nsteps, tiles_k, units, splits, steps_per_split;
};

// consecutive work units -- the same tokens, neighbouring k -- on one XCD
__device__ __forceinline__ int xcd_unit(int b, int units) {
  const int q = units / 8, r = units % 8, xcd = b % 8, local = b / 8;
  return xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
}

// the words, scales and zero points of one 8 x 8 block
struct Block {
  uint32_t w[8];
  uint16_t s[8];
  uint32_t z;
};

template <int DT, int GS, bool ASYM, int MW>
__global__ __launch_bounds__(kThreads) void dx_kernel(const DxParams p, const LoraTerm lora) {
  constexpr int BM = 64 * MW;
  constexpr int DYB = BM * kBN * 2;       // one dy buffer
  constexpr int NDMA = BM / 32;           // 1 KiB dy loads per wave and step
  __shared__ __attribute__((aligned(1024))) unsigned char ws0[kWBytes];
  __shared__ __attribute__((aligned(1024))) unsigned char ws1[kWBytes];
  __shared__ __attribute__((aligned(1024))) unsigned char ds0[DYB];
  __shared__ __attribute__((aligned(1024))) unsigned char ds1[DYB];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane & 31, h = lane >> 5;
  const int unit = xcd_unit(blockIdx.x, p.units);
  const int tile = unit / p.splits, split = unit - tile * p.splits;
  const int mt = tile / p.tiles_k, kt = tile - mt * p.tiles_k;
  const int m0 = mt * BM, k0 = kt * kBKX;
  const int s_begin = split * p.steps_per_split;
  const int s_end = min(p.nsteps, s_begin + p.steps_per_split);

  // ---- dy: load d of this wave fills LDS rows (wave NDMA + d) 8 + lane / 8;
  // position lane & 7 of a row holds its piece pos ^ (row & 7)
  const uint16_t* dyrow[NDMA];
  const int piece = (lane & 7) ^ ((lane >> 3) & 7);
#pragma unroll
  for (int d = 0; d < NDMA; ++d)
    dyrow[d] = p.dy + (size_t)min(m0 + (wave * NDMA + d) * 8 + (lane >> 3), p.M - 1) * p.ldy + 8 * piece;
  auto stage_dy = [&](int s, lds_u8* buf) {
    const bool in = s * kBN + 8 * piece < p.ldy;  // (dy is zero from N up to ldy)
#pragma unroll
    for (int d = 0; d < NDMA; ++d) {
      const void* src = in ? static_cast<const void*>(dyrow[d] + s * kBN) : p.zeros;
      __builtin_amdgcn_global_load_lds(src, buf + (wave * NDMA + d) * 1024, 16, 0, 0);
    }
  };

  // ---- weights: this thread's block is rows 8 o.. of the step, slice c of the tile
  const int c = tid & 31, o = tid >> 5;
  const int slice = min((k0 >> 3) + c, p.wpr - 1);
  const int g = (8 * slice) / GS * p.gmul;
  const int runs = p.wpr >> 4, tail = p.wpr & 15;
  const bool full_run = (slice >> 4) < runs;
  const int sl = slice & 15;
  // place of the slice in a complete tile of 16 rows, and in a row kept alone
  const uint32_t in_tile = full_run ? 256u * (uint32_t)(slice >> 4) + 64u * (uint32_t)(sl & 3) + (uint32_t)(sl >> 2)
                                    : 256u * (uint32_t)runs + (uint32_t)(slice - 16 * runs);
  const uint32_t tile_stride = full_run ? 4u : (uint32_t)tail;
  const uint32_t in_row = full_run ? (uint32_t)(slice - sl) + 4u * (uint32_t)(sl & 3) + (uint32_t)(sl >> 2) : (uint32_t)slice;
  auto load_block = [&](int s, Block& b) {
    const int n = s * kBN + 8 * o;
    const bool whole = (n | 15) < p.N;  // the block's 16-row tile is complete
    const uint32_t row16 = (uint32_t)(n & ~15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t at = whole ? row16 * (uint32_t)p.wpr + in_tile + (uint32_t)((n & 8) + i) * tile_stride
                                : (uint32_t)min(n + i, p.N - 1) * (uint32_t)p.wpr + in_row;
      b.w[i] = p.wq[at];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(n + i, p.N - 1);
      b.s[i] = p.scales[(size_t)r * p.sG + g];
      if (n + i >= p.N) b.s[i] = 0;  // rows past N weigh nothing
    }
    if constexpr (ASYM) b.z = p.zp[(size_t)(min(n, p.N - 1) >> 3) * p.sG + g];
  };
  // the block's eight operands (k = 0..7 of the slice) at [octet o][slice c][k ^ (c & 7)]
  auto put_block = [&](const Block& b, lds_u8* buf) {
    uint32_t out[8][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t z0 = ASYM ? (b.z >> (8 * q)) & 15u : 8u, z1 = ASYM ? (b.z >> (8 * q + 4)) & 15u : 8u;
      const uint32_t half[2] = {__builtin_amdgcn_perm(b.w[2 * q + 1], b.w[2 * q], 0x05040100u),
                                __builtin_amdgcn_perm(b.w[2 * q + 1], b.w[2 * q], 0x07060302u)};
      if constexpr (DT == DT_F16) {
        const uint32_t nmz = (Magic<DT_F16>::neg | z0) | ((Magic<DT_F16>::neg | z1) << 16);
        const half2_t sp = __builtin_bit_cast(half2_t, (uint32_t)b.s[2 * q] | ((uint32_t)b.s[2 * q + 1] << 16));
#pragma unroll
        for (int H = 0; H < 2; ++H)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            half2_t v = __builtin_bit_cast(half2_t, magic_pair<DT_F16>(half[H], i));
            v = v + __builtin_bit_cast(half2_t, nmz);
            v = v * sp;
            out[2 * i + H][q] = __builtin_bit_cast(uint32_t, v);
          }
      } else {
        const GroupConst<DT> g0 = group_const<DT, true>(b.s[2 * q], z0), g1 = group_const<DT, true>(b.s[2 * q + 1], z1);
#pragma unroll
        for (int H = 0; H < 2; ++H) {
          const uint32_t ev = mask_nibbles(half[H]), od = mask_nibbles(half[H] >> 4);
          const f32x2 e0 = __builtin_amdgcn_cvt_pk_f32_fp8(ev, false), e1 = __builtin_amdgcn_cvt_pk_f32_fp8(ev, true);
          const f32x2 o0 = __builtin_amdgcn_cvt_pk_f32_fp8(od, false), o1 = __builtin_amdgcn_cvt_pk_f32_fp8(od, true);
          auto pair = [&](float a, float b2) {
            return f32x2_to_act_pair<DT_BF16>(__builtin_fmaf(a, g0.s_f32, g0.c_f32), __builtin_fmaf(b2, g1.s_f32, g1.c_f32));
          };
          out[0 + H][q] = pair(e0[0], e1[0]);
          out[2 + H][q] = pair(o0[0], o1[0]);
          out[4 + H][q] = pair(e0[1], e1[1]);
          out[6 + H][q] = pair(o0[1], o1[1]);
        }
      }
    }
    typedef __attribute__((address_space(3))) u32x4 lds_out;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *(lds_out*)(buf + (uint32_t)(((o * 32 + c) * 8 + (k ^ (c & 7))) * 16)) = u32x4{out[k][0], out[k][1], out[k][2], out[k][3]};
  };

  const int wk = wave & 1, wm = wave >> 1;
  f32x16 acc[MW][4];
#pragma unroll
  for (int mb = 0; mb < MW; ++mb)
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[mb][kb][e] = 0.f;
  // operand addresses: k = 128 wk + 32 kb + j is slice 16 wk + 4 kb + j / 8, value j & 7
  const int cl = 16 * wk + (j >> 3);
  auto multiply = [&](const lds_u8* wbuf, const lds_u8* dbuf) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4 a[4], b[MW];
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const int cc = cl + 4 * kb;
        a[kb] = *(lds_u32x4*)(wbuf + (uint32_t)((((2 * ks + h) * 32 + cc) * 8 + ((j & 7) ^ (cc & 7))) * 16));
      }
#pragma unroll
      for (int mb = 0; mb < MW; ++mb)
        b[mb] = *(lds_u32x4*)(dbuf + (uint32_t)((wm * MW + mb) * 32 + j) * 128u + (uint32_t)(((2 * ks + h) ^ (j & 7)) * 16));
#pragma unroll
      for (int mb = 0; mb < MW; ++mb)
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) acc[mb][kb] = mfma32x32x16<DT>(a[kb], b[mb], acc[mb][kb]);
    }
  };

  lds_u8* const w0 = (lds_u8*)ws0;
  lds_u8* const w1 = (lds_u8*)ws1;
  lds_u8* const d0 = (lds_u8*)ds0;
  lds_u8* const d1 = (lds_u8*)ds1;
  if (s_begin < s_end) {
    Block b0 = {}, b1 = {};
    const int last = s_end - 1;
    load_block(s_begin, b0);
    stage_dy(s_begin, d0);
    load_block(min(s_begin + 1, last), b1);
    put_block(b0, w0);
    wait_vm_all();
    __syncthreads();
    // step s multiplies from (w0, d0) while step s + 1 is staged and
    // dequantised into (w1, d1); its words (b1) were loaded one step before
    auto step = [&](int s, lds_u8* wc, lds_u8* dc, lds_u8* wn, lds_u8* dn, Block& next, Block& after) {
      stage_dy(min(s + 1, last), dn);
      load_block(min(s + 2, last), after);
      multiply(wc, dc);
      put_block(next, wn);
      wait_vm_all();
      __syncthreads();
    };
    int s = s_begin;
    for (; s + 1 < s_end; s += 2) {
      step(s, w0, d0, w1, d1, b1, b0);
      step(s + 1, w1, d1, w0, d0, b0, b1);
    }
    if (s < s_end) multiply(w0, d0);
  }
  lora_steps<DT, MW, 4>(lora, p.M, p.K, m0 + 32 * MW * wm, k0 + 128 * wk, lane, split, p.splits, acc);

  // acc[mb][kb][4a + e]: token m0 + 32 (MW wm + mb) + j, k = k0 + 128 wk + 32 kb + 8a + 4h + e
#pragma unroll
  for (int mb = 0; mb < MW; ++mb) {
    const int m = m0 + 32 * (MW * wm + mb) + j;
    if (p.splits > 1) {
      float* const part = p.partial + ((size_t)split * p.M + m) * p.K;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int k = k0 + 128 * wk + 32 * kb + 8 * a + 4 * h;
          const f32x16& v = acc[mb][kb];
          if (m < p.M && k < p.K)
            *reinterpret_cast<f32x4*>(part + k) = f32x4{v[4 * a], v[4 * a + 1], v[4 * a + 2], v[4 * a + 3]};
        }
      continue;
    }
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t q[4][2];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x16& v = acc[mb][kb];
        q[a][0] = f32x2_to_act_pair<DT>(v[4 * a], v[4 * a + 1]);
        q[a][1] = f32x2_to_act_pair<DT>(v[4 * a + 2], v[4 * a + 3]);
      }
      // the lanes of a pair of quads swap halves: 8 consecutive k each
#pragma unroll
      for (int a = 0; a < 4; a += 2) {
        const auto x0 = __builtin_amdgcn_permlane32_swap(q[a][0], q[a + 1][0], false, false);
        const auto x1 = __builtin_amdgcn_permlane32_swap(q[a][1], q[a + 1][1], false, false);
        const int k = k0 + 128 * wk + 32 * kb + 8 * (a + h);
        if (m < p.M && k < p.K) *reinterpret_cast<u32x4*>(p.dx + (size_t)m * p.K + k) = u32x4{x0[0], x1[0], x0[1], x1[1]};
      }
    }
  }
}

template <int DT, int GS, bool ASYM>
hipError_t launch_mw(const DxParams& prm, const LoraTerm& lora, int mw, hipStream_t s) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(prm.units), dim3(kThreads), 0, s, prm, lora);
    return hipGetLastError();
  };
  switch (mw) {
    case 1: return go(dx_kernel<DT, GS, ASYM, 1>);
    case 2: return go(dx_kernel<DT, GS, ASYM, 2>);
    case 4: return go(dx_kernel<DT, GS, ASYM, 4>);
    default: return hipErrorInvalidValue;
  }
}

template <int DT>
hipError_t launch_g(const DxParams& prm, const LoraTerm& lora, int group, int mw, hipStream_t s) {
  const bool z = prm.zp != nullptr;
  switch (group) {
    case 32: return z ? launch_mw<DT, 32, true>(prm, lora, mw, s) : launch_mw<DT, 32, false>(prm, lora, mw, s);
    case 64: return z ? launch_mw<DT, 64, true>(prm, lora, mw, s) : launch_mw<DT, 64, false>(prm, lora, mw, s);
    case 128: return z ? launch_mw<DT, 128, true>(prm, lora, mw, s) : launch_mw<DT, 128, false>(prm, lora, mw, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

DxPlan plan_dx(int64_t M, int64_t N, int64_t K, int cu_count) {
  DxPlan best{};
  double best_t = 0.0;
  const int nsteps = (int)((N + kBN - 1) / kBN);
  const int64_t tiles_k = (K + kBKX - 1) / kBKX;
  for (int mw : {4, 2, 1}) {
    const int64_t tiles = (M + 64 * mw - 1) / (64 * mw) * tiles_k;
    for (int splits = 1; splits <= 16 && splits <= nsteps; ++splits) {
      const int sps = (nsteps + splits - 1) / splits;
      if ((nsteps + sps - 1) / sps != splits) continue;
      const int64_t rounds = (tiles * splits + cu_count - 1) / cu_count;
      const double t = rounds * (sps * (0.35 + 0.35 * mw) + 2.0) +
                       (splits > 1 ? 3.0 + (double)(splits + 1) * M * K * 4.0 / 3e6 : 0.0);
      if (best.tiles == 0 || t < best_t) {
        best_t = t;
        best = DxPlan{mw, splits, sps, (int)tiles_k, (int)tiles};
      }
    }
  }
  return best;
}

size_t dx_partial_bytes(const DxPlan& p, int64_t M, int64_t K) {
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)K * sizeof(float) : 0;
}

hipError_t launch_dx(const DxArgs& a, const DxPlan& p, const LoraTerm& lora, hipStream_t s) {
  if ((int64_t)p.tiles * p.splits > INT32_MAX) return hipErrorInvalidValue;
  DxParams prm;
  prm.dy = a.dy;
  prm.wq = reinterpret_cast<const uint32_t*>(a.wq);
  prm.scales = static_cast<const uint16_t*>(a.scales);
  prm.zp = reinterpret_cast<const uint32_t*>(a.zp);
  prm.dx = static_cast<uint16_t*>(a.dx);
  prm.zeros = a.zeros;
  prm.partial = a.partial;
  prm.M = (int)a.M;
  prm.N = (int)a.N;
  prm.K = (int)a.K;
  prm.ldy = a.ldy;
  prm.sG = a.sG;
  prm.gmul = a.gmul;
  prm.wpr = (int)(a.K / 8);
  prm.nsteps = (int)((a.N + kBN - 1) / kBN);
  prm.tiles_k = p.tiles_k;
  prm.splits = p.splits;
  prm.steps_per_split = p.steps_per_split;
  prm.units = p.tiles * p.splits;
  const hipError_t e = a.dtype == DT_F16 ? launch_g<DT_F16>(prm, lora, a.group, p.mw, s) : launch_g<DT_BF16>(prm, lora, a.group, p.mw, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_splitk_reduce(a.dtype, a.partial, nullptr, prm.dx, prm.M, prm.K, prm.K, p.splits, s);
}

}  // namespace w4a16
