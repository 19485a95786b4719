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
// direct global->LDS loads.  Both are double buffered, the words of the two
// steps after next in registers, and a step has one barrier.  Each weight is
// dequantised once per workgroup.
//
// Bound by instructions beside the matrix cores, one wave on each SIMD, as the
// forward GEMM: 1920 tokens, 4096 x 28672: 417-427 us, 1060-1080 TFLOP/s, the
// matrix cores busy 53-56 % of the time, and 14 us for the sum of its two ranges
// of n; 1921 tokens, 4096 x 6144, fp16: 109-116 us, 830-890 TFLOP/s; 128 tokens, 4096 x
// 4096: 19-20 us and 4.4, latency: eight ranges of eight steps.
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
  int tail_step;       // whose words come from the tail copy (-1: none),
  int64_t wq_to_tail;  // so many bytes from their place in wq
  const void* constants;
  uint16_t* dx;
  float* partial;
  int M, N, K, ldy, group;
  int wpr;      // words per weight row
  int nsteps, tiles_k, units, splits, steps_per_split;
};

// A wave-uniform global address in scalar registers: loads then take it with a
// 32-bit lane offset, without 64-bit vector address arithmetic.
typedef __attribute__((address_space(1))) const char g_char;
typedef __attribute__((address_space(1))) const uint32_t g_u32;
typedef __attribute__((address_space(1))) const u32x4 g_u32x4;
__device__ __forceinline__ g_char* uniform(uint64_t a) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return (g_char*)((uint64_t)lo | ((uint64_t)hi << 32));
}

// the words of one 8 x 8 block and its rows' constants: per pair of rows, what
// prep_kernel formed of their scales and zero points (dx_constants)
template <int DT>
struct Block {
  uint32_t w[8];
  u32x4 g[DT == DT_F16 ? 2 : 4];
};

template <int DT, int MW>
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
  const int unit = xcd_unit(blockIdx.x, p.units);  // the same tokens, neighbouring k on one XCD
  const int tile = unit / p.splits, split = unit - tile * p.splits;
  const int mt = tile / p.tiles_k, kt = tile - mt * p.tiles_k;
  const int m0 = mt * BM, k0 = kt * kBKX;
  const int s_begin = split * p.steps_per_split;
  const int s_end = min(p.nsteps, s_begin + p.steps_per_split);

  // ---- dy (rows of a multiple of 64 values, zero past N): load d of this wave
  // fills LDS rows (wave NDMA + d) 8 + lane / 8; position lane & 7 of a row
  // holds its piece pos ^ (row / 2 & 7)
  const uint64_t dytile = reinterpret_cast<uint64_t>(p.dy + (size_t)m0 * p.ldy);
  uint32_t dyoff[NDMA];  // (NDMA is even)
#pragma unroll
  for (int d = 0; d < NDMA; ++d) {
    const int row = min((wave * NDMA + d) * 8 + (lane >> 3), p.M - 1 - m0);
    dyoff[d] = (uint32_t)row * (uint32_t)p.ldy * 2u + 16u * (uint32_t)((lane & 7) ^ (4 * (d & 1) + (lane >> 4)));
  }
  auto stage_dy = [&](int s, lds_u8* buf) {
    g_char* base = uniform(dytile + (uint64_t)s * (kBN * 2));
#pragma unroll
    for (int d = 0; d < NDMA; ++d) {
      uint32_t at = dyoff[d];
      asm("" : "+v"(at));  // (as in load_block)
      __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const void*)(base + at), buf + (wave * NDMA + d) * 1024, 16, 0, 0);
    }
  };

  // ---- weights: this thread's block is rows 8 o.. of the step, slice c of the
  // tile; row i's word is woff + i wstride from the step's first (a complete
  // run keeps a tile's rows 16 bytes apart, an incomplete last one back to
  // back).  A last step that N ends inside comes from the tail copy, where it
  // is whole.
  const int c = tid & 31, o = tid >> 5;
  const int slice = min((k0 >> 3) + c, p.wpr - 1);
  const int runs = p.wpr >> 4, tail = p.wpr & 15;
  const bool full_run = (slice >> 4) < runs;
  const uint32_t wstride = full_run ? 16u : 4u * (uint32_t)tail;
  const uint32_t woff = 64u * (uint32_t)p.wpr * (uint32_t)(o >> 1) + 8u * (uint32_t)(o & 1) * wstride +
                        4u * (full_run ? 256u * (uint32_t)(slice >> 4) + 64u * (uint32_t)(slice & 3) + (uint32_t)((slice & 15) >> 2)
                                       : 256u * (uint32_t)runs + (uint32_t)(slice - 16 * runs));
  // constants: [group][rows of the padded N], 4 (fp16) or 8 bytes a row
  constexpr uint32_t kRowBytes = DT == DT_F16 ? 4 : 8;
  const uint32_t goff = kRowBytes * ((uint32_t)(8 * slice / p.group) * (uint32_t)p.ldy + 8u * (uint32_t)o);
  auto load_block = [&](int s, Block<DT>& b) {
    // (a mask rather than a choice of pointers, which became branches, and at a
    // branch the compiler waits for every load; N * K / 2 is below 4 GiB)
    const int64_t at_tail = -(int64_t)(s == p.tail_step);
    g_char* wb = uniform(reinterpret_cast<uint64_t>(p.wq) + (uint32_t)s * (uint32_t)(kBN * 4 * p.wpr) + (uint64_t)(at_tail & p.wq_to_tail));
    g_char* gb = uniform(reinterpret_cast<uint64_t>(p.constants) + (uint32_t)s * (kBN * kRowBytes));
    // the offsets are formed here, as 32-bit values that the compiler cannot
    // move out of the loop as 64-bit ones
    uint32_t at = woff, gat = goff;
    asm("" : "+v"(at), "+v"(gat));
#pragma unroll
    for (int i = 0; i < 8; ++i) b.w[i] = *(g_u32*)(wb + (at + i * wstride));
#pragma unroll
    for (int i = 0; i < (int)(kRowBytes / 2); ++i) b.g[i] = *(g_u32x4*)(gb + gat + 16 * i);
  };
  // Half of the block's operands: k = 0, 1, 4, 5 (part 0) or 2, 3, 6, 7 of the
  // slice -- the even or odd nibbles of the paired words -- each 16 bytes at
  // [octet o][slice c][k ^ (c / 2 & 7)]: sixteen lanes in a row,
  // writing (slices c) or reading (k of two slices), touch sixteen banks of 16
  // bytes.
  typedef __attribute__((address_space(3))) u32x4 lds_out;
  auto put_half = [&](const Block<DT>& b, lds_u8* buf, int part) {
    uint32_t out[4][4];  // [k of the part][row pair]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // rows 2q, 2q + 1 at the word's lower nibbles (even k) and upper ones (odd k)
      const uint32_t half[2] = {__builtin_amdgcn_perm(b.w[2 * q + 1], b.w[2 * q], 0x05040100u),
                                __builtin_amdgcn_perm(b.w[2 * q + 1], b.w[2 * q], 0x07060302u)};
      if constexpr (DT == DT_F16) {
        // both scales, then both -(1024 + z)
        const uint32_t sp = b.g[q >> 1][2 * (q & 1)], nmz = b.g[q >> 1][2 * (q & 1) + 1];
#pragma unroll
        for (int H = 0; H < 2; ++H)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t qz = add_f16x2(magic_pair<DT_F16>(half[H], part + 2 * e), nmz);
            out[2 * e + H][q] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, qz) * __builtin_bit_cast(half2_t, sp));
          }
      } else {
        // s 2^9 and -z s of either row
        const uint32_t kb[4] = {b.g[q][0], b.g[q][1], b.g[q][2], b.g[q][3]};
        float k[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = __builtin_bit_cast(float, kb[e]);
#pragma unroll
        for (int H = 0; H < 2; ++H) {
          // bytes: nibbles part and part + 2 of the first row, then of the second
          const uint32_t n = mask_nibbles(half[H] >> (4 * part));
          const f32x2 r0 = __builtin_amdgcn_cvt_pk_f32_fp8(n, false), r1 = __builtin_amdgcn_cvt_pk_f32_fp8(n, true);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            out[2 * e + H][q] = f32x2_to_act_pair<DT_BF16>(__builtin_fmaf(r0[e], k[0], k[1]), __builtin_fmaf(r1[e], k[2], k[3]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 4 * (i >> 1) + 2 * part + (i & 1);
      *(lds_out*)(buf + (uint32_t)(((o * 32 + c) * 8 + (k ^ ((c >> 1) & 7))) * 16)) = u32x4{out[i][0], out[i][1], out[i][2], out[i][3]};
    }
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
  u32x4 fa[2][4], fb[2][MW];  // operands of a k-sub (16 rows of W), by parity
  auto read = [&](const lds_u8* wbuf, const lds_u8* dbuf, int ks, u32x4 (&a)[4], u32x4 (&b)[MW]) {
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      const int cc = cl + 4 * kb;
      a[kb] = *(lds_u32x4*)(wbuf + (uint32_t)((((2 * ks + h) * 32 + cc) * 8 + ((j & 7) ^ ((cc >> 1) & 7))) * 16));
    }
#pragma unroll
    for (int mb = 0; mb < MW; ++mb)
      b[mb] = *(lds_u32x4*)(dbuf + (uint32_t)((wm * MW + mb) * 32 + j) * 128u + (uint32_t)(((2 * ks + h) ^ ((j >> 1) & 7)) * 16));
  };

  lds_u8* const w0 = (lds_u8*)ws0;
  lds_u8* const w1 = (lds_u8*)ws1;
  lds_u8* const d0 = (lds_u8*)ds0;
  lds_u8* const d1 = (lds_u8*)ds1;
  if (s_begin < s_end) {
    Block<DT> b0 = {}, b1 = {};
    const int last = s_end - 1;
    load_block(s_begin, b0);
    stage_dy(s_begin, d0);
    load_block(min(s_begin + 1, last), b1);
    stage_dy(min(s_begin + 1, last), d1);
    put_half(b0, w0, 0);
    put_half(b0, w0, 1);
    load_block(min(s_begin + 2, last), b0);
    wait_vm_all();
    __syncthreads();
    read(w0, d0, 0, fa[0], fb[0]);
    // Step s multiplies from (wc, dc), each k-sub's operands read one k-sub
    // ahead.  Meanwhile the block of step s + 1 is dequantised into wn, then the
    // words of step s + 3 are loaded in its place.  The barrier stands before
    // the last k-sub: by then every wave has written its part of wn, has its dy
    // of step s + 1 in dn and has read its last operands of (wc, dc), so dc takes
    // the dy of step s + 2.  It waits for everything but the kKeep words and
    // constants just loaded (the vector memory instructions since the last
    // dy load; the build checks that), which have the whole of step s + 1.
    constexpr int kKeep = 8 + (int)(kRowBytes / 2);
    auto step = [&](int s, lds_u8* wc, lds_u8* dc, lds_u8* wn, lds_u8* dn, Block<DT>& next, auto keep) {
static_for<0, 4>([&](auto kc) {
        constexpr int ks = decltype(kc)::value, cur = ks & 1, nx = cur ^ 1;
        constexpr int NM = 4 * MW;  // MFMAs
        if constexpr (ks < 3) {
          read(wc, dc, ks + 1, fa[nx], fb[nx]);
          if constexpr (ks < 2) put_half(next, wn, ks);
          if constexpr (ks == 2) load_block(min(s + 3, last), next);
        } else {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (decltype(keep)::value)
            __builtin_amdgcn_s_waitcnt((kKeep & 15) | ((kKeep >> 4) << 14) | (7 << 4));  // vmcnt(kKeep), lgkmcnt(0)
          else
            __builtin_amdgcn_s_waitcnt(0);
          asm volatile("s_barrier" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          read(wn, dn, 0, fa[nx], fb[nx]);
          stage_dy(min(s + 2, last), dc);
        }
#pragma unroll
        for (int mb = 0; mb < MW; ++mb)
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) acc[mb][kb] = mfma32x32x16<DT>(fa[cur][kb], fb[cur][mb], acc[mb][kb]);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // one MFMA
          if (i < 4 + MW) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
          __builtin_amdgcn_sched_group_barrier(0x002, ((ks < 2 ? 112 : 32) + NM - 1) / NM, 0);  // VALU
          if constexpr (ks >= 2) __builtin_amdgcn_sched_group_barrier(0x020, (18 + NM - 1) / NM, 0);  // global loads
          if constexpr (ks == 1 || ks == 2) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS writes
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    int s = s_begin;
    for (; s + 1 < s_end; s += 2) {
      step(s, w0, d0, w1, d1, b1, std::true_type{});
      step(s + 1, w1, d1, w0, d0, b0, std::true_type{});
    }
    // (what a peeled step loads is never used and may be dropped: no count)
    if (s < s_end) step(s, w0, d0, w1, d1, b1, std::false_type{});
    wait_vm_all();  // no load into LDS in flight past the loop
  }
  {
    // rows of 256 tokens take all four buffers, 128 to an array (the halves of
    // the tile that the waves own); shorter tiles one array each
    static_assert(128 * 256 <= kWBytes && (BM != 256 || 128 * 256 <= BM * 128), "rows of the tile's tokens");
    constexpr bool four = BM == 256;
    lora_stage(lora, p.M, m0, BM, tid, kThreads,
               [&](int m) { return four && m >= 128 ? w1 + 256 * (m - 128) : w0 + 256 * m; },
               [&](int m) { return !four ? w1 + 256 * m : m >= 128 ? d1 + 256 * (m - 128) : d0 + 256 * m; });
    const int first = 32 * MW * wm;
    const lds_u8* hi = four ? (wm ? w1 : w0) : w0 + 256 * first;
    const lds_u8* lo = four ? (wm ? d1 : d0) : w1 + 256 * first;
    lora_steps<DT, MW, 4>(lora, p.M, p.K, m0 + first, k0 + 128 * wk, lane, split, p.splits, hi, lo, acc);
  }

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

template <int DT>
hipError_t launch_mw(const DxParams& prm, const LoraTerm& lora, int mw, hipStream_t s) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(prm.units), dim3(kThreads), 0, s, prm, lora);
    return hipGetLastError();
  };
  switch (mw) {
    case 1: return go(dx_kernel<DT, 1>);
    case 2: return go(dx_kernel<DT, 2>);
    case 4: return go(dx_kernel<DT, 4>);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Tile height and split of n: time model in microseconds, fitted to every
// (height, split) timed on 14 shapes (M 32-2048, N and K 1216-28672, groups of
// 32, all in bf16; mean error 5.9 %, its picks 2.3 % from the best on average,
// 13 % at worst; fp16, whose dequantisation takes other instructions, uses the
// same model unswept: 1921 x 4096 x 6144 takes 125 us where it gives 108): a
// fixed part and a time per step and round of resident workgroups
// (64-token tiles: 1.08 us alone on a CU, 1.56 us for two that share one),
// and for a split its second launch and the partial sums' way through memory.
DxPlan plan_dx(int64_t M, int64_t N, int64_t K, int cu_count) {
  DxPlan best{};
  double best_t = 0.0;
  const int nsteps = (int)((N + kBN - 1) / kBN);
  const int64_t tiles_k = (K + kBKX - 1) / kBKX;
  for (int mw : {4, 2, 1}) {
    const int64_t tiles = (M + 64 * mw - 1) / (64 * mw) * tiles_k;
    for (int splits = 1; splits <= 32 && splits <= nsteps; ++splits) {
      const int sps = (nsteps + splits - 1) / splits;
      if ((nsteps + sps - 1) / sps != splits) continue;
      const int64_t units = tiles * splits;
      const bool pairs = mw == 1 && units > cu_count;
      const int64_t rounds = (units + cu_count * (pairs ? 2 : 1) - 1) / (cu_count * (pairs ? 2 : 1));
      const double step = mw == 4 ? 1.6 : mw == 2 ? 1.19 : pairs ? 1.56 : 1.08;
      const double fixed = mw == 4 ? 2.3 : mw == 2 ? 1.5 : 0.0;
      const double t = rounds * (fixed + sps * step) + (splits > 1 ? 4.2 + 0.387e-6 * splits * (double)M * (double)K * 4.0 : 0.0);
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
  prm.constants = a.constants;
  prm.dx = static_cast<uint16_t*>(a.dx);
  prm.partial = a.partial;
  prm.M = (int)a.M;
  prm.N = (int)a.N;
  prm.K = (int)a.K;
  prm.ldy = a.ldy;
  prm.group = a.group;
  prm.wpr = (int)(a.K / 8);
  prm.tail_step = -1;
  prm.wq_to_tail = 0;
  if (a.N % kBN) {
    const int64_t t = a.N / kBN;
    prm.tail_step = (int)t;
    prm.wq_to_tail = (int64_t)(reinterpret_cast<uintptr_t>(a.wq_tail) - reinterpret_cast<uintptr_t>(a.wq)) - t * kBN * 4 * (a.K / 8);
  }
  prm.nsteps = (int)((a.N + kBN - 1) / kBN);
  prm.tiles_k = p.tiles_k;
  prm.splits = p.splits;
  prm.steps_per_split = p.steps_per_split;
  prm.units = p.tiles * p.splits;
  const hipError_t e = a.dtype == DT_F16 ? launch_mw<DT_F16>(prm, lora, p.mw, s) : launch_mw<DT_BF16>(prm, lora, p.mw, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_splitk_reduce(a.dtype, a.partial, nullptr, prm.dx, prm.M, prm.K, prm.K, p.splits, s);
}

}  // namespace w4a16
