// Prefill W4A16 GEMM for gfx950: y = x . dequant(Wq)^T (+ bias) with fp16 /
// bf16 MFMA and fp32 accumulation.
//
// The pages route M above the decode threshold to a fused dequantise-then-
// GEMM kernel ("[ROCm][Kernel] Add HybridW4A16LinearKernel: Triton prefill +
// HIP skinny decode", description).  Here it is hand-written for CDNA4:
//
// * A workgroup (4 waves) owns BM = 32*MB tokens by 256 output features; each
//   wave owns 64 features (two 32-wide blocks) across all BM tokens, so every
//   weight is dequantised exactly once per workgroup, by the wave that
//   multiplies it.
// * A k-step is one stored 128-k run of each weight row.  The weights are the
//   MFMA A operand (v_mfma_f32_32x32x16): lane (j, h) needs 8 consecutive k of
//   row j, i.e. one packed word, and the run's 4x4 word transpose puts the
//   eight words a lane needs for the whole k-step into two 16-byte loads.
//   They are dequantised in registers (the exact per-weight value that
//   w4a16_dequant returns) and fed straight to the MFMA: no LDS round trip.
// * The activations x are the B operand.  They are staged in LDS by direct
//   global->LDS loads (global_load_lds_dwordx4), double buffered, with the
//   16-byte pieces of each 256-byte row XOR-swizzled by (row mod 16) so the
//   fragment reads of 16 consecutive lanes hit 16 different bank groups.
// * The output tile of a wave is 64 features x BM tokens; in the MFMA result
//   layout a lane holds 4 consecutive features of one token, and one
//   permlane32 swap turns two such quads into 16 contiguous output bytes.
// * Work units (tile, K split) are remapped so that consecutive units -- the
//   same token rows, neighbouring features -- run on the same XCD and share
//   its L2.  With more than one split, units store fp32 partial tiles and the
//   last one to finish a tile adds them up in split order (deterministic).
// * DENSE instances multiply already dequantised act-dtype weights w[N, K]
//   (the dequantised prefill copy): the same tiles, staging, pipeline and
//   epilogue, with each lane's A fragments loaded straight from w's rows
//   (eight 16-byte loads per column block and k-step) instead of unpacked
//   from codes.
#include <algorithm>

#include "w4a16_gemm_tile.hpp"
#include "w4a16_lora_bwd.hpp"


namespace w4a16 {

namespace {

template <int DT, int GS, bool ASYM, int MB, int CB, bool DENSE>
__global__ __launch_bounds__(kThreads) void gemm_kernel(const GemmParams p) {
  gemm_tile<DT, GS, ASYM, MB, CB, DENSE, false>(p, LoraTerm{});
}

// The K split's second pass: y = sum of the splits' fp32 partials, in split
// order, + bias in fp32, one rounding.  One thread per row and 4 consecutive
// features.
template <int DT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ partial,
                                                            const uint16_t* __restrict__ bias,
                                                            uint16_t* __restrict__ y, int M, int N,
                                                            int np, int splits) {
  const int qpr = np >> 2;
  const int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (q >= (int64_t)M * qpr) return;
  const int m = (int)(q / qpr), n = (int)(q % qpr) * 4;
  const size_t plane = (size_t)M * np;
  const float* src = partial + (size_t)m * np + n;
  f32x4 s = *reinterpret_cast<const f32x4*>(src);
  for (int sp = 1; sp < splits; ++sp) s += *reinterpret_cast<const f32x4*>(src + sp * plane);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < N) {
      float v = s[e];
      if (bias) v += act_to_f32<DT>(bias[n + e]);
      y[(size_t)m * N + n + e] = f32_to_act<DT>(v);
    }
}

template <int DT, int GS, bool ASYM, int MB, int CB, bool DENSE>
hipError_t launch_t(const GemmParams& prm, hipStream_t s) {
  hipLaunchKernelGGL((gemm_kernel<DT, GS, ASYM, MB, CB, DENSE>), dim3(prm.units), dim3(kThreads), 0, s, prm);
  return hipGetLastError();
}

// tile shapes: 32 mb tokens x 128 cb features; cb = 1 only for mb 1, 4 and 8
template <int DT, int GS, bool ASYM, bool DENSE = false>
hipError_t launch_mb(const GemmParams& prm, int mb, int cb, hipStream_t s) {
  if (cb == 1) {
    switch (mb) {
      case 1: return launch_t<DT, GS, ASYM, 1, 1, DENSE>(prm, s);
      case 4: return launch_t<DT, GS, ASYM, 4, 1, DENSE>(prm, s);
      case 8: return launch_t<DT, GS, ASYM, 8, 1, DENSE>(prm, s);
      default: return hipErrorInvalidValue;
    }
  }
  switch (mb) {
    case 1: return launch_t<DT, GS, ASYM, 1, 2, DENSE>(prm, s);
    case 4: return launch_t<DT, GS, ASYM, 4, 2, DENSE>(prm, s);
    case 6: return launch_t<DT, GS, ASYM, 6, 2, DENSE>(prm, s);
    case 8: return launch_t<DT, GS, ASYM, 8, 2, DENSE>(prm, s);
    default: return hipErrorInvalidValue;
  }
}

template <int DT, int GS>
hipError_t launch_z(const GemmParams& prm, int mb, int cb, hipStream_t s) {
  return prm.zp ? launch_mb<DT, GS, true>(prm, mb, cb, s) : launch_mb<DT, GS, false>(prm, mb, cb, s);
}

template <int DT>
hipError_t launch_g(const GemmParams& prm, int group, int mb, int cb, hipStream_t s) {
  switch (group) {
    case 32: return launch_z<DT, 32>(prm, mb, cb, s);
    case 64: return launch_z<DT, 64>(prm, mb, cb, s);
    case 128: return launch_z<DT, 128>(prm, mb, cb, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Tile shape and K split.  Cost model in cycles of one CU, fitted to
// measured k-step times (about 380 cycles per 32 tokens and 128 features of
// the tile plus a fixed 1000: MFMA issue, dequantisation and staging share
// one instruction stream per SIMD); units run in rounds of cu_count; splitting
// K adds the partial-tile hand-off.  Narrow tiles (128 features, one column
// block per wave) double the tile count at small M, where 256-feature tiles
// leave CUs idle or need K splits whose partial sums outweigh the weights.
// Tile heights 192 and 256 with 256-feature tiles, for the dtype / group /
// zero-point combinations whose kernel instances spill registers to scratch
// memory with this compiler (fp16 with groups of 32, or of 64 with zero
// points; bf16 with groups of 32 without): a k-step of four or two groups
// keeps its group constants and the next step's metadata beside 192-256
// accumulators.  Measured at M = 1920 on 6144x4096 they run 1.2-3.6x slower
// than the 128-token tile, so the planner leaves them out.
// Dense instances (no group constants) at tile heights 192 and 256 with
// 256-feature tiles: their eight 16-byte weight pieces per column block and
// k-step stand where the codes and metadata stood.
bool dense_tall_tile_spills(int dtype) {
  (void)dtype;
  return false;
}

bool wide_tall_tile_spills(int group, int dtype, bool asym) {
  if (dtype == DT_F16) return group == 32 || (group == 64 && asym);
  return group == 32 && !asym;
}

// Up to 64 tokens: 32-token tiles of 128 features (the weights of a tile
// are dequantised once for at most 32 tokens, so at small M the matrix cores
// no longer multiply up to 96 padding rows of a 128-token tile).  A thin
// tile's k-step is shorter than a memory round trip, so it prefetches two
// k-steps (the kernel's MB == 1 loop) and K is split until enough units are
// resident; time model in microseconds, fitted to every K split (1-16, both
// hand-off forms) at M = 16 and 48 on ten Llama- and Qwen-shaped layers
// (K 2560-28672; mean error 6 %, its picks 3.6 % from the best on average,
// 18 % at worst): 0.528 * k-steps per unit * max(1, units / 224) +
// 0.528 per extra K range + partial-sum traffic (0.108 us per MB two-pass,
// 0.314 one-pass) + 4.91 (- 0.06 two-pass).
// Against the 128-token tiles' plans: M = 9-32 -15 to -33 % on eight layers
// (Llama and Qwen shapes, fp16 and bf16, groups 32 and 128); M = 48 / 64
// lower where K <= 16384; 28672 x 4096 keeps the 128-token tiles above
// M = 32 (a tie at M = 48).
// the second kernel of a tail launch: its start after the first one drains
constexpr double kTailLaunchCycles = 4000.0;

static GemmPlan plan_gemm_thin(int64_t M, int64_t N, int64_t K) {
  GemmPlan best{};
  double best_t = 0.0;
  const int nsteps = (int)((K + kBK - 1) / kBK);
  const int64_t tiles_n = (N + 127) / 128;
  const int64_t tiles = ((M + 31) / 32) * tiles_n;
  for (int splits = 1; splits <= 16 && splits <= nsteps; ++splits) {
    const int sps = (nsteps + splits - 1) / splits;
    if ((nsteps + sps - 1) / sps != splits) continue;
    const int64_t units = tiles * splits;
    const double resident = units > 224 ? (double)units / 224.0 : 1.0;
    const double part_mb = splits > 1 ? (double)splits * (double)M * (double)N * 4.0 / 1e6 : 0.0;
    for (int tp = 0; tp < (splits > 1 ? 2 : 1); ++tp) {
      if (tp == 0 && splits > 1 && tiles > kMaxCounters) continue;
      const double t = 0.528 * sps * resident + 0.528 * (splits - 1) + (tp ? 0.108 : 0.314) * part_mb + 4.91 -
                       0.06 * tp;
      if (best.units == 0 || t < best_t) {
        best_t = t;
        best.mb = 1;
        best.cb = 1;
        best.splits = splits;
        best.steps_per_split = sps;
        best.tiles_n = (int)tiles_n;
        best.tiles = (int)tiles;
        best.units = (int)units;
        best.two_pass = tp == 1;
      }
    }
  }
  return best;
}

GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int group, int dtype, bool asym, int cu_count,
                   bool dense) {
  GemmPlan best{};
  const bool tall_wide_ok = dense ? !dense_tall_tile_spills(dtype) : !wide_tall_tile_spills(group, dtype, asym);
  // where the tall wide tiles are left out, narrow tiles are tried first, so
  // that near-ties go to them: at M = 1920 on 6144x4096 they beat the
  // 128-token wide tile by 1-20 % for those combinations
  const int cb_order[2] = {tall_wide_ok ? 2 : 1, tall_wide_ok ? 1 : 2};
  double best_cost = 0.0;
  // (the dense instances too: the same tiles and splits)
  const bool thin = M <= 32 || (M <= 64 && K <= 16384);
  if (thin) best = plan_gemm_thin(M, N, K);
  const int nsteps = (int)((K + kBK - 1) / kBK);
  const int cus = cu_count > 0 ? cu_count : 256;
  for (int cb : cb_order) {
    if (thin) break;
    const int64_t bn = 128 * cb;
    const int64_t tiles_n = (N + bn - 1) / bn;
    for (int mb : {8, 6, 4}) {
      if (cb == 1 && mb == 6) continue;
      if (cb == 2 && mb > 4 && !tall_wide_ok) continue;
      const int64_t bm = 32 * mb;
      const int64_t tiles = ((M + bm - 1) / bm) * tiles_n;
      for (int splits = 1; splits <= 16 && splits <= nsteps; ++splits) {
        const int sps = (nsteps + splits - 1) / splits;
        const int real_splits = (nsteps + sps - 1) / sps;
        if (real_splits != splits) continue;

        const int64_t units = tiles * splits;
        const int64_t rounds = (units + cus - 1) / cus;
        // a split unit writes its fp32 partial tile; the tile's last unit then
        // reads the others back, one memory round trip (~2500 cycles) per
        // split and 64-value chunk, plus the bytes (mostly from L2 / MALL)
        const double fixup = splits > 1 ? 2.0 * bm * bn * 4 / 40.0 +
                                             2500.0 * splits * (16.0 * cb * mb / 64.0) : 0.0;
        const double loop = sps * (380.0 * cb * mb + 1000.0);
        const double cost = (double)rounds * (loop + fixup);
        // two passes: each unit stores its partial tile (~64 bytes a cycle),
        // then a second kernel reads all partials plus its launch; the
        // partials' round trip is taken as 3 TB/s at 2.1 GHz (fitted to every
        // plan timed at M = 128-512 on 4096x6144, 4096x28672 and 14336x4096)
        const double np = (double)((N + 7) / 8 * 8);
        const double cost2 = (double)rounds * (loop + bm * bn * 4 / 64.0) +
                             (splits * (double)M * np * 4.0 + (double)M * N * 2.0) * (2.1e9 / 3e12) + 3000.0;
        for (int tp = 0; tp < (splits > 1 && mb == 4 ? 2 : 1); ++tp) {
          const double c = tp ? cost2 : cost;
          if (tp == 0 && splits > 1 && tiles > kMaxCounters) continue;
          if (best.units == 0 || c < best_cost * 0.98) {
            best_cost = c;
            best = GemmPlan{};
            best.mb = mb;
            best.cb = cb;
            best.splits = splits;
            best.steps_per_split = sps;
            best.tiles_n = (int)tiles_n;
            best.tiles = (int)tiles;
            best.units = (int)units;
            best.two_pass = tp == 1;
          }
        }
        // Tail launch: where the unsplit 256-token tiles end in a partial
        // round, the tiles past the last full round run as a second launch of
        // 128-token tiles, in one round; halves wholly past M cost nothing
        // (4096 x 28672 at M = 1920: 896 tiles of 256 x 256 are 3.5 rounds, the
        // last half of the CUs idle; as 3 rounds plus 144 tiles of 128 x 256
        // it measured -5.6 %).  A tail k-step takes at least 0.8 of the plan
        // tile's (its loads' round trip, not its MFMAs, sets the pace: measured
        // 0.77-0.82 for 128 x 256 tails, 0.89 for 128 x 128 tails of 256 x 256
        // tiles, which the planner therefore never picks).
        if (mb == 8 && splits == 1 && units > cus && units % cus != 0) {
          const int64_t full = units / cus * cus;
          int64_t busy = 0;  // halves with output to compute
          for (int64_t w = full; w < tiles; ++w) busy += (w / tiles_n) * bm + bm / 2 < M ? 2 : 1;
          const double tstep = std::max(380.0 * cb * 4 + 1000.0, 0.8 * (380.0 * cb * mb + 1000.0));
          const double tc = (double)(full / cus) * loop + (double)((busy + cus - 1) / cus) * nsteps * tstep +
                            kTailLaunchCycles;
          if (tc < best_cost * 0.98) {
            best_cost = tc;
            best = GemmPlan{};
            best.mb = mb;
            best.cb = cb;
            best.splits = 1;
            best.steps_per_split = sps;
            best.tiles_n = (int)tiles_n;
            best.tiles = (int)tiles;
            best.units = (int)full;
            best.tail_mb = 4;
            best.tail_tile0 = (int)full;
            best.tail_units = (int)(2 * (tiles - full));
          }
        }
      }
    }
  }
  // tuning override "mb,splits[,two_pass[,cb]]" (tile 32*mb x 128*cb, K ranges), e.g. for sweeps
  const Tuning& tu = tuning();
  if (tu.gemm_tile_n >= 2) {
    const int mb = tu.gemm_tile[0], splits = tu.gemm_tile[1];
    const int tp = tu.gemm_tile_n >= 3 ? tu.gemm_tile[2] : 0;
    const int cb = tu.gemm_tile_n >= 4 ? tu.gemm_tile[3] : 2;
    if ((mb == 1 || mb == 4 || mb == 6 || mb == 8) &&
        (cb == 2 || (cb == 1 && mb != 6)) && splits >= 1 && splits <= nsteps && (tp == 0 || mb == 1 || mb == 4)) {
      const int sps = (nsteps + splits - 1) / splits;
      const int64_t tiles_n = (N + 128 * cb - 1) / (128 * cb);
      const int64_t tiles = ((M + 32 * mb - 1) / (32 * mb)) * tiles_n;
      if (splits == 1 || tp == 1 || tiles <= kMaxCounters) {
        best = GemmPlan{};
        best.two_pass = splits > 1 && tp == 1;
        best.mb = mb;
        best.cb = cb;
        best.steps_per_split = sps;
        best.splits = (nsteps + sps - 1) / sps;
        best.tiles_n = (int)tiles_n;
        best.tiles = (int)tiles;
        best.units = (int)(tiles * best.splits);
      }
    }
  }
  return best;
}

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int group, int dtype, bool asym,
                            int cu_count, bool dense) {
  const GemmPlan p = plan_gemm(M, N, K, group, dtype, asym, cu_count, dense);
  if (p.splits <= 1) return 0;
  if (p.two_pass)
    return kCounterBytes + (size_t)p.splits * (size_t)M * (size_t)((N + 7) / 8 * 8) * sizeof(float);
  return kCounterBytes + (size_t)p.units * (size_t)(32 * p.mb) * (size_t)(128 * p.cb) * sizeof(float);
}

hipError_t launch_gemm(const LinearArgs& a, void* workspace, int cu_count, hipStream_t stream,
                       const LoraTerm* lora) {
  const GemmPlan plan = plan_gemm(a.M, a.N, a.K, a.group, a.dtype, a.zp != nullptr, cu_count, a.dense);
  GemmParams prm;
  prm.x = static_cast<const uint16_t*>(a.x);
  prm.wq = reinterpret_cast<const uint32_t*>(a.wq);
  prm.scales = static_cast<const uint16_t*>(a.scales);
  prm.zp = reinterpret_cast<const uint32_t*>(a.zp);
  prm.bias = static_cast<const uint16_t*>(a.bias);
  prm.y = static_cast<uint16_t*>(a.y);
  prm.counters = nullptr;
  prm.partial = nullptr;
  if (plan.splits > 1) {
    if (workspace == nullptr) return hipErrorInvalidValue;
    prm.counters = static_cast<uint32_t*>(workspace);
    prm.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  }
  prm.M = (int)a.M;
  prm.N = (int)a.N;
  prm.K = (int)a.K;
  prm.G = (int)(a.K / a.group);
  prm.sG = a.sG;
  prm.gmul = a.gmul;
  prm.wpr = (int)(a.K / 8);
  prm.nsteps = (int)((a.K + kBK - 1) / kBK);
  prm.full_steps = (int)(a.K / kBK);
  prm.tiles_n = plan.tiles_n;
  prm.units = plan.units;
  prm.tile0 = 0;
  prm.sub_m = 0;
  prm.splits = plan.splits;
  prm.steps_per_split = plan.steps_per_split;
  prm.vec_store = (a.N % 8 == 0) && (reinterpret_cast<uintptr_t>(a.y) % 16 == 0);
  prm.two_pass = plan.splits > 1 && plan.two_pass;
  if (prm.two_pass && plan.mb != 1 && plan.mb != 4) return hipErrorInvalidConfiguration;
  if (plan.tail_units > 0 && (2 * plan.tail_mb != plan.mb || plan.splits != 1)) return hipErrorInvalidConfiguration;
  prm.np = (int)((a.N + 7) / 8 * 8);
  auto tiles = [&](const GemmParams& q, int mb) {
    if (lora) return launch_gemm_lora_tiles(q, *lora, a.dtype, a.group, mb, plan.cb, stream);
    if (a.dense)
      return a.dtype == DT_F16 ? launch_mb<DT_F16, 128, false, true>(q, mb, plan.cb, stream)
                               : launch_mb<DT_BF16, 128, false, true>(q, mb, plan.cb, stream);
    return a.dtype == DT_F16 ? launch_g<DT_F16>(q, a.group, mb, plan.cb, stream)
                             : launch_g<DT_BF16>(q, a.group, mb, plan.cb, stream);
  };
  hipError_t e = tiles(prm, plan.mb);
  if (e == hipSuccess && plan.tail_units > 0) {
    GemmParams t = prm;
    t.units = plan.tail_units;
    t.tile0 = plan.tail_tile0;
    t.sub_m = 1;
    e = tiles(t, plan.tail_mb);
  }
  if (e != hipSuccess || !prm.two_pass) return e;
  return launch_splitk_reduce(a.dtype, prm.partial, prm.bias, prm.y, prm.M, prm.N, prm.np, prm.splits, stream);
}

hipError_t launch_splitk_reduce(int dtype, const float* partial, const uint16_t* bias, uint16_t* y, int M, int N, int np,
                                int splits, hipStream_t s) {
  const int64_t quads = (int64_t)M * (np / 4);
  const int blocks = (int)((quads + 255) / 256);
  if (dtype == DT_F16)
    hipLaunchKernelGGL(splitk_reduce_kernel<DT_F16>, dim3(blocks), dim3(256), 0, s, partial, bias, y, M, N, np, splits);
  else
    hipLaunchKernelGGL(splitk_reduce_kernel<DT_BF16>, dim3(blocks), dim3(256), 0, s, partial, bias, y, M, N, np, splits);
  return hipGetLastError();
}

}  // namespace w4a16
