// Host side of libw4a16: the C ABI declared in include/w4a16.h -- argument
// validation, packing, a per-device property cache, path selection, and the
// launch of the kernels on the caller's stream.
//
// Validation follows the accept set the pages describe for the kernel's
// `can_implement` (quantisation type, activation dtype, group size and K
// divisibility; "Upstream sync 67/N: merge 382bbd5144 HybridW4A16LinearKernel
// (conflict)", reviewer's item 2), and the zero-point contract of the same
// page's section "Upstream's Python side is kept -- and it does NOT work here".
#include "w4a16.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <cstring>
#include <exception>
#include <mutex>
#include <string>
#include <vector>

#include "w4a16_adamw.h"
#include "w4a16_internal.h"
#include "w4a16_lora_bwd.hpp"

namespace w4a16 {

namespace {

Tuning read_tuning() {
  Tuning t{};
  t.m_threshold = -1;
  if (const char* e = std::getenv("W4A16_FORCE_PATH")) {
    if (std::strcmp(e, "gemv") == 0) t.force_path = W4A16_PATH_GEMV;
    if (std::strcmp(e, "gemm") == 0) t.force_path = W4A16_PATH_GEMM;
  }
  if (const char* e = std::getenv("W4A16_M_THRESHOLD")) {
    char* end = nullptr;
    const long v = std::strtol(e, &end, 10);
    if (end != e && v >= 0 && v <= W4A16_GEMV_MAX_M) t.m_threshold = (int)v;
  }
  if (const char* e = std::getenv("W4A16_GEMM_TILE")) {
    const int n = std::sscanf(e, "%d,%d,%d,%d", &t.gemm_tile[0], &t.gemm_tile[1], &t.gemm_tile[2],
                              &t.gemm_tile[3]);
    t.gemm_tile_n = n > 0 ? n : 0;
  }
  if (const char* e = std::getenv("W4A16_GEMV_KPW")) t.gemv_kpw = std::atoi(e);
  if (const char* e = std::getenv("W4A16_GEMV_SPLITS")) t.gemv_splits = std::atoi(e);
  t.gemv_no_wgsz = std::getenv("W4A16_GEMV_NO_WGSZ") != nullptr;
  t.gemv_no_one = std::getenv("W4A16_GEMV_NO_ONE") != nullptr;
  if (const char* e = std::getenv("W4A16_LOG")) t.log = *e && std::strcmp(e, "0") != 0;
  return t;
}

// The current settings.  A reload publishes a new copy and keeps the old one
// (a few dozen bytes per reload), so a reader that still holds it stays valid.
std::atomic<const Tuning*> g_tuning{nullptr};
std::mutex g_tuning_mutex;

}  // namespace

const Tuning& tuning() {
  const Tuning* t = g_tuning.load(std::memory_order_acquire);
  if (t) return *t;
  std::lock_guard<std::mutex> lock(g_tuning_mutex);
  t = g_tuning.load(std::memory_order_acquire);
  if (!t) {
    t = new Tuning(read_tuning());
    g_tuning.store(t, std::memory_order_release);
  }
  return *t;
}

void reload_tuning() {
  std::lock_guard<std::mutex> lock(g_tuning_mutex);
  g_tuning.store(new Tuning(read_tuning()), std::memory_order_release);
}

}  // namespace w4a16

namespace {

thread_local std::string g_last_error;

w4a16_status fail(w4a16_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

w4a16_status ok() {
  g_last_error.clear();
  return W4A16_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a + na) and [b, b + nb) overlap
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

// ---- per-device properties, filled once per device ------------------------
struct DeviceInfo {
  bool ready = false;
  hipError_t err = hipSuccess;
  bool gfx950 = false;
  int cu_count = 0;
  char arch[64] = {0};
  // this device's copy of `scratch` (w4a16_linear_noalloc), set up on the
  // entry point's first call on the device
  bool scratch_ready = false;
  void* scratch_ptr = nullptr;
};

constexpr int kMaxDevices = 64;
DeviceInfo g_devices[kMaxDevices];
std::mutex g_device_mutex;

w4a16_status device_info(const DeviceInfo** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(W4A16_ERR_DEVICE, "hipGetDevice failed: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(W4A16_ERR_DEVICE, "device ordinal %d out of range", dev);
  DeviceInfo& d = g_devices[dev];
  {
    std::lock_guard<std::mutex> lock(g_device_mutex);
    if (!d.ready) {
      hipDeviceProp_t prop;
      d.err = hipGetDeviceProperties(&prop, dev);
      if (d.err == hipSuccess) {
        std::snprintf(d.arch, sizeof(d.arch), "%s", prop.gcnArchName);
        d.cu_count = prop.multiProcessorCount;
        d.gfx950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 &&
                   (prop.gcnArchName[6] == '\0' || prop.gcnArchName[6] == ':');
      }
      d.ready = true;
    }
  }
  if (d.err != hipSuccess)
    return fail(W4A16_ERR_DEVICE, "hipGetDeviceProperties failed: %s", hipGetErrorString(d.err));
  if (!d.gfx950)
    return fail(W4A16_ERR_UNSUPPORTED, "libw4a16 supports gfx950 only; this device is %s", d.arch);
  *out = &d;
  return W4A16_OK;
}

// ---- scratch of the allocation-free entry point ----------------------------
// w4a16_linear_noalloc takes its split-K workspace (completion counters, then
// fp32 partial sums) from this array instead of from the caller.  Every GPU
// the library runs on holds its own copy, from module load until the process
// ends.  In host code `scratch` names a host-side stand-in, not the device
// copy: the address a kernel needs comes from hipGetSymbolAddress, taken once
// per device with that device current (DeviceInfo::scratch_ptr).
constexpr size_t kScratchBytes = W4A16_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

std::mutex g_scratch_mutex;

// This device's scratch address; on the first call on the device the
// counter region is cleared by a kernel on `stream` (stream-ordered before
// the launch that follows).
w4a16_status scratch_for(DeviceInfo& d, int dev, hipStream_t stream, void** out) {
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (!d.scratch_ready) {
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != dev)
      return fail(W4A16_ERR_DEVICE, "noalloc: device %d is not current", dev);
    void* ptr = nullptr;
    const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess || ptr == nullptr)
      return fail(W4A16_ERR_DEVICE, "noalloc: hipGetSymbolAddress(scratch) failed: %s", hipGetErrorString(e));
    const hipError_t z = w4a16::launch_zero_words(ptr, w4a16::kCounterBytes, stream);
    if (z != hipSuccess)
      return fail(W4A16_ERR_LAUNCH, "noalloc: clearing the scratch counters failed: %s", hipGetErrorString(z));
    d.scratch_ptr = ptr;
    d.scratch_ready = true;
  }
  *out = d.scratch_ptr;
  return W4A16_OK;
}

size_t act_bytes(int64_t n) { return (size_t)n * 2; }

bool valid_group(int32_t g) { return g == 32 || g == 64 || g == 128; }

// Group sizes: the pages' accept set {32, 64, 128}, and per-channel scales
// (group_size == K, one scale and zero point per row) for K a multiple of 32.
bool group_ok(int32_t g, int64_t K) { return valid_group(g) || (g == K && K % 32 == 0); }

// The kernels' group for a group size: itself, or for per-channel scales the
// largest of 128, 64, 32 dividing K, every group of a row then reading the
// row's one scale (gmul = 0, row stride sG = 1).
struct GroupMap {
  int kgroup, sG, gmul;
};
GroupMap group_map(int32_t g, int64_t K) {
  if (valid_group(g)) return {g, (int)(K / g), 1};
  const int kg = K % 128 == 0 ? 128 : (K % 64 == 0 ? 64 : 32);
  return {kg, 1, 0};
}

// Decode-kernel threshold.  The pages route M <= 5 to their skinny kernel
// (tuned on RDNA).  Measured on MI355X (both kernels timed per launch over
// graphs rotating >= 1 GiB of weights; groups 32/64/128, symmetric and
// asymmetric, fp16 and bf16): the decode kernel is faster at every M <= 8
// (at K = 28672 within 1-3 % of the GEMM at M = 8).  Above that it takes one
// k-step per wave and the GEMM (32-token tiles up to M = 32) overtakes it by
// layer size:
//   K = 28672, and K = 14336 / 9728 from 32 M weights (14336 x 4096): the
//                           GEMM from M = 9 (-11 % there at M = 9-12);
//   K = 9728 x 2560:        decode through M = 12, the GEMM from 14;
//   K <= 4096, N >= 14336:  the GEMM from M = 9 at every group;
//   K <= 4096, 4096 x 6144: decode at M = 9, the GEMM 13-16 % faster at
//                           M = 10-14, a tie at 16;
//   K <= 4096, smaller (4096 x 4096, 4096 x 2560, 2560 x 6144): decode
//                           through M = 16.
int64_t gemv_threshold(int64_t N, int64_t K, int32_t group, int32_t dtype, int32_t has_zp) {
  (void)dtype; (void)has_zp;
  const int v = w4a16::tuning().m_threshold;
  if (v >= 0 && v <= W4A16_GEMV_MAX_M) return v;
  const int64_t weights = N * K;
  // K > 16384: from 160 Mi weights on, with groups of 64 or more, the GEMM's
  // 32-token tiles win from M = 7 (28672 x 8192: -7 to -26 % at M = 7 / 8)
  if (K > 16384) return weights >= (int64_t(160) << 20) && group >= 64 ? 6 : 8;
  if (K > 4096) return weights >= (int64_t(32) << 20) ? 8 : 12;
  if (N >= 14336) return 8;
  return weights >= (int64_t(20) << 20) ? 9 : 16;
}

w4a16_path resolve_path(int64_t M, int64_t N, int64_t K, int32_t group, int32_t dtype,
                        int32_t has_zp, int32_t path) {
  if (path == W4A16_PATH_GEMV || path == W4A16_PATH_GEMM) return (w4a16_path)path;
  const int forced = w4a16::tuning().force_path;
  if (forced == W4A16_PATH_GEMV || forced == W4A16_PATH_GEMM) return (w4a16_path)forced;
  return M <= gemv_threshold(N, K, group, dtype, has_zp) ? W4A16_PATH_GEMV : W4A16_PATH_GEMM;
}

constexpr int kPlanningCUs = 256;  // MI355X; the launch plan uses the device's own count

size_t workspace_for(int64_t M, int64_t N, int64_t K, int32_t group, int32_t dtype, bool asym,
                     w4a16_path path, int cu_count) {
  if (M <= 0) return 0;
  if (path == W4A16_PATH_GEMV) {
    const w4a16::GemvPlan plan = w4a16::plan_gemv(M, N, K, group, dtype, cu_count);
    return w4a16::gemv_workspace_bytes(plan, M, N);
  }
  return w4a16::gemm_workspace_bytes(M, N, K, group, dtype, asym, cu_count);
}

bool log_enabled() { return w4a16::tuning().log; }

// the sizes that the path p takes
w4a16_status check_path(w4a16_path p, int64_t M, int64_t N, int64_t K) {
  if (p == W4A16_PATH_GEMV && M > W4A16_GEMV_MAX_M)
    return fail(W4A16_ERR_UNSUPPORTED, "the decode kernel takes M <= %d, got M=%lld",
                W4A16_GEMV_MAX_M, (long long)M);
  if (p == W4A16_PATH_GEMV && (uint64_t)N * (uint64_t)K / 2 > 0xFFFFFFFFull)
    return fail(W4A16_ERR_UNSUPPORTED,
                "the decode kernel addresses weights with 32-bit byte offsets: N*K/2 must be "
                "below 4 GiB (N=%lld K=%lld)", (long long)N, (long long)K);
  if (p == W4A16_PATH_GEMM && ((uint64_t)N * (uint64_t)K / 2 > 0xFFFFFFFFull ||
                               (uint64_t)M * (uint64_t)K * 2 > 0xFFFFFFFFull))
    return fail(W4A16_ERR_UNSUPPORTED,
                "the prefill kernel addresses weights and activations with 32-bit byte "
                "offsets: N*K/2 and M*K*2 must be below 4 GiB (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
  return ok();
}

// the launch of a checked problem (M > 0) on the path p
w4a16_status linear_run(const DeviceInfo* dev, w4a16_path p, const GroupMap& gm, const void* x, const int32_t* wq,
                        const void* scales, const int32_t* zp, const void* bias, void* y, int64_t M, int64_t N,
                        int64_t K, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream,
                        const w4a16::LoraTerm* lora) {
  const int32_t group_size = gm.kgroup;  // the kernels' group
  const w4a16_status st = check_path(p, M, N, K);
  if (st != W4A16_OK) return st;
  const size_t need = workspace_for(M, N, K, group_size, dtype, zp != nullptr, p, dev->cu_count);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(W4A16_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need,
                workspace_bytes, workspace ? "" : " (NULL)");
  if (need > 0 && !aligned(workspace, 256))
    return fail(W4A16_ERR_ALIGNMENT, "workspace must be 256-byte aligned");

  w4a16::LinearArgs a{x, wq, scales, zp, bias, y, M, N, K, group_size, dtype, gm.sG, gm.gmul};
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (p == W4A16_PATH_GEMV) {
    const w4a16::GemvPlan plan = w4a16::plan_gemv(M, N, K, group_size, dtype, dev->cu_count);
    if (log_enabled())
      std::fprintf(stderr,
                   "[w4a16] gemv M=%lld N=%lld K=%lld g=%d %s %s tiles=%d splits=%d waves=%d\n",
                   (long long)M, (long long)N, (long long)K, group_size,
                   dtype == W4A16_F16 ? "f16" : "bf16", zp ? "asym" : "sym", plan.tiles,
                   plan.splits, plan.waves);
    e = w4a16::launch_gemv(a, plan, workspace, s, nullptr, lora);
  } else {
    if (log_enabled()) {
      const w4a16::GemmPlan plan = w4a16::plan_gemm(M, N, K, group_size, dtype, zp != nullptr, dev->cu_count);
      std::fprintf(stderr,
                   "[w4a16] gemm M=%lld N=%lld K=%lld g=%d %s %s bm=%d bn=%d splits=%d units=%d\n",
                   (long long)M, (long long)N, (long long)K, group_size,
                   dtype == W4A16_F16 ? "f16" : "bf16", zp ? "asym" : "sym", 32 * plan.mb,
                   128 * plan.cb, plan.splits, plan.units);
    }
    e = w4a16::launch_gemm(a, workspace, dev->cu_count, s, lora);
  }
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

w4a16_status linear_impl(const void* x, const int32_t* wq, const void* scales, const int32_t* zp,
                         const void* bias, void* y, int64_t M, int64_t N, int64_t K,
                         int32_t group_size, int32_t dtype, void* workspace,
                         size_t workspace_bytes, void* stream, int32_t path) {
  w4a16_status st = w4a16_check_args(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype);
  if (st != W4A16_OK) return st;
  const GroupMap gm = group_map(group_size, K);
  if (path < W4A16_PATH_AUTO || path > W4A16_PATH_GEMM)
    return fail(W4A16_ERR_INVALID_ARG, "unknown path %d", (int)path);
  if (M == 0) return ok();
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const w4a16_path p = resolve_path(M, N, K, gm.kgroup, dtype, zp != nullptr, path);
  return linear_run(dev, p, gm, x, wq, scales, zp, bias, y, M, N, K, dtype, workspace, workspace_bytes, stream, nullptr);
}

// the CU count that plans are made for: the current device's, or MI355X's
// where none is visible
int planning_cus() {
  int cus = kPlanningCUs, dev = -1;
  if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices) {
    const DeviceInfo* d = nullptr;
    if (device_info(&d) == W4A16_OK) cus = d->cu_count;
    g_last_error.clear();
  }
  return cus;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// ---- low-rank adapters ------------------------------------------------------
w4a16_status check_adapters(const char* what, const void* la, const void* lb, const int32_t* ids,
                            const float* alpha, int64_t M, int64_t N, int64_t K, int64_t S, int64_t R) {
  if (S < 1 || S > INT32_MAX) return fail(W4A16_ERR_INVALID_ARG, "%s: need at least one adapter, got S=%lld", what, (long long)S);
  if (R < 8 || R % 8) return fail(W4A16_ERR_INVALID_ARG, "%s: the rank must be a positive multiple of 8, got %lld", what, (long long)R);
  if (R > w4a16::kMaxRank)
    return fail(W4A16_ERR_UNSUPPORTED, "%s: ranks above %d are not supported, got %lld", what, w4a16::kMaxRank, (long long)R);
  if (S > INT64_MAX / 4 / (R * std::max(N, K)))
    return fail(W4A16_ERR_INVALID_ARG, "%s: adapter stacks too large", what);
  if (M == 0) return ok();
  if (!la || !lb || !ids) return fail(W4A16_ERR_INVALID_ARG, "%s: la, lb and ids must not be NULL", what);
  if (!aligned(la, 16) || !aligned(lb, 16)) return fail(W4A16_ERR_ALIGNMENT, "%s: la and lb must be 16-byte aligned", what);
  if (!aligned(ids, 4) || (alpha && !aligned(alpha, 4)))
    return fail(W4A16_ERR_ALIGNMENT, "%s: ids and alpha must be 4-byte aligned", what);
  return ok();
}

// [out, out + bytes) against the adapters' inputs
bool overlaps_adapters(const void* out, size_t bytes, const void* la, const void* lb, const int32_t* ids,
                       const float* alpha, int64_t M, int64_t N, int64_t K, int64_t S, int64_t R) {
  return overlap(out, bytes, la, act_bytes(S * R * K)) || overlap(out, bytes, lb, act_bytes(S * N * R)) ||
         overlap(out, bytes, ids, (size_t)M * 4) || (alpha && overlap(out, bytes, alpha, (size_t)S * 4));
}

// The kernel beside adapters: the decode kernel for every M it takes, also
// where the thin GEMM tiles alone would be faster (they need the K ranges of u
// added by a launch of their own, and mostly a second pass for their K split).
w4a16_path lora_path(int64_t M, int64_t N, int64_t K, int32_t group, int32_t dtype, int32_t has_zp) {
  const w4a16_path p = resolve_path(M, N, K, group, dtype, has_zp, W4A16_PATH_AUTO);
  return M <= W4A16_GEMV_MAX_M && w4a16::tuning().force_path == 0 && w4a16::tuning().m_threshold < 0 ? W4A16_PATH_GEMV : p;
}

// the workspace of w4a16_lora_linear: the projection's own (its counter region
// always kept, so that one workspace serves every entry point), then the K
// ranges' sums of u (one range goes to the caller's u where it is kept), and
// alpha * u as operands for the matrix tiles
struct LoraPlan {
  w4a16_path path;
  w4a16::ShrinkPlan shrink;
  size_t u_at, op_at, shift_at, bytes;
};
LoraPlan plan_lora(int64_t M, int64_t N, int64_t K, int32_t kgroup, int32_t dtype, bool asym, int R, bool save_u, int cus) {
  LoraPlan p;
  p.path = lora_path(M, N, K, kgroup, dtype, asym);
  p.shrink = w4a16::plan_shrink(M, K, R, cus, p.path == W4A16_PATH_GEMV);
  p.u_at = round256(std::max(w4a16::kCounterBytes, workspace_for(M, N, K, kgroup, dtype, asym, p.path, cus)));
  const size_t plane = (size_t)M * (size_t)R * sizeof(float);
  p.op_at = p.u_at + round256(save_u && p.shrink.splits == 1 ? 0 : (size_t)p.shrink.splits * plane);
  p.shift_at = p.op_at + (p.path == W4A16_PATH_GEMV ? 0 : round256(plane));
  p.bytes = p.shift_at + (p.path == W4A16_PATH_GEMV || dtype != W4A16_F16 ? 0 : round256((size_t)M * 4));
  return p;
}

// the workspace of w4a16_lora_backward, by byte offsets behind the counter
// region that every entry point leaves zero
struct BackwardPlan {
  int64_t np;  // N rounded up to 64: the rows of dy and of the transposed lb
  w4a16::ShrinkPlan shrink;
  w4a16::OuterPlan outer;
  w4a16::DxPlan dx;
  int64_t places;  // of the tokens' order
  size_t zeros, order, start, count, la_t, lb_t, dy_pad, part, g, op[2], g_shift, op_shift[2], outer_part, dx_part, tail_w,
      constants, bytes;
  size_t zero_bytes;  // the outer products' counters, zero when they start
};
BackwardPlan plan_backward(int64_t M, int64_t N, int64_t K, int32_t group_size, int64_t S, int64_t R, int32_t dtype, int cus) {
  BackwardPlan p;
  p.np = (N + 63) / 64 * 64;
  p.shrink = w4a16::plan_shrink(M, p.np, (int)R, cus, false);
  p.outer = w4a16::plan_outer(M, K, N, (int)S, (int)R, cus);
  p.dx = w4a16::plan_dx(M, N, K, cus);
  size_t at = w4a16::kCounterBytes;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += round256(n);
    return was;
  };
  p.zero_bytes = w4a16::outer_counter_bytes(p.outer, (int)S);
  p.zeros = take(p.zero_bytes);
  p.places = w4a16::order_places(M, S);
  p.order = take((size_t)p.places * 4);
  p.start = take((size_t)S * 4);
  p.count = take((size_t)S * 4);
  p.la_t = take(act_bytes(S * K * R));
  p.lb_t = take(act_bytes(S * p.np * R));
  p.dy_pad = take(p.np != N ? act_bytes(M * p.np) : 0);
  p.part = take((size_t)p.shrink.splits * (size_t)M * (size_t)R * 4);
  p.g = take((size_t)M * (size_t)R * 4);
  for (size_t& o : p.op) o = take(act_bytes(2 * R * p.places));
  const bool shifted = dtype == W4A16_F16;
  p.g_shift = take(shifted ? (size_t)M * 4 : 0);
  for (size_t& o : p.op_shift) o = take(shifted ? (size_t)w4a16::shift_row(R) * (size_t)(p.places / 32) : 0);
  // the two are not in use at the same time, but both stay clear of the rest
  p.outer_part = take(w4a16::outer_partial_bytes(p.outer, p.places));
  p.dx_part = take(w4a16::dx_partial_bytes(p.dx, M, K));
  p.tail_w = take(p.np != N ? (size_t)K * 32 : 0);
  p.constants = take(w4a16::dx_constant_bytes(p.np, K / group_size, dtype));
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" {

int w4a16_abi_version(void) { return W4A16_ABI_VERSION; }

void w4a16_reload_tuning(void) { w4a16::reload_tuning(); }

const char* w4a16_last_error(void) { return g_last_error.c_str(); }

// nibble t of a word holds k-offset (0,2,4,6,1,3,5,7)[t]; the inverse map:
static const int kSlotOfKoff[8] = {0, 4, 1, 5, 2, 6, 3, 7};

// The 8-k slice held by stored word j of a row of J words: complete runs of
// 16 words are stored as the 4x4 transpose (word 4r+t <-> slice 4t+r, its own
// inverse); an incomplete last run is stored in order.
static int64_t slice_of_stored_word(int64_t j, int64_t J) {
  const int64_t run = j / 16, p = j % 16;
  if ((run + 1) * 16 > J) return j;
  return run * 16 + 4 * (p % 4) + p / 4;
}

// Where stored word j of row n sits in the packed tensor.  Rows are grouped
// in tiles of 16; a complete tile holds, for each complete run, one block of
// 256 words whose 16-byte piece 16 r + (n mod 16) is the row's run words
// 4r..4r+3, then the 16 rows' incomplete runs row after row.  The rows of a
// final incomplete tile are stored one after another.
static int64_t stored_position(int64_t n, int64_t j, int64_t N, int64_t J) {
  const int64_t tile = n / 16, row = n % 16;
  if ((tile + 1) * 16 > N) return n * J + j;
  const int64_t runs = J / 16, tail = J - 16 * runs;
  const int64_t base = tile * 16 * J;
  if (j < 16 * runs) {
    const int64_t run = j / 16, p = j % 16;
    return base + 256 * run + 4 * (16 * (p / 4) + row) + p % 4;
  }
  return base + 256 * runs + tail * row + (j - 16 * runs);
}

w4a16_status w4a16_pack_weights(const uint8_t* q, int64_t N, int64_t K, int32_t* wq) {
  if (!q || !wq) return fail(W4A16_ERR_INVALID_ARG, "pack_weights: NULL pointer");
  if (N < 0 || K < 0 || K % 8) return fail(W4A16_ERR_INVALID_ARG, "pack_weights: need N >= 0, K >= 0, K %% 8 == 0 (N=%lld K=%lld)", (long long)N, (long long)K);
  for (int64_t i = 0; i < N * K; ++i)
    if (q[i] > 15) return fail(W4A16_ERR_INVALID_ARG, "pack_weights: code %u at %lld exceeds 15", (unsigned)q[i], (long long)i);
  const int64_t J = K / 8;
  for (int64_t n = 0; n < N; ++n)
    for (int64_t j = 0; j < J; ++j) {
      const uint8_t* src = q + n * K + slice_of_stored_word(j, J) * 8;
      uint32_t w = 0;
      for (int i = 0; i < 8; ++i) w |= (uint32_t)src[i] << (4 * kSlotOfKoff[i]);
      wq[stored_position(n, j, N, J)] = (int32_t)w;
    }
  return ok();
}

w4a16_status w4a16_unpack_weights(const int32_t* wq, int64_t N, int64_t K, uint8_t* q) {
  if (!q || !wq) return fail(W4A16_ERR_INVALID_ARG, "unpack_weights: NULL pointer");
  if (N < 0 || K < 0 || K % 8) return fail(W4A16_ERR_INVALID_ARG, "unpack_weights: need N >= 0, K >= 0, K %% 8 == 0");
  const int64_t J = K / 8;
  for (int64_t n = 0; n < N; ++n)
    for (int64_t j = 0; j < J; ++j) {
      const uint32_t w = (uint32_t)wq[stored_position(n, j, N, J)];
      uint8_t* dst = q + n * K + slice_of_stored_word(j, J) * 8;
      for (int i = 0; i < 8; ++i) dst[i] = (uint8_t)((w >> (4 * kSlotOfKoff[i])) & 0xFu);
    }
  return ok();
}

w4a16_status w4a16_pack_zeros(const uint8_t* z, int64_t N, int64_t G, int32_t* zpk) {
  if (!z || !zpk) return fail(W4A16_ERR_INVALID_ARG, "pack_zeros: NULL pointer");
  if (N < 0 || G < 0 || N % 8) return fail(W4A16_ERR_INVALID_ARG, "pack_zeros: need N >= 0, G >= 0, N %% 8 == 0 (N=%lld)", (long long)N);
  for (int64_t i = 0; i < N * G; ++i)
    if (z[i] > 15) return fail(W4A16_ERR_INVALID_ARG, "pack_zeros: zero point %u at %lld exceeds 15", (unsigned)z[i], (long long)i);
  for (int64_t r = 0; r < N / 8; ++r)
    for (int64_t g = 0; g < G; ++g) {
      uint32_t w = 0;
      for (int i = 0; i < 8; ++i) w |= (uint32_t)z[(r * 8 + i) * G + g] << (4 * i);
      zpk[r * G + g] = (int32_t)w;
    }
  return ok();
}

w4a16_status w4a16_unpack_zeros(const int32_t* zpk, int64_t N, int64_t G, uint8_t* z) {
  if (!z || !zpk) return fail(W4A16_ERR_INVALID_ARG, "unpack_zeros: NULL pointer");
  if (N < 0 || G < 0 || N % 8) return fail(W4A16_ERR_INVALID_ARG, "unpack_zeros: need N >= 0, G >= 0, N %% 8 == 0");
  for (int64_t r = 0; r < N / 8; ++r)
    for (int64_t g = 0; g < G; ++g) {
      const uint32_t w = (uint32_t)zpk[r * G + g];
      for (int i = 0; i < 8; ++i) z[(r * 8 + i) * G + g] = (uint8_t)((w >> (4 * i)) & 0xFu);
    }
  return ok();
}

// everything of w4a16_check_args but the overlap of y
static w4a16_status check_problem(const void* x, const int32_t* wq, const void* scales,
                                  const int32_t* zp, const void* bias, const void* y, int64_t M,
                                  int64_t N, int64_t K, int32_t group_size, int32_t dtype) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "activation dtype must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (!group_ok(group_size, K))
    return fail(W4A16_ERR_UNSUPPORTED,
                "group size must be 32, 64, 128 or K (per-channel, K %% 32 == 0), got %d (K=%lld)",
                (int)group_size, (long long)K);
  if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M must be >= 0, got %lld", (long long)M);
  if (N < 1) return fail(W4A16_ERR_INVALID_ARG, "N must be >= 1, got %lld", (long long)N);
  if (K < group_size || K % group_size)
    return fail(W4A16_ERR_INVALID_ARG, "K must be a positive multiple of the group size %d, got K=%lld",
                (int)group_size, (long long)K);
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || M * K > INT64_MAX / 2 || N * K > INT64_MAX / 2)
    return fail(W4A16_ERR_INVALID_ARG, "problem too large");
  if (K > w4a16::kMaxK)
    return fail(W4A16_ERR_UNSUPPORTED, "K above %lld is not supported (the kernels' 32-bit offsets), got K=%lld",
                (long long)w4a16::kMaxK, (long long)K);
  if (zp && N % 8)
    return fail(W4A16_ERR_INVALID_ARG, "packed zero points need N %% 8 == 0, got N=%lld", (long long)N);
  if (M == 0) return ok();
  if (!x || !wq || !scales || !y) return fail(W4A16_ERR_INVALID_ARG, "x, wq, scales and y must not be NULL");
  if (!aligned(x, 16)) return fail(W4A16_ERR_ALIGNMENT, "x must be 16-byte aligned");
  if (!aligned(wq, 16)) return fail(W4A16_ERR_ALIGNMENT, "wq must be 16-byte aligned");
  if (!aligned(scales, 2) || !aligned(y, 2) || (bias && !aligned(bias, 2)))
    return fail(W4A16_ERR_ALIGNMENT, "scales, bias and y must be 2-byte aligned");
  if (zp && !aligned(zp, 4)) return fail(W4A16_ERR_ALIGNMENT, "zp must be 4-byte aligned");
  return ok();
}

w4a16_status w4a16_check_args(const void* x, const int32_t* wq, const void* scales,
                              const int32_t* zp, const void* bias, const void* y, int64_t M,
                              int64_t N, int64_t K, int32_t group_size, int32_t dtype) {
  const w4a16_status st = check_problem(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype);
  if (st != W4A16_OK || M == 0) return st;
  const int64_t G = K / group_size;
  const size_t ybytes = act_bytes(M * N);
  if (overlap(y, ybytes, x, act_bytes(M * K)) || overlap(y, ybytes, wq, (size_t)N * (K / 8) * 4) ||
      overlap(y, ybytes, scales, act_bytes(N * G)) ||
      (zp && overlap(y, ybytes, zp, (size_t)(N / 8) * G * 4)) ||
      (bias && overlap(y, ybytes, bias, act_bytes(N))))
    return fail(W4A16_ERR_INVALID_ARG, "y must not overlap any input");
  return ok();
}

w4a16_path w4a16_select_path(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                             int32_t has_zp) {
  return resolve_path(M, N, K, group_size, dtype, has_zp, W4A16_PATH_AUTO);
}

size_t w4a16_workspace_size(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                            int32_t has_zp, int32_t path) {
  if (M <= 0 || N <= 0 || K <= 0 || !group_ok(group_size, K) || K % group_size) return 0;
  const int kgroup = group_map(group_size, K).kgroup;
  const w4a16_path p = resolve_path(M, N, K, kgroup, dtype, has_zp, path);
  int cus = kPlanningCUs;
  int dev = -1;
  if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices) {
    const DeviceInfo* d = nullptr;
    if (device_info(&d) == W4A16_OK) cus = d->cu_count;
    g_last_error.clear();
  }
  return workspace_for(M, N, K, kgroup, dtype, has_zp != 0, p, cus);
}

w4a16_status w4a16_plan(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                        int32_t has_zp, int32_t path, w4a16_plan_info* out) {
  if (!out) return fail(W4A16_ERR_INVALID_ARG, "plan: out must not be NULL");
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "activation dtype must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (!group_ok(group_size, K))
    return fail(W4A16_ERR_UNSUPPORTED,
                "group size must be 32, 64, 128 or K (per-channel, K %% 32 == 0), got %d (K=%lld)",
                (int)group_size, (long long)K);
  if (M < 1 || N < 1 || K < group_size || K % group_size || M > INT32_MAX || N > INT32_MAX)
    return fail(W4A16_ERR_INVALID_ARG, "plan: need M >= 1, N >= 1 and K a positive multiple of the group");
  if (K > w4a16::kMaxK)
    return fail(W4A16_ERR_UNSUPPORTED, "K above %lld is not supported", (long long)w4a16::kMaxK);
  if (has_zp && N % 8)
    return fail(W4A16_ERR_INVALID_ARG, "packed zero points need N %% 8 == 0, got N=%lld", (long long)N);
  if (path < W4A16_PATH_AUTO || path > W4A16_PATH_GEMM)
    return fail(W4A16_ERR_INVALID_ARG, "unknown path %d", (int)path);
  const GroupMap gm = group_map(group_size, K);
  const w4a16_path p = resolve_path(M, N, K, gm.kgroup, dtype, has_zp, path);
  if (p == W4A16_PATH_GEMV && M > W4A16_GEMV_MAX_M)
    return fail(W4A16_ERR_UNSUPPORTED, "the decode kernel takes M <= %d, got M=%lld",
                W4A16_GEMV_MAX_M, (long long)M);
  int cus = kPlanningCUs;
  int dev = -1;
  if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices) {
    const DeviceInfo* d = nullptr;
    if (device_info(&d) == W4A16_OK) cus = d->cu_count;
  }
  w4a16_plan_info r{};
  r.path = p;
  if (p == W4A16_PATH_GEMV) {
    const w4a16::GemvPlan g = w4a16::plan_gemv(M, N, K, gm.kgroup, dtype, cus);
    r.tile_features = w4a16::kGemvRowsPerTile;
    r.tile_tokens = w4a16::kGemvMaxM;
    r.tiles = g.tiles;
    if (g.one_kpw && gm.gmul == 1) {
      // the single-token instance (given 16-byte aligned scales and zero points)
      r.kernel = 1;
      r.splits = g.one_splits;
      r.waves = g.one_waves;
      r.launches = 1;
      r.counter_tiles = g.one_splits > 1 ? g.tiles : 0;
    } else {
      r.splits = g.splits;
      r.waves = g.waves;
      r.launches = g.splits > 1 ? (int32_t)((g.tiles + w4a16::kMaxCounters - 1) / w4a16::kMaxCounters) : 1;
      r.counter_tiles = g.splits > 1 ? std::min<int64_t>(g.tiles, w4a16::kMaxCounters) : 0;
    }
  } else {
    const w4a16::GemmPlan g = w4a16::plan_gemm(M, N, K, gm.kgroup, dtype, has_zp != 0, cus);
    r.tile_features = 128 * g.cb;
    r.tile_tokens = 32 * g.mb;
    r.splits = g.splits;
    r.tiles = g.tiles;
    r.waves = 4;
    r.two_pass = g.splits > 1 && g.two_pass;
    r.launches = (r.two_pass ? 2 : 1) + (g.tail_units > 0 ? 1 : 0);
    r.counter_tiles = g.splits > 1 && !g.two_pass ? g.tiles : 0;
    if (g.tail_units > 0) {
      r.tail_tile_tokens = 32 * g.tail_mb;
      r.tail_tile_features = 128 * g.cb;
      r.tail_tiles = g.tail_units;
    }
  }
  r.workspace_bytes = workspace_for(M, N, K, gm.kgroup, dtype, has_zp != 0, p, cus);
  *out = r;
  return ok();
}

w4a16_status w4a16_linear(const void* x, const int32_t* wq, const void* scales, const int32_t* zp,
                          const void* bias, void* y, int64_t M, int64_t N, int64_t K,
                          int32_t group_size, int32_t dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return linear_impl(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype, workspace,
                     workspace_bytes, stream, W4A16_PATH_AUTO);
}

w4a16_status w4a16_linear_path(const void* x, const int32_t* wq, const void* scales,
                               const int32_t* zp, const void* bias, void* y, int64_t M, int64_t N,
                               int64_t K, int32_t group_size, int32_t dtype, void* workspace,
                               size_t workspace_bytes, void* stream, int32_t path) {
  return linear_impl(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype, workspace,
                     workspace_bytes, stream, path);
}

w4a16_status w4a16_linear_noalloc(const void* x, const int32_t* wq, const void* scales,
                                  const int32_t* zp, const void* bias, void* y, int64_t M,
                                  int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                                  void* stream) {
  w4a16_status st = w4a16_check_args(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype);
  if (st != W4A16_OK) return st;
  if (M == 0) return ok();
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const GroupMap gm = group_map(group_size, K);
  const w4a16_path p = resolve_path(M, N, K, gm.kgroup, dtype, zp != nullptr, W4A16_PATH_AUTO);
  const size_t need = workspace_for(M, N, K, gm.kgroup, dtype, zp != nullptr, p, dev->cu_count);
  if (need > kScratchBytes)
    return fail(W4A16_ERR_UNSUPPORTED,
                "w4a16_linear_noalloc: this problem needs %zu bytes of split-K workspace, above the "
                "%zu bytes of scratch it holds; call w4a16_linear with a workspace instead",
                need, kScratchBytes);
  void* ws = nullptr;
  if (need > 0) {
    int d = -1;
    if (hipGetDevice(&d) != hipSuccess || d < 0 || d >= kMaxDevices)
      return fail(W4A16_ERR_DEVICE, "noalloc: no current device");
    st = scratch_for(g_devices[d], d, static_cast<hipStream_t>(stream), &ws);
    if (st != W4A16_OK) return st;
  }
  return linear_impl(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype, ws, need, stream,
                     W4A16_PATH_AUTO);
}

w4a16_status w4a16_dequant(const int32_t* wq, const void* scales, const int32_t* zp, void* w,
                           int64_t N, int64_t K, int32_t group_size, int32_t dtype, void* stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "activation dtype must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (!group_ok(group_size, K))
    return fail(W4A16_ERR_UNSUPPORTED,
                "group size must be 32, 64, 128 or K (per-channel, K %% 32 == 0), got %d (K=%lld)",
                (int)group_size, (long long)K);
  if (N < 1 || K < group_size || K % group_size)
    return fail(W4A16_ERR_INVALID_ARG, "need N >= 1 and K a positive multiple of the group size");
  if (zp && N % 8) return fail(W4A16_ERR_INVALID_ARG, "packed zero points need N %% 8 == 0");
  if (!wq || !scales || !w) return fail(W4A16_ERR_INVALID_ARG, "wq, scales and w must not be NULL");
  if (!aligned(wq, 4) || !aligned(w, 16) || !aligned(scales, 2) || (zp && !aligned(zp, 4)))
    return fail(W4A16_ERR_ALIGNMENT, "w must be 16-byte aligned, wq and zp 4-byte, scales 2-byte");
  const DeviceInfo* dev = nullptr;
  w4a16_status st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const GroupMap gm = group_map(group_size, K);
  hipError_t e = w4a16::launch_dequant(wq, scales, zp, gm.sG, gm.gmul, w, N, K, gm.kgroup, dtype,
                                       static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

w4a16_status w4a16_moe_linear(const void* x, const int32_t* wq, const void* scales,
                              const int32_t* zp, const void* bias, const int32_t* topk_ids,
                              const float* topk_weights, void* y, int64_t M, int64_t topk,
                              int64_t E, int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                              int32_t x_per_slot, void* stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "activation dtype must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (!group_ok(group_size, K))
    return fail(W4A16_ERR_UNSUPPORTED,
                "group size must be 32, 64, 128 or K (per-channel, K %% 32 == 0), got %d (K=%lld)",
                (int)group_size, (long long)K);
  if (M < 0 || topk < 1 || E < 1 || N < 1)
    return fail(W4A16_ERR_INVALID_ARG, "need M >= 0, topk >= 1, E >= 1, N >= 1");
  if (K < group_size || K % group_size)
    return fail(W4A16_ERR_INVALID_ARG, "K must be a positive multiple of the group size %d, got K=%lld",
                (int)group_size, (long long)K);
  if (zp && N % 8)
    return fail(W4A16_ERR_INVALID_ARG, "packed zero points need N %% 8 == 0, got N=%lld", (long long)N);
  if (M * topk > w4a16::kMaxGridZ || N > INT32_MAX || K > INT32_MAX || E > INT32_MAX)
    return fail(W4A16_ERR_UNSUPPORTED, "M * topk must be at most %lld", (long long)w4a16::kMaxGridZ);
  if ((uint64_t)N * (uint64_t)K / 2 > 0xFFFFFFFFull)
    return fail(W4A16_ERR_UNSUPPORTED, "one expert's weights must be below 4 GiB (N*K/2)");
  if (K > w4a16::kMaxK)
    return fail(W4A16_ERR_UNSUPPORTED, "K above %lld is not supported (the kernels' 32-bit offsets), got K=%lld",
                (long long)w4a16::kMaxK, (long long)K);
  if (M == 0) return ok();
  if (!x || !wq || !scales || !topk_ids || !y)
    return fail(W4A16_ERR_INVALID_ARG, "x, wq, scales, topk_ids and y must not be NULL");
  if (!aligned(x, 16) || !aligned(wq, 16))
    return fail(W4A16_ERR_ALIGNMENT, "x and wq must be 16-byte aligned");
  if (!aligned(scales, 2) || !aligned(y, 2) || (bias && !aligned(bias, 2)) || !aligned(topk_ids, 4) ||
      (topk_weights && !aligned(topk_weights, 4)) || (zp && !aligned(zp, 4)))
    return fail(W4A16_ERR_ALIGNMENT, "scales, bias and y must be 2-byte aligned; zp, topk_ids and "
                "topk_weights 4-byte aligned");
  const int64_t slots = M * topk;
  const int64_t G = K / group_size;
  const size_t ybytes = act_bytes(slots * N);
  if (overlap(y, ybytes, x, act_bytes((x_per_slot ? slots : M) * K)) ||
      overlap(y, ybytes, wq, (size_t)E * N * (K / 8) * 4) || overlap(y, ybytes, scales, act_bytes(E * N * G)) ||
      (zp && overlap(y, ybytes, zp, (size_t)E * (N / 8) * G * 4)) ||
      (bias && overlap(y, ybytes, bias, act_bytes(E * N))) || overlap(y, ybytes, topk_ids, (size_t)slots * 4) ||
      (topk_weights && overlap(y, ybytes, topk_weights, (size_t)slots * 4)))
    return fail(W4A16_ERR_INVALID_ARG, "y must not overlap any input");
  const DeviceInfo* dev = nullptr;
  w4a16_status st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const GroupMap gm = group_map(group_size, K);
  // one K range per slot (the slots fill the device): planned as if for one CU
  const w4a16::GemvPlan plan = w4a16::plan_gemv(1, N, K, gm.kgroup, dtype, 1);
  w4a16::LinearArgs a{x, wq, scales, zp, bias, y, 1, N, K, gm.kgroup, dtype, gm.sG, gm.gmul};
  w4a16::MoeArgs moe{topk_ids, topk_weights, topk, E, slots, x_per_slot != 0};
  if (plan.splits != 1 && !w4a16::gemv_one_runs(a, plan, &moe))
    return fail(W4A16_ERR_UNSUPPORTED, "K=%lld is too large for one decode workgroup per slot",
                (long long)K);
  hipError_t e = w4a16::launch_gemv(a, plan, nullptr, static_cast<hipStream_t>(stream), &moe);
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

size_t w4a16_dense_workspace_size(int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t has_bias) {
  (void)has_bias;
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 || (dtype != W4A16_F16 && dtype != W4A16_BF16)) return 0;
  int cus = kPlanningCUs;
  int dev = -1;
  if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices) {
    const DeviceInfo* d = nullptr;
    if (device_info(&d) == W4A16_OK) cus = d->cu_count;
    g_last_error.clear();
  }
  return w4a16::gemm_workspace_bytes(M, N, K, 128, dtype, false, cus, true);
}

w4a16_status w4a16_linear_dense(const void* x, const void* w, const void* bias, void* y, int64_t M,
                                int64_t N, int64_t K, int32_t dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_INVALID_ARG, "activation dtype must be fp16 (0) or bf16 (1), got %d", (int)dtype);
  if (M < 0 || N < 1 || K < 32 || K % 32)
    return fail(W4A16_ERR_INVALID_ARG, "need M >= 0, N >= 1 and K a positive multiple of 32 (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
  if ((uint64_t)N * (uint64_t)K * 2 > 0xFFFFFFFFull || (uint64_t)M * (uint64_t)K * 2 > 0xFFFFFFFFull ||
      M > INT32_MAX || N > INT32_MAX)
    return fail(W4A16_ERR_UNSUPPORTED,
                "the dense path addresses w and x with 32-bit byte offsets: N*K*2 and M*K*2 must be "
                "below 4 GiB (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
  if (M == 0) return ok();
  if (!x || !w || !y) return fail(W4A16_ERR_INVALID_ARG, "x, w and y must not be NULL");
  if (!aligned(x, 16) || !aligned(w, 16))
    return fail(W4A16_ERR_ALIGNMENT, "x and w must be 16-byte aligned");
  if (!aligned(y, 2) || (bias && !aligned(bias, 2)))
    return fail(W4A16_ERR_ALIGNMENT, "bias and y must be 2-byte aligned");
  const size_t ny = act_bytes(M * N);
  if (overlap(y, ny, x, act_bytes(M * K)) || overlap(y, ny, w, act_bytes(N * K)) ||
      overlap(y, ny, bias, bias ? act_bytes(N) : 0))
    return fail(W4A16_ERR_INVALID_ARG, "y must not overlap x, w or bias");
  const DeviceInfo* dev = nullptr;
  w4a16_status st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const size_t need = w4a16::gemm_workspace_bytes(M, N, K, 128, dtype, false, dev->cu_count, true);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(W4A16_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need,
                workspace_bytes, workspace ? "" : " (NULL)");
  if (need > 0 && !aligned(workspace, 256))
    return fail(W4A16_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (need > 0 && (overlap(workspace, need, y, ny) || overlap(workspace, need, x, act_bytes(M * K)) ||
                   overlap(workspace, need, w, act_bytes(N * K))))
    return fail(W4A16_ERR_INVALID_ARG, "the workspace must not overlap x, w or y");
  // the prefill GEMM's dense instances: w in place of the packed codes, no
  // scales or zero points
  w4a16::LinearArgs a{x, static_cast<const int32_t*>(w), nullptr, nullptr, bias, y, M, N, K, 128, dtype, 0, 0};
  a.dense = true;
  const hipError_t e = w4a16::launch_gemm(a, workspace, dev->cu_count, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

size_t w4a16_lora_workspace_size(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t dtype,
                                 int32_t has_zp, int64_t R, int32_t save_u) {
  if (M <= 0 || N <= 0 || K <= 0 || !group_ok(group_size, K) || K % group_size || R < 8 || R % 8 || R > w4a16::kMaxRank ||
      (dtype != W4A16_F16 && dtype != W4A16_BF16))
    return 0;
  return plan_lora(M, N, K, group_map(group_size, K).kgroup, dtype, has_zp != 0, (int)R, save_u != 0, planning_cus()).bytes;
}

w4a16_status w4a16_lora_linear(const void* x, const int32_t* wq, const void* scales, const int32_t* zp,
                               const void* bias, const void* la, const void* lb, const int32_t* ids,
                               const float* alpha, void* y, float* u, int64_t M, int64_t N, int64_t K,
                               int32_t group_size, int64_t S, int64_t R, int32_t dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
  w4a16_status st = w4a16_check_args(x, wq, scales, zp, bias, y, M, N, K, group_size, dtype);
  if (st != W4A16_OK) return st;
  st = check_adapters("lora_linear", la, lb, ids, alpha, M, N, K, S, R);
  if (st != W4A16_OK) return st;
  if (M == 0) return ok();
  if (u && !aligned(u, 16)) return fail(W4A16_ERR_ALIGNMENT, "lora_linear: u must be 16-byte aligned");
  const size_t ubytes = (size_t)M * (size_t)R * sizeof(float), ybytes = act_bytes(M * N);
  if (overlaps_adapters(y, ybytes, la, lb, ids, alpha, M, N, K, S, R) ||
      (u && (overlaps_adapters(u, ubytes, la, lb, ids, alpha, M, N, K, S, R) || overlap(u, ubytes, y, ybytes) ||
             overlap(u, ubytes, x, act_bytes(M * K)) || overlap(u, ubytes, wq, (size_t)N * (K / 8) * 4) ||
             overlap(u, ubytes, scales, act_bytes(N * (K / group_size))) ||
             (zp && overlap(u, ubytes, zp, (size_t)(N / 8) * (K / group_size) * 4)) ||
             (bias && overlap(u, ubytes, bias, act_bytes(N))))))
    return fail(W4A16_ERR_INVALID_ARG, "lora_linear: y and u must not overlap any input or each other");
  const GroupMap gm = group_map(group_size, K);
  // (before u is formed, so that a refused call has launched nothing)
  st = check_path(lora_path(M, N, K, gm.kgroup, dtype, zp != nullptr), M, N, K);
  if (st != W4A16_OK) return st;
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const LoraPlan plan = plan_lora(M, N, K, gm.kgroup, dtype, zp != nullptr, (int)R, u != nullptr, dev->cu_count);
  if (workspace == nullptr || workspace_bytes < plan.bytes)
    return fail(W4A16_ERR_WORKSPACE, "lora_linear: workspace of %zu bytes needed, got %zu%s", plan.bytes, workspace_bytes,
                workspace ? "" : " (NULL)");
  if (!aligned(workspace, 256)) return fail(W4A16_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (overlaps_adapters(workspace, plan.bytes, la, lb, ids, alpha, M, N, K, S, R) ||
      overlap(workspace, plan.bytes, y, ybytes) || overlap(workspace, plan.bytes, u, ubytes) ||
      overlap(workspace, plan.bytes, x, act_bytes(M * K)) || overlap(workspace, plan.bytes, wq, (size_t)N * (K / 8) * 4) ||
      overlap(workspace, plan.bytes, scales, act_bytes(N * (K / group_size))) ||
      overlap(workspace, plan.bytes, zp, (size_t)(N / 8) * (K / group_size) * 4) ||
      overlap(workspace, plan.bytes, bias, act_bytes(N)))
    return fail(W4A16_ERR_INVALID_ARG, "lora_linear: the workspace must not overlap an input or an output");
  const w4a16_path p = plan.path;
  const w4a16::ShrinkPlan& sp = plan.shrink;
  // Decode: the epilogue adds the K ranges' sums itself, which saves a launch
  // (a few floats per output).  Above it every tile of the GEMM reads all of
  // its tokens' alpha * u as operands, made once, before it.
  float* const part = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.u_at);
  uint16_t* const op = p == W4A16_PATH_GEMV ? nullptr : reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + plan.op_at);
  int32_t* const shift = op && dtype == W4A16_F16 ? reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + plan.shift_at) : nullptr;
  const w4a16::ShrinkArgs sa{x, la, ids, part, u, op, shift, alpha, M, K, (int)S, (int)R, dtype};
  const hipError_t e = w4a16::launch_shrink(sa, sp, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  w4a16::LoraTerm t;
  t.ids = ids;
  t.up = lb;
  t.u = u ? u : part;
  t.alpha = alpha;
  t.op = op;
  t.shift = shift;
  t.S = (int)S;
  t.R = (int)R;
  t.usplits = u ? 1 : sp.splits;
  return linear_run(dev, p, gm, x, wq, scales, zp, bias, y, M, N, K, dtype, workspace, plan.u_at, stream, &t);
}

size_t w4a16_lora_backward_workspace_size(int64_t M, int64_t N, int64_t K, int32_t group_size, int64_t S, int64_t R,
                                          int32_t dtype) {
  if (M <= 0 || N <= 0 || K <= 0 || !group_ok(group_size, K) || K % group_size || S < 1 || S > 65535 || R < 8 || R % 8 ||
      R > w4a16::kMaxRank || (dtype != W4A16_F16 && dtype != W4A16_BF16))
    return 0;
  return plan_backward(M, N, K, group_size, S, R, dtype, planning_cus()).bytes;
}

w4a16_status w4a16_lora_backward(const void* dy, const void* x, const float* u, const int32_t* wq, const void* scales,
                                 const int32_t* zp, const void* la, const void* lb, const int32_t* ids,
                                 const float* alpha, void* dx, void* dla, void* dlb, int64_t M, int64_t N, int64_t K,
                                 int32_t group_size, int64_t S, int64_t R, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  // the projection's rules (dy stands where its output would)
  w4a16_status st = check_problem(x, wq, scales, zp, nullptr, dy, M, N, K, group_size, dtype);
  if (st != W4A16_OK) return st;
  st = check_adapters("lora_backward", la, lb, ids, alpha, M, N, K, S, R);
  if (st != W4A16_OK) return st;
  if (w4a16::order_places(M, S) * 4 > INT32_MAX)
    return fail(W4A16_ERR_UNSUPPORTED, "lora_backward: too many tokens, got M=%lld", (long long)M);
  if (S > 65535) return fail(W4A16_ERR_UNSUPPORTED, "lora_backward: at most 65535 adapters, got %lld", (long long)S);
  if ((uint64_t)N * (uint64_t)K / 2 > 0xFFFFFFFFull)
    return fail(W4A16_ERR_UNSUPPORTED, "lora_backward: N*K/2 must be below 4 GiB (N=%lld K=%lld)", (long long)N, (long long)K);
  // a tile's 256 rows of dy (of N rounded up to 64) lie below 4 GiB
  if (N > (1 << 23) - 64)
    return fail(W4A16_ERR_UNSUPPORTED, "lora_backward: N above %d is not supported, got %lld", (1 << 23) - 64, (long long)N);
  if (M > 0 && !u) return fail(W4A16_ERR_INVALID_ARG, "lora_backward: u must not be NULL");
  if (!dla || !dlb) return fail(W4A16_ERR_INVALID_ARG, "lora_backward: dla and dlb must not be NULL");
  if ((dy && !aligned(dy, 16)) || (u && !aligned(u, 16)) || (dx && !aligned(dx, 16)) || !aligned(dla, 16) || !aligned(dlb, 16))
    return fail(W4A16_ERR_ALIGNMENT, "lora_backward: dy, u, dx, dla and dlb must be 16-byte aligned");
  const int64_t G = K / group_size;
  const struct { const void* p; size_t n; } out[3] = {{dx, act_bytes(M * K)}, {dla, act_bytes(S * R * K)}, {dlb, act_bytes(S * N * R)}},
      in[6] = {{dy, act_bytes(M * N)}, {x, act_bytes(M * K)}, {u, (size_t)M * R * 4}, {wq, (size_t)N * (K / 8) * 4},
               {scales, act_bytes(N * G)}, {zp, zp ? (size_t)(N / 8) * G * 4 : 0}};
  for (int i = 0; i < 3; ++i) {
    bool bad = overlaps_adapters(out[i].p, out[i].n, la, lb, ids, alpha, M, N, K, S, R);
    for (int j = 0; j < 6; ++j) bad |= overlap(out[i].p, out[i].n, in[j].p, in[j].n);
    for (int j = 0; j < i; ++j) bad |= overlap(out[i].p, out[i].n, out[j].p, out[j].n);
    if (bad) return fail(W4A16_ERR_INVALID_ARG, "lora_backward: dx, dla and dlb must not overlap any input or each other");
  }
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (M == 0) {
    // no tokens: the gradients are zero (S R K and S N R are multiples of 8)
    e = w4a16::launch_zero_words(dla, act_bytes(S * R * K), s);
    if (e == hipSuccess) e = w4a16::launch_zero_words(dlb, act_bytes(S * N * R), s);
    return e == hipSuccess ? ok() : fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  }
  const BackwardPlan p = plan_backward(M, N, K, group_size, S, R, dtype, dev->cu_count);
  if (workspace == nullptr || workspace_bytes < p.bytes)
    return fail(W4A16_ERR_WORKSPACE, "lora_backward: workspace of %zu bytes needed, got %zu%s", p.bytes, workspace_bytes,
                workspace ? "" : " (NULL)");
  if (!aligned(workspace, 256)) return fail(W4A16_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  bool inside = overlaps_adapters(workspace, p.bytes, la, lb, ids, alpha, M, N, K, S, R);
  for (const auto& o : out) inside |= overlap(workspace, p.bytes, o.p, o.n);
  for (const auto& i : in) inside |= overlap(workspace, p.bytes, i.p, i.n);
  if (inside) return fail(W4A16_ERR_INVALID_ARG, "lora_backward: the workspace must not overlap an input or an output");
  if (log_enabled())
    std::fprintf(stderr,
                 "[w4a16] lora_backward M=%lld N=%lld K=%lld g=%d %s %s S=%lld R=%lld dx bm=%d splits=%d sums tokens=%d splits=%d\n",
                 (long long)M, (long long)N, (long long)K, group_size, dtype == W4A16_F16 ? "f16" : "bf16",
                 zp ? "asym" : "sym", (long long)S, (long long)R, dx ? 64 * p.dx.mw : 0, dx ? p.dx.splits : 0,
                 p.outer.tokens, p.outer.splits);
  char* const ws = static_cast<char*>(workspace);
  auto at = [&](size_t o) { return static_cast<void*>(ws + o); };
  const bool pad = p.np != N;
  w4a16::PrepArgs prep;
  prep.ids = ids;
  prep.order = static_cast<int32_t*>(at(p.order));
  prep.start = static_cast<int32_t*>(at(p.start));
  prep.count = static_cast<int32_t*>(at(p.count));
  prep.places = (int)p.places;
  prep.la = static_cast<const uint16_t*>(la);
  prep.lb = static_cast<const uint16_t*>(lb);
  prep.la_t = static_cast<uint16_t*>(at(p.la_t));
  prep.lb_t = static_cast<uint16_t*>(at(p.lb_t));
  prep.dy = static_cast<const uint16_t*>(dy);
  prep.dy_pad = pad ? static_cast<uint16_t*>(at(p.dy_pad)) : nullptr;
  prep.zero = static_cast<uint32_t*>(at(p.zeros));
  prep.zero_words = (int)(p.zero_bytes / 4);
  prep.M = (int)M;
  prep.N = (int)N;
  prep.K = (int)K;
  prep.S = (int)S;
  prep.R = (int)R;
  prep.np = (int)p.np;
  if (dx) {
    prep.dx.wq = reinterpret_cast<const uint32_t*>(wq);
    prep.dx.scales = static_cast<const uint16_t*>(scales);
    prep.dx.zp = reinterpret_cast<const uint32_t*>(zp);
    prep.dx.constants = at(p.constants);
    prep.dx.wq_tail = pad ? static_cast<uint32_t*>(at(p.tail_w)) : nullptr;
    prep.dx.G = (int)G;
    prep.dx.dtype = dtype;
  }
  const uint16_t* const dyr = pad ? prep.dy_pad : prep.dy;
  uint16_t* const g = static_cast<uint16_t*>(at(p.g));
  e = w4a16::launch_prep(prep, s);
  if (e == hipSuccess) {
    // g / alpha = dy . B: the transposed lb in the first factor's place
    const w4a16::ShrinkArgs sa{dyr, prep.lb_t, ids, static_cast<float*>(at(p.part)), nullptr, nullptr, nullptr, nullptr, M, p.np, (int)S, (int)R, dtype};
    e = w4a16::launch_shrink(sa, p.shrink, s);
  }
  uint16_t* const op[2] = {static_cast<uint16_t*>(at(p.op[0])), static_cast<uint16_t*>(at(p.op[1]))};
  int32_t* const g_shift = static_cast<int32_t*>(at(p.g_shift));
  int8_t* const op_shift[2] = {static_cast<int8_t*>(at(p.op_shift[0])), static_cast<int8_t*>(at(p.op_shift[1]))};
  if (e == hipSuccess) {
    const w4a16::OperandArgs pa{static_cast<const float*>(at(p.part)), u, ids, prep.order, alpha, g, {op[0], op[1]}, g_shift,
                                {op_shift[0], op_shift[1]}, (int)M, (int)S, (int)R, p.shrink.splits, (int)p.places, dtype};
    e = w4a16::launch_operands(pa, s);
  }
  if (e == hipSuccess && dx) {
    const w4a16::DxArgs da{dyr, wq, prep.dx.wq_tail, prep.dx.constants, dx, static_cast<float*>(at(p.dx_part)), M, N, K,
                           (int)p.np, group_size, dtype};
    w4a16::LoraTerm t;
    t.ids = ids;
    t.up = prep.la_t;
    t.op = g;
    t.shift = g_shift;
    t.S = (int)S;
    t.R = (int)R;
    e = w4a16::launch_dx(da, p.dx, t, s);
  }
  if (e == hipSuccess) {
    w4a16::OuterArgs oa;
    oa.p[0] = {static_cast<const uint16_t*>(x), op[0], op_shift[0], static_cast<uint16_t*>(dla), (int)K, (int)K, 1};
    oa.p[1] = {dyr, op[1], op_shift[1], static_cast<uint16_t*>(dlb), (int)p.np, (int)N, 0};
    oa.order = prep.order;
    oa.start = prep.start;
    oa.count = prep.count;
    oa.places = (int)p.places;
    oa.partial = static_cast<float*>(at(p.outer_part));
    oa.counters = prep.zero;
    oa.M = (int)M;
    oa.S = (int)S;
    oa.R = (int)R;
    oa.dtype = dtype;
    e = w4a16::launch_outer(oa, p.outer, s);
  }
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

static int elem_bytes(int32_t dtype) { return dtype == W4A16_F32 ? 4 : 2; }

// blocks of a list of tensors and the chunks they are cut into, or -1 where a
// size is out of range
static int64_t adamw_chunks(const w4a16_adamw_tensor* t, int64_t count, int64_t* blocks) {
  *blocks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > (int64_t(1) << 38)) return -1;
    *blocks += (t[i].n + 255) / 256;
    if (*blocks > (int64_t(1) << 40)) return -1;
  }
  const int64_t per = 4 * w4a16::adamw_blocks_per_wave(*blocks);
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += ((t[i].n + 255) / 256 + per - 1) / per;
  return chunks > INT32_MAX ? -1 : chunks;
}

size_t w4a16_adamw_table_size(const w4a16_adamw_tensor* tensors, int64_t count) {
  if (!tensors || count < 1 || count > INT32_MAX) return 0;
  int64_t blocks = 0;
  const int64_t chunks = adamw_chunks(tensors, count, &blocks);
  return chunks < 0 ? 0 : (size_t)count * sizeof(w4a16::AdamwTensor) + (size_t)chunks * sizeof(w4a16::AdamwChunk);
}

w4a16_status w4a16_adamw_table(const w4a16_adamw_tensor* tensors, int64_t count, int32_t state_bits,
                               int32_t param_dtype, int32_t grad_dtype, int32_t copy_dtype, void* table,
                               size_t table_bytes, w4a16_adamw_plan* plan) {
  if (!tensors || !table || !plan || count < 1 || count > INT32_MAX)
    return fail(W4A16_ERR_INVALID_ARG, "adamw_table: need at least one tensor, a table and a plan");
  if (state_bits != 8 && state_bits != 32)
    return fail(W4A16_ERR_INVALID_ARG, "adamw_table: moments are held in 8 or 32 bits, got %d", (int)state_bits);
  if (param_dtype < W4A16_F16 || param_dtype > W4A16_F32 || grad_dtype < W4A16_F16 || grad_dtype > W4A16_F32)
    return fail(W4A16_ERR_INVALID_ARG, "adamw_table: parameters and gradients must be fp16, bf16 or fp32");
  int64_t total = 0;
  const int64_t chunks = adamw_chunks(tensors, count, &total);
  if (chunks < 0) return fail(W4A16_ERR_INVALID_ARG, "adamw_table: a tensor's size is out of range");
  const size_t need = w4a16_adamw_table_size(tensors, count);
  if (table_bytes < need)
    return fail(W4A16_ERR_WORKSPACE, "adamw_table: %zu bytes needed, got %zu", need, table_bytes);
  if (!aligned(table, 8)) return fail(W4A16_ERR_ALIGNMENT, "adamw_table: the table must be 8-byte aligned");
  const int pb = elem_bytes(param_dtype), gb = elem_bytes(grad_dtype), sb = state_bits == 8 ? 1 : 4;
  // first every tensor is checked, then the table is written
  struct Range { uintptr_t begin, end; int64_t tensor; };
  std::vector<Range> ranges;  // that a step writes
  try {
    ranges.reserve((size_t)count * 6);
  } catch (const std::exception&) {
    return fail(W4A16_ERR_UNSUPPORTED, "adamw_table: no host memory to check %lld tensors", (long long)count);
  }
  for (int64_t i = 0; i < count; ++i) {
    const w4a16_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale)))
      return fail(W4A16_ERR_INVALID_ARG, "adamw_table: tensor %lld has a NULL pointer", (long long)i);
    if (t.copy && copy_dtype != W4A16_F16 && copy_dtype != W4A16_BF16)
      return fail(W4A16_ERR_INVALID_ARG, "adamw_table: copies must be fp16 or bf16");
    if (!aligned(t.param, pb) || !aligned(t.grad, gb) || !aligned(t.m, sb) || !aligned(t.v, sb) ||
        (t.copy && !aligned(t.copy, 2)) || (state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
      return fail(W4A16_ERR_ALIGNMENT, "adamw_table: a pointer of tensor %lld is not aligned to its elements", (long long)i);
    const struct { const void* p; size_t n; } own[6] = {
        {t.param, (size_t)t.n * pb}, {t.m, (size_t)t.n * sb}, {t.v, (size_t)t.n * sb},
        {state_bits == 8 ? t.m_scale : nullptr, (size_t)((t.n + 255) / 256) * 4},
        {state_bits == 8 ? t.v_scale : nullptr, (size_t)((t.n + 255) / 256) * 4},
        {t.copy, (size_t)t.n * 2}};
    for (int a = 0; a < 6; ++a) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(own[a].p);
      if (own[a].p) ranges.push_back({at, at + own[a].n, i});
    }
  }
  // no element is written by two of them, none is read as a gradient
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  for (size_t i = 1; i < ranges.size(); ++i)
    if (ranges[i].begin < ranges[i - 1].end)
      return fail(W4A16_ERR_INVALID_ARG, "adamw_table: buffers of tensors %lld and %lld overlap", (long long)ranges[i - 1].tensor,
                  (long long)ranges[i].tensor);
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].n == 0) continue;
    const uintptr_t begin = reinterpret_cast<uintptr_t>(tensors[i].grad), end = begin + (size_t)tensors[i].n * gb;
    const auto r = std::lower_bound(ranges.begin(), ranges.end(), end, [](const Range& a, uintptr_t e) { return a.begin < e; });
    if (r != ranges.begin() && (r - 1)->end > begin)
      return fail(W4A16_ERR_INVALID_ARG, "adamw_table: the gradient of tensor %lld and a buffer of tensor %lld overlap",
                  (long long)i, (long long)(r - 1)->tensor);
  }
  w4a16::AdamwTensor* out = static_cast<w4a16::AdamwTensor*>(table);
  w4a16::AdamwChunk* ch = reinterpret_cast<w4a16::AdamwChunk*>(out + count);
  int64_t first = 0;
  for (int64_t i = 0; i < count; ++i) {
    const w4a16_adamw_tensor& t = tensors[i];
    const bool vec = aligned(t.param, 4 * pb) && aligned(t.grad, 4 * gb) && aligned(t.m, 4 * sb) &&
                     aligned(t.v, 4 * sb) && (!t.copy || aligned(t.copy, 8));
    out[i] = w4a16::AdamwTensor{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n, first, copy_dtype, vec};
    const int64_t blocks = (t.n + 255) / 256;
    for (int64_t b = 0; b < blocks; b += 4 * w4a16::adamw_blocks_per_wave(total)) *ch++ = {(int32_t)i, (int32_t)b};
    first += blocks;
  }
  *plan = w4a16_adamw_plan{count, chunks, first, state_bits, param_dtype, grad_dtype, 0};
  return ok();
}

static w4a16_status check_adamw_plan(const char* what, const void* table, const w4a16_adamw_plan* plan) {
  if (!plan || plan->tensors < 1 || plan->tensors > INT32_MAX || plan->chunks < 0 || plan->chunks > INT32_MAX ||
      (plan->state_bits != 8 && plan->state_bits != 32) || plan->param_dtype < W4A16_F16 || plan->param_dtype > W4A16_F32 ||
      plan->grad_dtype < W4A16_F16 || plan->grad_dtype > W4A16_F32)
    return fail(W4A16_ERR_INVALID_ARG, "%s: not a plan of w4a16_adamw_table", what);
  if (!table) return fail(W4A16_ERR_INVALID_ARG, "%s: the table must not be NULL", what);
  if (!aligned(table, 8)) return fail(W4A16_ERR_ALIGNMENT, "%s: the table must be 8-byte aligned", what);
  return ok();
}

w4a16_status w4a16_adamw_step(const void* table, const w4a16_adamw_plan* plan, double lr, double beta1, double beta2,
                              double eps, double weight_decay, int64_t step, double grad_scale, uint32_t seed,
                              void* stream) {
  w4a16_status st = check_adamw_plan("adamw_step", table, plan);
  if (st != W4A16_OK) return st;
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || step < 1 || !std::isfinite(lr) ||
      !std::isfinite(weight_decay) || !std::isfinite(eps) || !std::isfinite(grad_scale))
    return fail(W4A16_ERR_INVALID_ARG, "adamw_step: need betas in [0, 1), eps >= 0, finite rates and step >= 1");
  if (plan->chunks == 0) return ok();
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  w4a16::AdamwScalars h;
  h.beta1 = (float)beta1;
  h.one_beta1 = (float)(1.0 - beta1);
  h.beta2 = (float)beta2;
  h.one_beta2 = (float)(1.0 - beta2);
  h.eps = (float)eps;
  h.decay = (float)(1.0 - lr * weight_decay);
  h.rate = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  h.root = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  h.grad_scale = (float)grad_scale;
  h.seed = seed * 0x9E3779B9u;
  const hipError_t e = w4a16::launch_adamw(table, (int)plan->tensors, (int)plan->chunks,
                                           w4a16::adamw_blocks_per_wave(plan->blocks), plan->param_dtype,
                                           plan->grad_dtype, plan->state_bits, h, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

w4a16_status w4a16_adamw_moments(const void* table, const w4a16_adamw_plan* plan, float* m, float* v, void* stream) {
  w4a16_status st = check_adamw_plan("adamw_moments", table, plan);
  if (st != W4A16_OK) return st;
  if (plan->state_bits != 8)
    return fail(W4A16_ERR_UNSUPPORTED, "adamw_moments: moments in 32 bits are read where they lie");
  if (plan->chunks == 0) return ok();
  if (!m || !v) return fail(W4A16_ERR_INVALID_ARG, "adamw_moments: m and v must not be NULL");
  if (!aligned(m, 16) || !aligned(v, 16)) return fail(W4A16_ERR_ALIGNMENT, "adamw_moments: m and v must be 16-byte aligned");
  if (overlap(m, (size_t)plan->blocks * 1024, v, (size_t)plan->blocks * 1024))
    return fail(W4A16_ERR_INVALID_ARG, "adamw_moments: m and v must not overlap");
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A16_OK) return st;
  const hipError_t e = w4a16::launch_adamw_moments(table, (int)plan->tensors, (int)plan->chunks,
                                                   w4a16::adamw_blocks_per_wave(plan->blocks), m, v,
                                                   static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

w4a16_status w4a16_unpack_device(const int32_t* wq, uint8_t* q, int64_t N, int64_t K, void* stream) {
  if (N < 0 || K < 0 || K % 8) return fail(W4A16_ERR_INVALID_ARG, "need N >= 0, K >= 0, K %% 8 == 0");
  if (N == 0 || K == 0) return ok();
  if (!wq || !q) return fail(W4A16_ERR_INVALID_ARG, "wq and q must not be NULL");
  if (!aligned(wq, 4) || !aligned(q, 8)) return fail(W4A16_ERR_ALIGNMENT, "wq must be 4-byte and q 8-byte aligned");
  const DeviceInfo* dev = nullptr;
  w4a16_status st = device_info(&dev);
  if (st != W4A16_OK) return st;
  hipError_t e = w4a16::launch_unpack(wq, q, N, K, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W4A16_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
