// AdamW over many tensors in one launch (gfx950), with the moments in 32 bits
// or in 8 bits with one scale per 256 consecutive elements.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in fp32 whatever the tensors' types, without contraction (this file is
// compiled so), so that every operation rounds once and a plain sequence of
// fp32 operations gives the same bits.
//
// 8-bit moments: a code is a power law of the value's share of the largest in
// its block,
//   m = sign(c) (c / 127)^2 ms,  c in -127..127, ms = max |m|
//   v = r^2, r = (c / 255)^2 rs, c in 0..255,    rs = max sqrt(v)
// which needs no table, one square root per code, and gives v ten decades
// with steps of 1.6 % at the top.  Codes are rounded up or down at random
// (code = floor(exact + dither), the dither a hash of the seed and the
// element): with b2 near 1 a step moves v by less than half a code, and
// rounding to nearest would never move it at all.  A v above zero keeps a
// code of at least 1, so no moment is divided by eps alone.
//
// One wave takes one block of 256 elements at a time, four consecutive
// elements a lane, so a block's largest value is a wave reduction and every
// access of a full block is one vector load or store.  The step is bound by
// the memory it moves: 35.7 M elements with 32-bit moments 185 us (5.4 TB/s),
// 143 M with 8-bit moments 440 us (5.2 TB/s) and 248 us for their decoded
// moments; a copy reaches 5.2.  One layer's 0.8 M elements: 6.6 us, latency.
#include "w4a16_adamw.h"
#include "w4a16_device.hpp"
#include "w4a16_internal.h"

namespace w4a16 {

namespace {

// Tensors' pointers come out of the table, so their address space has to be
// said: the accesses would be flat ones, which also wait for LDS.
#define W4A16_GLOBAL __attribute__((address_space(1)))

// four consecutive elements as they lie in memory, and their fp32 values
template <int DT>
struct Quad {
  using raw = u32x2;
  using elem = uint16_t;
  __device__ static f32x4 value(raw q) {
    const uint32_t a = q[0], b = q[1];
    return f32x4{act_to_f32<DT>((uint16_t)a), act_to_f32<DT>((uint16_t)(a >> 16)), act_to_f32<DT>((uint16_t)b),
                 act_to_f32<DT>((uint16_t)(b >> 16))};
  }
  __device__ static raw pack(const f32x4& v) {
    return raw{f32x2_to_act_pair<DT>(v[0], v[1]), f32x2_to_act_pair<DT>(v[2], v[3])};
  }
  __device__ static float one(elem e) { return act_to_f32<DT>(e); }
  __device__ static elem narrow(float v) { return f32_to_act<DT>(v); }
};
template <>
struct Quad<DT_F32> {
  using raw = f32x4;
  using elem = float;
  __device__ static f32x4 value(raw q) { return q; }
  __device__ static raw pack(const f32x4& v) { return v; }
  __device__ static float one(elem e) { return e; }
  __device__ static elem narrow(float v) { return v; }
};

// WHOLE: the quad is inside the tensor and takes one vector access;
// otherwise the first n of its elements, one by one
template <int DT, bool WHOLE>
__device__ __forceinline__ f32x4 load4(const void* p, size_t i, int n) {
  using Q = Quad<DT>;
  if constexpr (WHOLE) {
    return Q::value(((W4A16_GLOBAL const typename Q::raw*)p)[i >> 2]);
  } else {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) v[e] = Q::one(((W4A16_GLOBAL const typename Q::elem*)p)[i + e]);
    return v;
  }
}
template <int DT, bool WHOLE>
__device__ __forceinline__ void store4(void* p, size_t i, int n, const f32x4& v) {
  using Q = Quad<DT>;
  if constexpr (WHOLE) {
    ((W4A16_GLOBAL typename Q::raw*)p)[i >> 2] = Q::pack(v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) ((W4A16_GLOBAL typename Q::elem*)p)[i + e] = Q::narrow(v[e]);
  }
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_codes(const void* p, size_t i, int n) {
  if constexpr (WHOLE) {
    return ((W4A16_GLOBAL const uint32_t*)p)[i >> 2];
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) w |= (uint32_t)((W4A16_GLOBAL const uint8_t*)p)[i + e] << (8 * e);
    return w;
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(void* p, size_t i, int n, uint32_t w) {
  if constexpr (WHOLE) {
    ((W4A16_GLOBAL uint32_t*)p)[i >> 2] = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) ((W4A16_GLOBAL uint8_t*)p)[i + e] = (uint8_t)(w >> (8 * e));
  }
}

__device__ __forceinline__ float decode_m(uint32_t w, int e, float ms) {
  const float c = (float)(int8_t)(w >> (8 * e)) * (float)(1.0 / 127.0);
  return (c * __builtin_fabsf(c)) * ms;
}
__device__ __forceinline__ float decode_r(uint32_t w, int e, float rs) {
  const float c = (float)(uint8_t)(w >> (8 * e)) * (float)(1.0 / 255.0);
  return (c * c) * rs;
}

// The largest of the wave's non-negative values by their bits, which order as
// the values do and put a NaN above them all: four rotations inside the
// 16-lane rows, then the rows.
template <int CTRL>
__device__ __forceinline__ uint32_t rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ float wave_max(uint32_t v) {
  v = max(v, rotate<0x128>(v));
  v = max(v, rotate<0x124>(v));
  v = max(v, rotate<0x122>(v));
  v = max(v, rotate<0x121>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max((uint32_t)b[0], (uint32_t)b[1]);
  return __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// a published 32-bit integer finaliser (shift, exclusive or, multiply; the
// "lowbias32" constants of C. Wellons' hash prospector)
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// Square root of 2^-100 <= x <= 2^100, rounded to nearest: the hardware's
// reciprocal square root, then one Newton step whose residual x - s^2 is exact
// in one fma.  (Compared with the compiler's correctly rounded one for every
// fp32 value of the range: equal.  It takes 9 issue slots where that one, for
// all of fp32, takes 17, three times an element: 143 M elements with bf16
// gradients and copies 610 us with that one, 545 us so.  The update's quotient
// stays a division: m times the hardware's reciprocal takes 520 us there, and
// nothing less in a step without copies, but p would no longer be the plain
// sequence's.)
__device__ __forceinline__ float sqrt_mid(float x) {
  const float r = __builtin_amdgcn_rsqf(x), s = x * r;
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * r, s);
}
// the same for 0 <= x <= 2^100 where only (a multiple of it plus a dither)'s
// whole part counts: below 2^-100 as good as zero
__device__ __forceinline__ float sqrt_code(float x) { return x >= 0x1p-100f ? sqrt_mid(x) : 0.f; }

// the chunk of this workgroup: its tensor and its first block there
__device__ __forceinline__ AdamwChunk chunk_of(const void* table, int tensors) {
  const AdamwChunk* c = reinterpret_cast<const AdamwChunk*>(static_cast<const AdamwTensor*>(table) + tensors);
  return c[blockIdx.x];
}

// one lane's quad of a block, before and after the step
template <bool EIGHT>
struct State {
  f32x4 p, g, m, v;
  uint32_t cm, cv;  // 8 bits: codes, and the block's scales
  float ms, rs;
};

template <int PD, int GD, bool EIGHT, bool WHOLE>
__device__ __forceinline__ void load_state(const AdamwTensor& t, int64_t b, int lane, int n, State<EIGHT>& s) {
  const size_t i = (size_t)b * 256 + 4 * lane;
  s.p = load4<PD, WHOLE>(t.param, i, n);
  s.g = load4<GD, WHOLE>(t.grad, i, n);
  if constexpr (EIGHT) {
    s.cm = load_codes<WHOLE>(t.m, i, n);
    s.cv = load_codes<WHOLE>(t.v, i, n);
    s.ms = ((W4A16_GLOBAL const float*)t.m_scale)[b];
    s.rs = ((W4A16_GLOBAL const float*)t.v_scale)[b];
  } else {
    s.m = load4<DT_F32, WHOLE>(t.m, i, n);
    s.v = load4<DT_F32, WHOLE>(t.v, i, n);
  }
}

template <int PD, bool EIGHT, bool WHOLE>
__device__ __forceinline__ void step_and_store(const AdamwTensor& t, int64_t b, int lane, int n, const AdamwScalars& h,
                                               State<EIGHT>& s) {
  const size_t i = (size_t)b * 256 + 4 * lane;
  float r[4];
  uint32_t far = 0;  // how far v's bits lie above those of 2^-100 (wrapping below it)
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (EIGHT) {
      s.m[e] = decode_m(s.cm, e, s.ms);
      r[e] = decode_r(s.cv, e, s.rs);
      s.v[e] = r[e] * r[e];
    }
    const float g = s.g[e] * h.grad_scale;
    s.m[e] = s.m[e] * h.beta1 + g * h.one_beta1;
    s.v[e] = s.v[e] * h.beta2 + (g * g) * h.one_beta2;
    const float v = s.v[e];
    far = max(far, __builtin_bit_cast(uint32_t, v) - __builtin_bit_cast(uint32_t, 0x1p-100f));
  }
  // 8 bits: the short square root where every v of the wave is in its range (no
  // zeros, infinities or NaN); the bits are the same either way
  constexpr uint32_t span = __builtin_bit_cast(uint32_t, 0x1p100f) - __builtin_bit_cast(uint32_t, 0x1p-100f);
  if (EIGHT && __all(far <= span)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = sqrt_mid(s.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __builtin_sqrtf(s.v[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s.p[e] = s.p[e] * h.decay - (s.m[e] / (r[e] * h.root + h.eps)) * h.rate;
  store4<PD, WHOLE>(t.param, i, n, s.p);
  if (t.copy) {
    if (t.copy_dtype == DT_F16)
      store4<DT_F16, WHOLE>(t.copy, i, n, s.p);
    else
      store4<DT_BF16, WHOLE>(t.copy, i, n, s.p);
  }
  if constexpr (EIGHT) {
    uint32_t am = 0, ar = 0;  // elements past the tensor's end are zero
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      am = max(am, __builtin_bit_cast(uint32_t, __builtin_fabsf(s.m[e])));
      ar = max(ar, __builtin_bit_cast(uint32_t, __builtin_fabsf(r[e])));
    }
    const float ms = wave_max(am), rs = wave_max(ar);
    const float im = ms > 0x1p-100f ? 1.f / ms : 0.f, ir = rs > 0x1p-100f ? 1.f / rs : 0.f;
    uint32_t cm = 0, cv = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t d = mix32((uint32_t)((t.first_block + b) * 256 + 4 * lane + e) + h.seed);
      const float qm = __builtin_floorf(sqrt_code(__builtin_fabsf(s.m[e]) * im) * 127.f + (float)(d & 0xFFFFu) * 0x1p-16f);
      const float qv = __builtin_floorf(sqrt_code(r[e] * ir) * 255.f + (float)(d >> 16) * 0x1p-16f);
      const int c = (int)__builtin_fminf(qm, 127.f);
      const int u = (int)__builtin_fminf(r[e] > 0.f ? __builtin_fmaxf(qv, 1.f) : qv, 255.f);
      cm |= (uint32_t)(uint8_t)(s.m[e] < 0.f ? -c : c) << (8 * e);
      cv |= (uint32_t)(uint8_t)u << (8 * e);
    }
    store_codes<WHOLE>(t.m, i, n, cm);
    store_codes<WHOLE>(t.v, i, n, cv);
    if (lane == 0) {
      ((W4A16_GLOBAL float*)t.m_scale)[b] = ms;
      ((W4A16_GLOBAL float*)t.v_scale)[b] = rs;
    }
  } else {
    store4<DT_F32, WHOLE>(t.m, i, n, s.m);
    store4<DT_F32, WHOLE>(t.v, i, n, s.v);
  }
}

// BPW blocks a wave: one in small tables, so that they fill the CUs, four in
// large ones, whose loads are all issued before the first step.
template <int PD, int GD, bool EIGHT, int BPW>
__global__ __launch_bounds__(256) void adamw_kernel(const void* __restrict__ table, int tensors, const AdamwScalars h) {
  const AdamwChunk ch = chunk_of(table, tensors);
  const AdamwTensor t = static_cast<const AdamwTensor*>(table)[ch.tensor];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t.vec && ((int64_t)ch.block + 4 * BPW) * 256 <= t.n) {
    State<EIGHT> s[BPW];
#pragma unroll
    for (int k = 0; k < BPW; ++k) load_state<PD, GD, EIGHT, true>(t, ch.block + wave + 4 * k, lane, 4, s[k]);
#pragma unroll
    for (int k = 0; k < BPW; ++k) step_and_store<PD, EIGHT, true>(t, ch.block + wave + 4 * k, lane, 4, h, s[k]);
    return;
  }
  for (int k = 0; k < BPW; ++k) {
    const int64_t b = ch.block + wave + 4 * k;
    const int64_t left = t.n - b * 256;  // elements from this block on
    if (left <= 0) return;
    const int n = (int)min((int64_t)4, max((int64_t)0, left - 4 * lane));
    State<EIGHT> s;
    load_state<PD, GD, EIGHT, false>(t, b, lane, n, s);
    step_and_store<PD, EIGHT, false>(t, b, lane, n, h, s);
  }
}

// the moments the codes stand for, blocks in the table's order, zero past a tensor's end
template <int BPW>
__global__ __launch_bounds__(256) void moments_kernel(const void* __restrict__ table, int tensors, float* __restrict__ mo,
                                                      float* __restrict__ vo) {
  const AdamwChunk ch = chunk_of(table, tensors);
  const AdamwTensor t = static_cast<const AdamwTensor*>(table)[ch.tensor];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto block = [&](int64_t b, int n, uint32_t cm, uint32_t cv, float ms, float rs) {
    f32x4 m, v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = e < n ? decode_m(cm, e, ms) : 0.f;
      const float r = decode_r(cv, e, rs);
      v[e] = e < n ? r * r : 0.f;
    }
    const size_t o = ((size_t)(t.first_block + b) * 256 + 4 * lane) >> 2;
    reinterpret_cast<f32x4*>(mo)[o] = m;
    reinterpret_cast<f32x4*>(vo)[o] = v;
  };
  auto scale = [&](const float* p, int64_t b) { return ((W4A16_GLOBAL const float*)p)[b]; };
  if (t.vec && ((int64_t)ch.block + 4 * BPW) * 256 <= t.n) {
    uint32_t cm[BPW], cv[BPW];
    float ms[BPW], rs[BPW];
#pragma unroll
    for (int k = 0; k < BPW; ++k) {
      const int64_t b = ch.block + wave + 4 * k;
      cm[k] = load_codes<true>(t.m, (size_t)b * 256 + 4 * lane, 4);
      cv[k] = load_codes<true>(t.v, (size_t)b * 256 + 4 * lane, 4);
      ms[k] = scale(t.m_scale, b);
      rs[k] = scale(t.v_scale, b);
    }
#pragma unroll
    for (int k = 0; k < BPW; ++k) block(ch.block + wave + 4 * k, 4, cm[k], cv[k], ms[k], rs[k]);
    return;
  }
  for (int k = 0; k < BPW; ++k) {
    const int64_t b = ch.block + wave + 4 * k;
    const int64_t left = t.n - b * 256;
    if (left <= 0) return;
    const size_t i = (size_t)b * 256 + 4 * lane;
    const int n = (int)min((int64_t)4, max((int64_t)0, left - 4 * lane));
    block(b, n, load_codes<false>(t.m, i, n), load_codes<false>(t.v, i, n), scale(t.m_scale, b), scale(t.v_scale, b));
  }
}

template <int PD, int GD, bool EIGHT>
hipError_t launch_bpw(const void* table, int tensors, int chunks, int bpw, const AdamwScalars& h, hipStream_t s) {
  if (bpw == 1)
    hipLaunchKernelGGL((adamw_kernel<PD, GD, EIGHT, 1>), dim3(chunks), dim3(256), 0, s, table, tensors, h);
  else
    hipLaunchKernelGGL((adamw_kernel<PD, GD, EIGHT, 4>), dim3(chunks), dim3(256), 0, s, table, tensors, h);
  return hipGetLastError();
}
template <int PD, int GD>
hipError_t launch_bits(const void* table, int tensors, int chunks, int bpw, int bits, const AdamwScalars& h, hipStream_t s) {
  return bits == 8 ? launch_bpw<PD, GD, true>(table, tensors, chunks, bpw, h, s)
                   : launch_bpw<PD, GD, false>(table, tensors, chunks, bpw, h, s);
}
template <int PD>
hipError_t launch_grad(const void* table, int tensors, int chunks, int bpw, int gd, int bits, const AdamwScalars& h,
                       hipStream_t s) {
  switch (gd) {
    case DT_F16: return launch_bits<PD, DT_F16>(table, tensors, chunks, bpw, bits, h, s);
    case DT_BF16: return launch_bits<PD, DT_BF16>(table, tensors, chunks, bpw, bits, h, s);
    default: return launch_bits<PD, DT_F32>(table, tensors, chunks, bpw, bits, h, s);
  }
}

}  // namespace

hipError_t launch_adamw(const void* table, int tensors, int chunks, int blocks_per_wave, int param_dtype, int grad_dtype,
                        int bits, const AdamwScalars& h, hipStream_t s) {
  switch (param_dtype) {
    case DT_F16: return launch_grad<DT_F16>(table, tensors, chunks, blocks_per_wave, grad_dtype, bits, h, s);
    case DT_BF16: return launch_grad<DT_BF16>(table, tensors, chunks, blocks_per_wave, grad_dtype, bits, h, s);
    default: return launch_grad<DT_F32>(table, tensors, chunks, blocks_per_wave, grad_dtype, bits, h, s);
  }
}

hipError_t launch_adamw_moments(const void* table, int tensors, int chunks, int blocks_per_wave, float* m, float* v,
                                hipStream_t s) {
  if (blocks_per_wave == 1)
    hipLaunchKernelGGL(moments_kernel<1>, dim3(chunks), dim3(256), 0, s, table, tensors, m, v);
  else
    hipLaunchKernelGGL(moments_kernel<4>, dim3(chunks), dim3(256), 0, s, table, tensors, m, v);
  return hipGetLastError();
}

}  // namespace w4a16
