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
// the memory it moves.
#include "w4a16_adamw.h"
#include "w4a16_device.hpp"
#include "w4a16_internal.h"

namespace w4a16 {

namespace {

constexpr int kBlocksPerWave = kAdamwChunkBlocks / 4;

// four consecutive elements as they lie in memory, and their fp32 values
template <int DT>
struct Quad {
  using raw = u32x2;
  __device__ static f32x4 value(const raw& q) {
    return f32x4{act_to_f32<DT>((uint16_t)q[0]), act_to_f32<DT>((uint16_t)(q[0] >> 16)),
                 act_to_f32<DT>((uint16_t)q[1]), act_to_f32<DT>((uint16_t)(q[1] >> 16))};
  }
  __device__ static raw pack(const f32x4& v) {
    return raw{f32x2_to_act_pair<DT>(v[0], v[1]), f32x2_to_act_pair<DT>(v[2], v[3])};
  }
  __device__ static float one(const void* p, size_t i) { return act_to_f32<DT>(static_cast<const uint16_t*>(p)[i]); }
  __device__ static void put(void* p, size_t i, float v) { static_cast<uint16_t*>(p)[i] = f32_to_act<DT>(v); }
};
template <>
struct Quad<DT_F32> {
  using raw = f32x4;
  __device__ static f32x4 value(const raw& q) { return q; }
  __device__ static raw pack(const f32x4& v) { return v; }
  __device__ static float one(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }
  __device__ static void put(void* p, size_t i, float v) { static_cast<float*>(p)[i] = v; }
};

// n valid elements from i on (4: a whole quad); `vec`: the tensor takes vector accesses
template <int DT>
__device__ __forceinline__ f32x4 load4(const void* p, size_t i, int n, bool vec) {
  using Q = Quad<DT>;
  if (vec && n == 4) return Q::value(reinterpret_cast<const typename Q::raw*>(p)[i >> 2]);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) v[e] = Q::one(p, i + e);
  return v;
}
template <int DT>
__device__ __forceinline__ void store4(void* p, size_t i, int n, bool vec, const f32x4& v) {
  using Q = Quad<DT>;
  if (vec && n == 4) {
    reinterpret_cast<typename Q::raw*>(p)[i >> 2] = Q::pack(v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) Q::put(p, i + e, v[e]);
}
__device__ __forceinline__ uint32_t load_codes(const void* p, size_t i, int n, bool vec) {
  if (vec && n == 4) return static_cast<const uint32_t*>(p)[i >> 2];
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) w |= (uint32_t)static_cast<const uint8_t*>(p)[i + e] << (8 * e);
  return w;
}
__device__ __forceinline__ void store_codes(void* p, size_t i, int n, bool vec, uint32_t w) {
  if (vec && n == 4) {
    static_cast<uint32_t*>(p)[i >> 2] = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) static_cast<uint8_t*>(p)[i + e] = (uint8_t)(w >> (8 * e));
}

__device__ __forceinline__ float decode_m(uint32_t w, int e, float ms) {
  const float c = (float)(int8_t)(w >> (8 * e)) * (float)(1.0 / 127.0);
  return (c * __builtin_fabsf(c)) * ms;
}
__device__ __forceinline__ float decode_r(uint32_t w, int e, float rs) {
  const float c = (float)(uint8_t)(w >> (8 * e)) * (float)(1.0 / 255.0);
  return (c * c) * rs;
}

// the largest of the wave's values, NaN if one of them is
__device__ __forceinline__ float wave_max(float v) {
  const bool nan = __any(v != v);
#pragma unroll
  for (int d = 32; d; d >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d));
  return nan ? __builtin_nanf("") : v;
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

// the chunk of this workgroup: its tensor and its first block there
__device__ __forceinline__ AdamwChunk chunk_of(const void* table, int tensors) {
  const AdamwChunk* c = reinterpret_cast<const AdamwChunk*>(static_cast<const AdamwTensor*>(table) + tensors);
  return c[blockIdx.x];
}

template <int PD, int GD, bool EIGHT>
__global__ __launch_bounds__(256) void adamw_kernel(const void* __restrict__ table, int tensors, AdamwScalars h) {
  const AdamwChunk ch = chunk_of(table, tensors);
  const AdamwTensor t = static_cast<const AdamwTensor*>(table)[ch.tensor];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool vec = t.vec != 0;
#pragma unroll
  for (int k = 0; k < kBlocksPerWave; ++k) {
    const int64_t b = ch.block + wave + 4 * k;
    const int64_t left = t.n - b * 256;  // elements from this block on
    if (left <= 0) return;
    const size_t i = (size_t)b * 256 + 4 * lane;
    const int n = (int)min((int64_t)4, max((int64_t)0, left - 4 * lane));
    f32x4 p = load4<PD>(t.param, i, n, vec);
    const f32x4 g = load4<GD>(t.grad, i, n, vec);
    f32x4 m, v, r;
    if constexpr (EIGHT) {
      const uint32_t cm = load_codes(t.m, i, n, vec), cv = load_codes(t.v, i, n, vec);
      const float ms = t.m_scale[b], rs = t.v_scale[b];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = decode_m(cm, e, ms);
        r[e] = decode_r(cv, e, rs);
        v[e] = r[e] * r[e];
      }
    } else {
      m = load4<DT_F32>(t.m, i, n, vec);
      v = load4<DT_F32>(t.v, i, n, vec);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ge = g[e] * h.grad_scale;
      m[e] = m[e] * h.beta1 + ge * h.one_beta1;
      v[e] = v[e] * h.beta2 + (ge * ge) * h.one_beta2;
      r[e] = __builtin_sqrtf(v[e]);
      p[e] = p[e] * h.decay - (m[e] / (r[e] * h.root + h.eps)) * h.rate;
    }
    store4<PD>(t.param, i, n, vec, p);
    if (t.copy) {
      if (t.copy_dtype == DT_F16)
        store4<DT_F16>(t.copy, i, n, vec, p);
      else
        store4<DT_BF16>(t.copy, i, n, vec, p);
    }
    if constexpr (EIGHT) {
      float am = 0.f, ar = 0.f;  // elements past the tensor's end are zero
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_fabsf(m[e]);
        am = am != am || x != x ? __builtin_nanf("") : __builtin_fmaxf(am, x);
        ar = ar != ar || r[e] != r[e] ? __builtin_nanf("") : __builtin_fmaxf(ar, r[e]);
      }
      const float ms = wave_max(am), rs = wave_max(ar);
      const float im = ms > 0x1p-100f ? 1.f / ms : 0.f, ir = rs > 0x1p-100f ? 1.f / rs : 0.f;
      uint32_t cm = 0, cv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t d = mix32((uint32_t)((t.first_block + b) * 256 + 4 * lane + e) + h.seed);
        const float qm = __builtin_floorf(__builtin_sqrtf(__builtin_fabsf(m[e]) * im) * 127.f + (float)(d & 0xFFFFu) * 0x1p-16f);
        const float qv = __builtin_floorf(__builtin_sqrtf(r[e] * ir) * 255.f + (float)(d >> 16) * 0x1p-16f);
        const int c = (int)__builtin_fminf(qm, 127.f);
        const int u = (int)__builtin_fminf(r[e] > 0.f ? __builtin_fmaxf(qv, 1.f) : qv, 255.f);
        cm |= (uint32_t)(uint8_t)(m[e] < 0.f ? -c : c) << (8 * e);
        cv |= (uint32_t)(uint8_t)u << (8 * e);
      }
      store_codes(t.m, i, n, vec, cm);
      store_codes(t.v, i, n, vec, cv);
      if (lane == 0) {
        t.m_scale[b] = ms;
        t.v_scale[b] = rs;
      }
    } else {
      store4<DT_F32>(t.m, i, n, vec, m);
      store4<DT_F32>(t.v, i, n, vec, v);
    }
  }
}

// the moments the codes stand for, blocks in the table's order, zero past a tensor's end
__global__ __launch_bounds__(256) void moments_kernel(const void* __restrict__ table, int tensors, float* __restrict__ mo,
                                                      float* __restrict__ vo) {
  const AdamwChunk ch = chunk_of(table, tensors);
  const AdamwTensor t = static_cast<const AdamwTensor*>(table)[ch.tensor];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool vec = t.vec != 0;
#pragma unroll
  for (int k = 0; k < kBlocksPerWave; ++k) {
    const int64_t b = ch.block + wave + 4 * k;
    const int64_t left = t.n - b * 256;
    if (left <= 0) return;
    const size_t i = (size_t)b * 256 + 4 * lane;
    const int n = (int)min((int64_t)4, max((int64_t)0, left - 4 * lane));
    const uint32_t cm = load_codes(t.m, i, n, vec), cv = load_codes(t.v, i, n, vec);
    const float ms = t.m_scale[b], rs = t.v_scale[b];
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
  }
}

template <int PD, int GD>
hipError_t launch_bits(const void* table, int tensors, int chunks, int bits, const AdamwScalars& h, hipStream_t s) {
  if (bits == 8)
    hipLaunchKernelGGL((adamw_kernel<PD, GD, true>), dim3(chunks), dim3(256), 0, s, table, tensors, h);
  else
    hipLaunchKernelGGL((adamw_kernel<PD, GD, false>), dim3(chunks), dim3(256), 0, s, table, tensors, h);
  return hipGetLastError();
}
template <int PD>
hipError_t launch_grad(const void* table, int tensors, int chunks, int gd, int bits, const AdamwScalars& h, hipStream_t s) {
  switch (gd) {
    case DT_F16: return launch_bits<PD, DT_F16>(table, tensors, chunks, bits, h, s);
    case DT_BF16: return launch_bits<PD, DT_BF16>(table, tensors, chunks, bits, h, s);
    default: return launch_bits<PD, DT_F32>(table, tensors, chunks, bits, h, s);
  }
}

}  // namespace

hipError_t launch_adamw(const void* table, int tensors, int chunks, int param_dtype, int grad_dtype, int bits,
                        const AdamwScalars& h, hipStream_t s) {
  switch (param_dtype) {
    case DT_F16: return launch_grad<DT_F16>(table, tensors, chunks, grad_dtype, bits, h, s);
    case DT_BF16: return launch_grad<DT_BF16>(table, tensors, chunks, grad_dtype, bits, h, s);
    default: return launch_grad<DT_F32>(table, tensors, chunks, grad_dtype, bits, h, s);
  }
}

hipError_t launch_adamw_moments(const void* table, int tensors, int chunks, float* m, float* v, hipStream_t s) {
  hipLaunchKernelGGL(moments_kernel, dim3(chunks), dim3(256), 0, s, table, tensors, m, v);
  return hipGetLastError();
}

}  // namespace w4a16
