// What the linear kernels do with a sum before it is stored (see nvfp4_linear):
// bias, pre-activation output, activation, residual, one rounding.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

// 1 / (1 + exp(-z)) by an exponential in (0, 1] and the reciprocal of a number in
// (1, 2].  __expf(-|z|) is within 2 + 1.18 |z| units in the last place (CUDA's bound),
// the reciprocal within one: below an absolute 2^-21 everywhere, but relative to a result
// near 0 the error grows with |z| (2^-19 at z = -6, 2^-16 at -87: less than the rounding to
// 16 bits, which FP32 outputs and bias sums do not have).  An accurate expf and a division
// take z / (1 + expf(-z))
// to the slow path of the division for far negative z (8192 x 4096 x 4096 with silu 243
// us instead of 160), and a gradient's pass over dy and z to its arithmetic.
__device__ __forceinline__ float sigmoid(float z) {
  const float e = __expf(-fabsf(z));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (z < 0.f ? e : 1.f) * r;
}
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }

// act(z) of the activations with one argument.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case kActSilu: return silu(z);
    case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case kActGeluTanh: return z * sigmoid(1.59576912f * (z + 0.044715f * z * z * z));  // (1 + tanh a) / 2 = sigmoid 2a
    default: return z;
  }
}

// min and max that keep a NaN.
__device__ __forceinline__ float at_most(float z, float bound) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(bound));
  return r;
}
__device__ __forceinline__ float at_least(float z, float bound) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(bound));
  return r;
}

__device__ __forceinline__ float swiglu(float g, float u, float gate_limit, float up_limit) {
  return silu(at_most(g, gate_limit)) * at_least(at_most(u, up_limit), -up_limit);
}

// Two 16-bit values of one word.
__device__ __forceinline__ void unpack2(int type, uint32_t v, float& a, float& b) {
  if (type == kTypeBf16) {
    a = bf16_lo(v), b = bf16_hi(v);
  } else {
    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&v));
    a = d.x, b = d.y;
  }
}
__device__ __forceinline__ uint32_t pack2(int type, float a, float b) {
  if (type == kTypeBf16) return pack_bf16x2(a, b);
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// W consecutive values of a row (8, 16 or 32), of which `left` exist (a multiple of 8);
// v8: the addresses are multiples of 32 bytes, and whole sectors are moved (eight 16-bit
// values, half a sector, by 16 bytes all the same).
template <int WORDS>
__device__ __forceinline__ void load_row(const void* p, bool v8, int left, uint32_t (&u)[WORDS]) {
  const uint32_t* q = static_cast<const uint32_t*>(p);
  if (WORDS % 8 == 0 && v8 && left >= 2 * WORDS) {
#pragma unroll
    for (int i = 0; i + 8 <= WORDS; i += 8)
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3]), "=r"(u[i + 4]), "=r"(u[i + 5]),
                     "=r"(u[i + 6]), "=r"(u[i + 7])
                   : "l"(q + i));
    return;
  }
#pragma unroll
  for (int i = 0; i < WORDS; i += 4) {
    const uint4 v = 2 * i < left ? *reinterpret_cast<const uint4*>(q + i) : make_uint4(0, 0, 0, 0);
    u[i] = v.x, u[i + 1] = v.y, u[i + 2] = v.z, u[i + 3] = v.w;
  }
}
template <int W>
__device__ __forceinline__ void add_row(int type, const uint32_t (&r)[W / 2], float (&z)[W]) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    float a, b;
    unpack2(type, r[i], a, b);
    z[2 * i] += a, z[2 * i + 1] += b;
  }
}
template <int W, int WORDS>
__device__ __forceinline__ void store_words(void* p, bool v8, int left, const uint32_t (&u)[WORDS]) {
  uint32_t* q = static_cast<uint32_t*>(p);
  if (WORDS % 8 == 0 && v8 && left >= W) {
#pragma unroll
    for (int i = 0; i + 8 <= WORDS; i += 8)
      st_global_v8(q + i, u[i], u[i + 1], u[i + 2], u[i + 3], u[i + 4], u[i + 5], u[i + 6], u[i + 7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < WORDS; i += 4)
    if (i * W / WORDS < left) *reinterpret_cast<uint4*>(q + i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
}
template <int W>
__device__ __forceinline__ void pack_row(int type, const float (&f)[W], uint32_t (&u)[W / 2]) {
  if (type == kTypeBf16) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pack2(kTypeBf16, f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pack2(kTypeF16, f[2 * i], f[2 * i + 1]);
  }
}
template <int W>
__device__ __forceinline__ void store_row(void* p, int type, bool v8, int left, const float (&f)[W]) {
  if (type == kTypeF32) {
    uint32_t u[W];
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = __float_as_uint(f[i]);
    store_words<W>(p, v8, left, u);
    return;
  }
  uint32_t u[W / 2];
  pack_row(type, f, u);
  store_words<W>(p, v8, left, u);
}

template <int ACT, int N>
__device__ __forceinline__ void activate_as(float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = activate(ACT, z[i]);
}
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&z)[N]) {
  switch (act) {
    case kActRelu: return activate_as<kActRelu>(z);
    case kActSilu: return activate_as<kActSilu>(z);
    case kActGelu: return activate_as<kActGelu>(z);
    case kActGeluTanh: return activate_as<kActGeluTanh>(z);
  }
}

// N (4 or 8) consecutive values of a 16-bit or FP32 row.
template <int N>
__device__ __forceinline__ void load_cols(const void* p, int64_t at, int type, float (&f)[N]) {
  if (type == kTypeF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = q[i];
      f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
    return;
  }
  const uint2* q = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
  uint32_t u[N / 2];
  if constexpr (N == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(q);
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  } else {
    const uint2 v = *q;
    u[0] = v.x, u[1] = v.y;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) unpack2(type, u[i], f[2 * i], f[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void store_cols(void* p, int64_t at, int type, const float (&f)[N]) {
  if (type == kTypeF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    return;
  }
  uint16_t* q = static_cast<uint16_t*>(p) + at;
  uint32_t u[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) u[i] = pack2(type, f[2 * i], f[2 * i + 1]);
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(q) = make_uint4(u[0], u[1], u[2], u[3]);
  else
    *reinterpret_cast<uint2*>(q) = make_uint2(u[0], u[1]);
}

// What an epilogue's code has to know of the activation: a kernel that is compiled for
// one kind holds only that code.
enum LinearEpi { kEpiPlain, kEpiActivation, kEpiSwiglu, kEpiAny };

template <int EPI>
__device__ __forceinline__ bool is_swiglu(const LinearEpilogue& p) {
  return EPI == kEpiSwiglu || (EPI == kEpiAny && p.act == kActSwiglu);
}

// The bias of N columns (and, for SwiGLU, of their up columns) of group g, and their
// residual: zeros where there is none.
template <int EPI, int N>
__device__ __forceinline__ void load_bias(const LinearEpilogue& p, int g, int col, float (&b)[N], float (&bu)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = bu[i] = 0.f;
  if (!p.bias || col >= p.N) return;
  const int64_t at = (int64_t)g * p.wide + col;
  load_cols<N>(p.bias, at, p.bias_type, b);
  if (is_swiglu<EPI>(p)) load_cols<N>(p.bias, at + p.N, p.bias_type, bu);
}
template <int N>
__device__ __forceinline__ void load_residual(const LinearEpilogue& p, int64_t row, int col, float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = 0.f;
  if (p.residual) load_cols<N>(p.residual, row * p.ld_residual + col, p.type, r);
}

// Columns col .. col + N - 1 of an output row from their sums z (SwiGLU: the gate's, and
// the up's u), bias and residual.
template <int EPI, int N>
__device__ __forceinline__ void finish(const LinearEpilogue& p, int64_t row, int col, float (&z)[N], float (&u)[N],
                                       const float (&b)[N], const float (&bu)[N], const float (&r)[N]) {
  const bool pairs = is_swiglu<EPI>(p);
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += b[i], u[i] += bu[i];
  }
  if (p.preact) {
    store_cols<N>(p.preact, row * p.ld_preact + col, p.type, z);
    if (pairs) store_cols<N>(p.preact, row * p.ld_preact + p.N + col, p.type, u);
  }
  if (pairs) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = swiglu(z[i], u[i], p.gate_limit, p.up_limit);
  } else if (EPI != kEpiPlain) {
    activate_all(p.act, z);
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += r[i];
  }
  store_cols<N>(p.out, row * p.ld_out + col, p.out_type, z);
}

}  // namespace nvfp4
