// What the linear kernels do with a sum before it is stored (see nvfp4_linear):
// bias, pre-activation output, activation, residual, one rounding.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"

namespace nvfp4 {

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }

// act(z) of the activations with one argument.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case kActSilu: return silu(z);
    case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case kActGeluTanh: return 0.5f * z * (1.f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

// min and max that keep a NaN, as a comparison with a bound does.
__device__ __forceinline__ float at_most(float z, float bound) { return z > bound ? bound : z; }
__device__ __forceinline__ float at_least(float z, float bound) { return z < bound ? bound : z; }

// Eight consecutive values of a 16-bit or FP32 row.
__device__ __forceinline__ void load8(const void* p, int64_t at, int type, float (&f)[8]) {
  if (type == kTypeF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    return;
  }
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == kTypeBf16) {
      f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
    } else {
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = d.x, f[2 * i + 1] = d.y;
    }
  }
}
__device__ __forceinline__ void store8(void* p, int64_t at, int type, const float (&f)[8]) {
  if (type == kTypeF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
    return;
  }
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == kTypeBf16) {
      u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
}

// The bias of eight columns (and, for SwiGLU, of their up columns) of group g.
__device__ __forceinline__ void load_bias(const LinearEpilogue& p, int g, int col, float (&b)[8], float (&bu)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = bu[i] = 0.f;
  if (!p.bias) return;
  const int64_t at = (int64_t)g * p.wide + col;
  load8(p.bias, at, p.bias_type, b);
  if (p.act == kActSwiglu) load8(p.bias, at + p.N, p.bias_type, bu);
}

// Columns col .. col + 7 of an output row from their sums z (SwiGLU: the gate's, and the up's u).
__device__ __forceinline__ void finish8(const LinearEpilogue& p, int64_t row, int col, float (&z)[8], float (&u)[8],
                                        const float (&b)[8], const float (&bu)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
  if (p.act == kActSwiglu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] += bu[i];
  }
  if (p.preact) {
    store8(p.preact, row * p.ld_preact + col, p.type, z);
    if (p.act == kActSwiglu) store8(p.preact, row * p.ld_preact + p.N + col, p.type, u);
  }
  if (p.act == kActSwiglu) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      z[i] = silu(at_most(z[i], p.gate_limit)) * at_least(at_most(u[i], p.up_limit), -p.up_limit);
  } else if (p.act != kActNone) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = activate(p.act, z[i]);
  }
  if (p.residual) {
    float r[8];
    load8(p.residual, row * p.ld_residual + col, p.type, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
  store8(p.out, row * p.ld_out + col, p.out_type, z);
}

}  // namespace nvfp4
