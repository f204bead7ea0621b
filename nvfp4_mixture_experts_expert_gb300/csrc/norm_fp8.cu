// Residual addition, RMSNorm and FP8 quantization of hidden states in one pass.
//
//   s = x + residual                       (FP32; bf16(s) is the next residual)
//   y = s * rsqrt(mean(s^2) + eps) * w     (FP32; bf16(y) is the normed output)
//   per block of 128 columns of a row:
//     scale = max(max|y|, 2^-40) / 448,  q = E4M3(y / scale)       (both quotients in FP32)
//
// s and y stay in FP32 registers; every output is rounded once.  The floor of
// 2^-40 keeps the scale of an all-zero block finite (its codes are 0).  A NaN
// in a row makes the whole row NaN (scales included), and so does a mean square
// of 0 without eps.
//
// Bound: HBM.  A row is read once and its outputs written once, 9 bytes an
// element with every output.  8192 x 4096 (302 MB, 44.5 us at the 6.79 TB/s of a
// copy) takes 45.0 us in a graph of calls, 1 x 4096 2.1, 1001 x 3584 with FP32
// weights 6.5, 2048 x 7168 20.7 (132 MB: 19.5).  What made the difference, at the
// time: the norm weight is loaded beside x and the residual instead of behind the
// row's sum (53.7 -> 49 us: a block's loads are one trip to memory, not two), and
// launches are chained (pdl_wait at the start; the blocks of the next kernel take
// a SM's place as this one's leave it: 49 -> 45.1, 1 x 4096 4.2 -> 2.1, 1001 x
// 3584 8.3 -> 5.1 before the codes' quotients).  Tried and dropped: blocks that loop
// over rows with the next row's loads in flight (56 us: fewer threads a SM),
// one vector a thread (50 us), streaming cache hints (50 us).
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr float kMinAmax = 9.094947017729282e-13f;  // 2^-40

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// a / b in FP32 from the rounded reciprocal of b: the product's remainder is exact in a fused multiply-add and
// corrects it (Markstein, IBM J. Res. Dev. 34, 1990).  An infinite b (reciprocal 0) gives a * 0.  The product
// alone lies an ulp or two off, and beside a tie takes the neighbouring code; eight divisions a vector would take
// 47.9 us instead of 44.9 at 8192 x 4096, 27.1 instead of 22.5 at 2048 x 7168.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float q = a * inv;
  return inv == 0.f ? q : fmaf(fmaf(-q, b, a), inv, q);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Eight columns of the norm weight, as loaded.
template <bool F32>
struct Weight {
  uint4 v;
  __device__ __forceinline__ void load(const void* w, int at) { v = __ldg(static_cast<const uint4*>(w) + at); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(v, f); }
};
template <>
struct Weight<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* w, int at) {
    a = __ldg(static_cast<const float4*>(w) + 2 * at), b = __ldg(static_cast<const float4*>(w) + 2 * at + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// One row per block; thread i holds vectors i, i + blockDim, ... (8 columns
// each), so 16 consecutive lanes hold one 128-column block.
template <int V, int MAX_THREADS, int MIN_BLOCKS, bool F32>
__global__ void __launch_bounds__(MAX_THREADS, MIN_BLOCKS) add_rmsnorm_fp8_kernel(const NormArgs p) {
  const int64_t row = blockIdx.x;
  const int nvec = p.H / 8, nt = blockDim.x, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  __shared__ float s_sum[32];
  pdl_wait();
  uint4 x[V] = {}, r[V] = {};
  Weight<F32> w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = v * nt + tid;
    if (at < nvec) {
      x[v] = *reinterpret_cast<const uint4*>(p.x + row * p.ld_x + at * 8);
      if (p.residual) r[v] = *reinterpret_cast<const uint4*>(p.residual + row * p.ld_residual + at * 8);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * nt + tid < nvec) w[v].load(p.weight, v * nt + tid);
  float s[V][8], sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    unpack8(x[v], s[v]);
    if (p.residual) {
      float f[8];
      unpack8(r[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[v][i] += f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(s[v][i], s[v][i], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = lane < (nt >> 5) ? s_sum[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float rstd = rsqrtf(sum / (float)p.H + p.eps);
  const int cols = (p.H + 127) / 128;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = v * nt + tid;
    const bool in = at < nvec;
    float y[8], amax = 0.f;
    if (in) {
      float f[8];
      w[v].get(f);
      if (p.residual_out) *reinterpret_cast<uint4*>(p.residual_out + row * p.ld_residual_out + at * 8) = pack8(s[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = s[v][i] * rstd * f[i];
        amax = max_nan(amax, fabsf(y[i]));
      }
      if (p.normed) *reinterpret_cast<uint4*>(p.normed + row * p.H + at * 8) = pack8(y);
    }
    if (p.q) {
#pragma unroll
      for (int o = 8; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = max_nan(amax, kMinAmax);
      const float scale = quotient(amax, 448.f, 1.f / 448.f), inv = 1.f / scale;
      if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = quotient(y[i], scale, inv);
        uint2 c;
        c.x = e4m3x2_code(y[0], y[1]) | (e4m3x2_code(y[2], y[3]) << 16);
        c.y = e4m3x2_code(y[4], y[5]) | (e4m3x2_code(y[6], y[7]) << 16);
        *reinterpret_cast<uint2*>(p.q + row * p.H + at * 8) = c;
        if ((lane & 15) == 0) p.scales[row * cols + at / 16] = scale;
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm_fp8(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.H / 8;
  const dim3 grid((unsigned)a.T);
  auto go = [&](auto bf16, auto f32, int v) {
    const dim3 block(((nvec + v - 1) / v + 31) / 32 * 32);
    return launch_kernel(a.weight_f32 ? f32 : bf16, grid, block, 0, s, true, a);
  };
  // Two vectors a thread up to H = 4096, in the most blocks a SM whose
  // registers do not spill; four above, where two are slower (2048 x 7168 25.6 us
  // instead of 20.7, 1024 x 16384 33.9 instead of 33.8): 1024 threads reach H =
  // 32768, though they spill a little (512 x 32768 33.6 us, with eight vectors in
  // 512 threads 34.7).  Rows this long leave a SM one or two blocks, whose loads
  // nothing overlaps with stores: 1.5 times the floor of 22.3 us.
  if (nvec <= 512) return go(add_rmsnorm_fp8_kernel<2, 256, 5, false>, add_rmsnorm_fp8_kernel<2, 256, 4, true>, 2);
  if (nvec <= 2048) return go(add_rmsnorm_fp8_kernel<4, 512, 1, false>, add_rmsnorm_fp8_kernel<4, 512, 1, true>, 4);
  return go(add_rmsnorm_fp8_kernel<4, 1024, 1, false>, add_rmsnorm_fp8_kernel<4, 1024, 1, true>, 4);
}

}  // namespace nvfp4
