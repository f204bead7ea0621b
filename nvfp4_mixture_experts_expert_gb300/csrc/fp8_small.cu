// FP8 linear with block scales for few rows of activations (see nvfp4_fp8_linear):
//
//   out[m][n] = sum_c sa[m][c] * sw[n / 128][c] * sum_{k in block c} a[m][k] * w[n][k]
//
// A block computes 16 rows of w against up to 8 rows of a.  w is the M operand
// of mma.sync.m16n8k32 (E4M3 x E4M3): the K order inside a 128-block is free as
// long as both operands use the same, so a lane holds 32 consecutive bytes of
// its rows (the four lanes of a quad together one 128-byte line) and no
// shared-memory staging or conversion is needed.  The blocks' warps split K by
// 128-blocks; each block's product is scaled in FP32 and added to the running
// sum, and the warps' sums are added in a fixed order.
//
// Bound: reading w.  Launches are chained, and a block has its part of w fetched
// into L2 before it waits for the kernel before, from which only a may come.
// 8 x 4096 x 4096 in 4.5 us in a row of calls with different w (floor 2.5 us;
// 5.5 without the fetch, 8.2 without the chaining), 1 x 48 x 4096 in 3.1.  Two
// and four tiles of 8 rows in a block took 8.9 and 12.6 us at 16 and 32 rows
// (every block reads all of a): fp8_split.cu takes 6.3 and 7.2.
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 16;

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes at p + off (16-byte granules past `end` read as zero).
__device__ __forceinline__ void load32(const uint8_t* p, int off, int end, uint32_t (&v)[8]) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = off < end ? __ldg(reinterpret_cast<const uint4*>(p + off)) : z;
  const uint4 b = off + 16 < end ? __ldg(reinterpret_cast<const uint4*>(p + off + 16)) : z;
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__global__ void __launch_bounds__(kWarps * 32) fp8_small_kernel(const Fp8Args p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int kbs = (p.K + 127) / 128;
  __shared__ float4 part[kWarps][32];
  const uint8_t* w0 = p.w + (int64_t)min(n0 + g, p.N - 1) * p.K;
  const uint8_t* w1 = p.w + (int64_t)min(n0 + g + 8, p.N - 1) * p.K;
  const float* sw = p.w_scale + (int64_t)(n0 / 128) * kbs;
  for (int kb = warp; kb < kbs; kb += kWarps) {
    const int off = kb * 128 + q * 32;
    if (off < p.K) {
      prefetch_l2(w0 + off);
      prefetch_l2(w1 + off);
    }
  }
  pdl_trigger();
  pdl_wait();
  float acc[4] = {};
  for (int kb = warp; kb < kbs; kb += kWarps) {
    const int off = kb * 128 + q * 32;
    uint32_t a0[8], a1[8], b[8] = {};
    load32(w0, off, p.K, a0);
    load32(w1, off, p.K, a1);
    if (g < p.M) load32(p.a + g * p.ld_a, off, p.K, b);
    const float s = __ldg(sw + kb);
    const int m = 2 * q;
    const float s0 = m < p.M ? __ldg(p.a_scale + (int64_t)m * kbs + kb) * s : 0.f;
    const float s1 = m + 1 < p.M ? __ldg(p.a_scale + (int64_t)(m + 1) * kbs + kb) * s : 0.f;
    float d[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma_e4m3(d, a0[2 * i], a1[2 * i], a0[2 * i + 1], a1[2 * i + 1], b[2 * i], b[2 * i + 1]);
    acc[0] = fmaf(d[0], s0, acc[0]);
    acc[1] = fmaf(d[1], s1, acc[1]);
    acc[2] = fmaf(d[2], s0, acc[2]);
    acc[3] = fmaf(d[3], s1, acc[3]);
  }
  part[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  // thread -> (row of a, row of w); the 16 rows of w are consecutive outputs
  if (threadIdx.x < 8 * 16) {
    const int r = threadIdx.x & 15, m = threadIdx.x >> 4;
    const int src = (r & 7) * 4 + m / 2, c = (r >> 3) * 2 + (m & 1);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += reinterpret_cast<const float*>(&part[w][src])[c];
    if (m < p.M && n0 + r < p.N) {
      if (p.out_f32)
        static_cast<float*>(p.out)[m * p.ld_out + n0 + r] = v;
      else
        static_cast<uint16_t*>(p.out)[m * p.ld_out + n0 + r] = (uint16_t)pack_bf16x2(v, v);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_small(const Fp8Args& a, cudaStream_t s) {
  return launch_kernel(fp8_small_kernel, dim3((a.N + 15) / 16), dim3(kWarps * 32), 0, s, true, a);
}

}  // namespace nvfp4
