// FP8 linear with block scales for few rows of activations (see nvfp4_fp8_linear):
//
//   out[m][n] = sum_c sa[m][c] * sw[n / 128][c] * sum_{k in block c} a[m][k] * w[n][k]
//
// A block computes 16 rows of w against 8 * NT rows of a.  w is the M operand
// of mma.sync.m16n8k32 (E4M3 x E4M3): the K order inside a 128-block is free as
// long as both operands use the same, so a lane holds 32 consecutive bytes of
// its rows (the four lanes of a quad together one 128-byte line) and no
// shared-memory staging or conversion is needed.  The blocks' warps split K by
// 128-blocks; each block's product is scaled in FP32 and added to the running
// sum, and the warps' sums are added in a fixed order.
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

template <int NT>
__global__ void __launch_bounds__(kWarps * 32) fp8_small_kernel(const Fp8Args p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int64_t m0 = (int64_t)blockIdx.y * (8 * NT);
  const int kbs = (p.K + 127) / 128;
  __shared__ float4 part[kWarps][NT][32];
  const uint8_t* w0 = p.w + (int64_t)min(n0 + g, p.N - 1) * p.K;
  const uint8_t* w1 = p.w + (int64_t)min(n0 + g + 8, p.N - 1) * p.K;
  const float* sw = p.w_scale + (int64_t)(n0 / 128) * kbs;
  float acc[NT][4] = {};
  for (int kb = warp; kb < kbs; kb += kWarps) {
    const int off = kb * 128 + q * 32;
    uint32_t a0[8], a1[8];
    load32(w0, off, p.K, a0);
    load32(w1, off, p.K, a1);
    const float s = __ldg(sw + kb);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t b[8] = {};
      const int64_t m = m0 + j * 8 + g;
      if (m < p.M) load32(p.a + m * p.ld_a, off, p.K, b);
      const int64_t mc = m0 + j * 8 + 2 * q;
      const float s0 = mc < p.M ? __ldg(p.a_scale + mc * kbs + kb) * s : 0.f;
      const float s1 = mc + 1 < p.M ? __ldg(p.a_scale + (mc + 1) * kbs + kb) * s : 0.f;
      float d[4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_e4m3(d, a0[2 * i], a1[2 * i], a0[2 * i + 1], a1[2 * i + 1], b[2 * i], b[2 * i + 1]);
      acc[j][0] = fmaf(d[0], s0, acc[j][0]);
      acc[j][1] = fmaf(d[1], s1, acc[j][1]);
      acc[j][2] = fmaf(d[2], s0, acc[j][2]);
      acc[j][3] = fmaf(d[3], s1, acc[j][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[warp][j][lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  // thread -> (row of a, row of w); the 16 rows of w are consecutive outputs
  for (int i = threadIdx.x; i < NT * 8 * 16; i += kWarps * 32) {
    const int r = i & 15, t = i >> 4;
    const int src = (r & 7) * 4 + (t & 7) / 2, c = (r >> 3) * 2 + (t & 1);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += reinterpret_cast<const float*>(&part[w][t >> 3][src])[c];
    const int64_t m = m0 + t;
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
  const int nt = a.M <= 8 ? 1 : a.M <= 16 ? 2 : 4;
  const dim3 grid((a.N + 15) / 16, (unsigned)((a.M + 8 * nt - 1) / (8 * nt)));
  const dim3 block(kWarps * 32);
  if (nt == 1) return launch_kernel(fp8_small_kernel<1>, grid, block, 0, s, false, a);
  if (nt == 2) return launch_kernel(fp8_small_kernel<2>, grid, block, 0, s, false, a);
  return launch_kernel(fp8_small_kernel<4>, grid, block, 0, s, false, a);
}

}  // namespace nvfp4
