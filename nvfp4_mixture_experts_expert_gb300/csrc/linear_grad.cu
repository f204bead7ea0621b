// The elementwise half of the linear's gradient (see nvfp4_linear_grad):
//
//   dz[m][n] = dy[m][n] * act'(z[m][n]),   dbias[n] = sum over a group's rows m of dz[m][n]
//
// in one pass over dy and z.  dz is rounded to the operands' type, which the
// tensor cores multiply (half a step of that type for each term of dx and dw; two
// terms an element would double the products); the sums take it unrounded, in FP32:
// 8 warps a slab of kSlabRows rows, their sums in order into one partial row a slab,
// and a second launch adds the slabs of a group in order.  Bound: HBM.
#include <cuda_runtime.h>

#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kSlabRows = 64;
constexpr int kWarps = 8;

// d act(z) / dz.
__device__ __forceinline__ float slope(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    case kActSilu: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case kActGelu: return 0.5f * (1.f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
    case kActGeluTanh: {
      const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
      return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * (0.79788456f * (1.f + 0.134145f * z * z));
    }
    default: return 1.f;
  }
}

// The slab of a block: its group and rows.  Slabs of a group are neighbours.
struct Slab {
  int g, rows;
  int64_t row0;
};
__device__ __forceinline__ bool slab_at(const LinearGradArgs& p, int s, Slab& out, int* shared) {
  if (!p.counts) {
    out = {0, (int)min((int64_t)kSlabRows, (int64_t)p.M - (int64_t)s * kSlabRows), (int64_t)s * kSlabRows};
    return out.rows > 0;
  }
  if (threadIdx.x < 32) {  // the group whose slabs hold s
    int before = 0, g = -1, at = 0;
    for (int base = 0; base < p.G && g < 0; base += 32) {
      const int i = base + threadIdx.x, c = i < p.G ? (p.counts[i] + kSlabRows - 1) / kSlabRows : 0;
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if ((int)threadIdx.x >= o) incl += x;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, s < before + incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        g = base + l;
        at = before + __shfl_sync(0xffffffffu, incl - c, l);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (threadIdx.x == 0) {
      shared[0] = g;
      shared[1] = at;
    }
  }
  __syncthreads();
  out.g = shared[0];
  if (out.g < 0) return false;
  const int from = (s - shared[1]) * kSlabRows;
  out.rows = min(kSlabRows, p.counts[out.g] - from);
  out.row0 = (int64_t)p.offsets[out.g] + from;
  return true;
}

// 256 columns of a slab a block, eight a lane.
template <bool PAIRS>
__global__ void __launch_bounds__(kWarps * 32) linear_dz_kernel(const LinearGradArgs p) {
  pdl_trigger();
  pdl_wait();
  __shared__ int found[2];
  __shared__ float part[kWarps][PAIRS ? 2 : 1][256];
  Slab s;
  if (!slab_at(p, blockIdx.x, s, found)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.y * 256 + lane * 8;
  float sum[8] = {}, sum_u[8] = {};
  if (col < p.N) {
    for (int r = warp; r < s.rows; r += kWarps) {
      const int64_t row = s.row0 + r;
      float d[8], z[8], u[8];
      load8(p.dy, row * p.ld_dy + col, p.type, d);
      if (PAIRS) {
        load8(p.z, row * p.wide + col, p.type, z);
        load8(p.z, row * p.wide + p.N + col, p.type, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = at_most(z[i], p.gate_limit), uc = at_least(at_most(u[i], p.up_limit), -p.up_limit);
          const float sg = sigmoid(g);
          const float dg = z[i] > p.gate_limit ? 0.f : d[i] * uc * (sg * (1.f + g * (1.f - sg)));
          const float du = fabsf(u[i]) > p.up_limit ? 0.f : d[i] * (g * sg);
          z[i] = dg, u[i] = du;
          sum[i] += dg, sum_u[i] += du;
        }
      } else {
        if (p.act != kActNone) {
          load8(p.z, row * p.wide + col, p.type, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = d[i] * slope(p.act, z[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = d[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += z[i];
      }
      if (p.dz) {
        store8(p.dz, row * p.wide + col, p.type, z);
        if (PAIRS) store8(p.dz, row * p.wide + p.N + col, p.type, u);
      }
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    part[warp][0][lane * 8 + i] = sum[i];
    if (PAIRS) part[warp][PAIRS ? 1 : 0][lane * 8 + i] = sum_u[i];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < (PAIRS ? 2 : 1); ++h) {
    const int c = blockIdx.y * 256 + threadIdx.x;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][h][threadIdx.x];
    if (c < p.N) p.partial[(int64_t)blockIdx.x * p.wide + h * p.N + c] = v;
  }
}

// dbias[g][c]: the partial rows of group g's slabs, in order.
__global__ void __launch_bounds__(256) linear_dbias_kernel(const LinearGradArgs p) {
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  __shared__ int first;
  int slabs = (p.M + kSlabRows - 1) / kSlabRows;
  if (p.counts) {
    if (threadIdx.x < 32) {
      int n = 0;
      for (int i = threadIdx.x; i < g; i += 32) n += (p.counts[i] + kSlabRows - 1) / kSlabRows;
#pragma unroll
      for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (threadIdx.x == 0) first = n;
    }
    slabs = (p.counts[g] + kSlabRows - 1) / kSlabRows;
  } else if (threadIdx.x == 0) {
    first = 0;
  }
  __syncthreads();
  if (c >= p.wide) return;
  const float* from = p.partial + (int64_t)first * p.wide + c;
  float v = 0.f;
#pragma unroll 8
  for (int s = 0; s < slabs; ++s) v += from[(int64_t)s * p.wide];
  p.dbias[(int64_t)g * p.wide + c] = v;
}

}  // namespace

int64_t linear_grad_slabs(int64_t M, int groups) { return (M + kSlabRows - 1) / kSlabRows + groups; }

cudaError_t launch_linear_dz(const LinearGradArgs& p, cudaStream_t s) {
  const dim3 grid((unsigned)linear_grad_slabs(p.M, p.counts ? p.G : 0), (p.N + 255) / 256);
  cudaError_t e = launch_kernel(p.act == kActSwiglu ? linear_dz_kernel<true> : linear_dz_kernel<false>, grid,
                                dim3(kWarps * 32), 0, s, true, p);
  if (e != cudaSuccess || !p.partial) return e;
  return launch_kernel(linear_dbias_kernel, dim3((p.wide + 255) / 256, p.G), dim3(256), 0, s, true, p);
}

}  // namespace nvfp4
