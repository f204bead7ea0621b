// The elementwise half of the linear's gradient (see nvfp4_linear_grad):
//
//   dz[m][n] = dy[m][n] * act'(z[m][n]),   dbias[n] = sum over a group's rows m of dz[m][n]
//
// in one pass over dy and z.  dz is rounded to the operands' type, which the
// tensor cores multiply (half a step of that type for each term of dx and dw; two
// terms an element would double the products); the sums take it unrounded, in FP32:
// 8 warps a slab of kSlabRows rows, their sums in order into one partial row a slab,
// and a second launch adds the slabs of a group in order.
//
// Bound: HBM and, close to it, the arithmetic of the slope.  12294 x 2048 (bf16) without
// an activation, sums alone, 10 us (50 MB, floor 7.4), SiLU with dz 27 (150 MB, 22),
// SwiGLU with dz 49 (250 MB, 37), GELU by erf 44 (its erff and exp).  A kernel for each
// activation and type: with both chosen inside it 2048 x 6144 took 35 us instead of 17.
// Slabs of 32 and 128 rows, four rows a warp at a time: the same or up to 40 % slower.
#include <cuda_runtime.h>

#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kSlabRows = 64;
constexpr int kWarps = 8;

// d act(z) / dz.  The terms with a factor z vanish long before kFar, and are 0 * inf
// at an infinite z without it.
constexpr float kFar = 1e4f;
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  const float f = at_least(at_most(z, kFar), -kFar);
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    return s + f * s * (1.f - s);
  }
  if constexpr (ACT == kActGelu)
    return 0.5f * (1.f + erff(z * 0.70710678f)) + f * expf(-0.5f * f * f) * 0.39894228f;
  if constexpr (ACT == kActGeluTanh) {
    const float s = sigmoid(1.59576912f * (z + 0.044715f * z * z * z));
    return s + f * s * (1.f - s) * (1.59576912f * (1.f + 0.134145f * f * f));
  }
  return 1.f;
}
// dy act'(z).  Where relu' is 0 nothing of dy passes, also not an infinity (a product's
// 0 * inf would reach a row of dx and of dw, and dbias); z NaN: NaN.
template <int ACT>
__device__ __forceinline__ float through(float d, float z) {
  if constexpr (ACT == kActNone) return d;
  if constexpr (ACT == kActRelu) return z > 0.f ? d : z <= 0.f ? 0.f : z;
  return d * slope<ACT>(z);
}

// What eight columns of a row need of dy and z, as loaded (z and u: SwiGLU's gate and up).
struct Piece {
  uint4 d, z, u;
};
template <int ACT>
__device__ __forceinline__ void load_piece(const LinearGradArgs& p, int64_t row, int col, Piece& v) {
  v.d = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dy) + row * p.ld_dy + col);
  const uint16_t* z = static_cast<const uint16_t*>(p.z) + row * p.wide + col;
  if constexpr (ACT != kActNone) v.z = *reinterpret_cast<const uint4*>(z);
  if constexpr (ACT == kActSwiglu) v.u = *reinterpret_cast<const uint4*>(z + p.N);
}
template <int TYPE>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  unpack2(TYPE, v.x, f[0], f[1]), unpack2(TYPE, v.y, f[2], f[3]);
  unpack2(TYPE, v.z, f[4], f[5]), unpack2(TYPE, v.w, f[6], f[7]);
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

// 256 columns of a slab a block, eight a lane; a warp's rows two at a time (SwiGLU: one).
template <int ACT, int TYPE>
__global__ void __launch_bounds__(kWarps * 32, 4) linear_dz_kernel(const LinearGradArgs p) {
  constexpr bool PAIRS = ACT == kActSwiglu;
  constexpr int ROWS = PAIRS ? 1 : 2;  // SwiGLU: 49 us instead of 58 at 12294 x 2048 (the dz pass alone)
  pdl_trigger();
  pdl_wait();
  __shared__ int found[2];
  __shared__ float part[kWarps][PAIRS ? 2 : 1][256];
  Slab s;
  if (!slab_at(p, blockIdx.x, s, found)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.y * 256 + lane * 8;
  float sum[8] = {}, sum_u[8] = {};  // of the rounded products (no fused multiply-add): the same with and without dz
  if (col < p.N) {
    for (int r0 = warp; r0 < s.rows; r0 += ROWS * kWarps) {
      Piece v[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
        if (r0 + j * kWarps < s.rows) load_piece<ACT>(p, s.row0 + r0 + j * kWarps, col, v[j]);
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if (r0 + j * kWarps >= s.rows) break;
        const int64_t at = (s.row0 + r0 + j * kWarps) * p.wide + col;
        float d[8], z[8], u[8];
        unpack8<TYPE>(v[j].d, d);
        if constexpr (ACT != kActNone) unpack8<TYPE>(v[j].z, z);
        if constexpr (PAIRS) {
          unpack8<TYPE>(v[j].u, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = at_least(at_most(z[i], p.gate_limit), -kFar);
            const float uc = at_least(at_most(u[i], p.up_limit), -p.up_limit);
            const float sg = sigmoid(g), h = g * sg;
            // a gate without a limit may be infinite: h is cut as slope() cuts z
            z[i] = z[i] > p.gate_limit ? 0.f : __fmul_rn(d[i] * uc, fmaf(at_most(h, kFar), 1.f - sg, sg));
            u[i] = u[i] == uc ? __fmul_rn(d[i], h) : 0.f;
            const float du = u[i];
            sum[i] = __fadd_rn(sum[i], z[i]), sum_u[i] = __fadd_rn(sum_u[i], du);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[i] = through<ACT>(d[i], z[i]);
            sum[i] = __fadd_rn(sum[i], z[i]);
          }
        }
        if (p.dz) {
          store_cols<8>(p.dz, at, TYPE, z);
          if (PAIRS) store_cols<8>(p.dz, at + p.N, TYPE, u);
        }
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

// dbias[g][c]: the partial rows of group g's slabs.  32 columns a block; each warp
// adds every eighth slab in order, then the warps' sums in order.
__global__ void __launch_bounds__(kWarps * 32) linear_dbias_kernel(const LinearGradArgs p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.y, c = blockIdx.x * 32 + lane;
  __shared__ float part[kWarps][32];
  int first = 0, slabs = (p.M + kSlabRows - 1) / kSlabRows;
  if (p.counts) {
    for (int i = lane; i < g; i += 32) first += (p.counts[i] + kSlabRows - 1) / kSlabRows;
#pragma unroll
    for (int o = 16; o; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
    slabs = (p.counts[g] + kSlabRows - 1) / kSlabRows;
  }
  float v = 0.f;
  if (c < p.wide) {
    const float* from = p.partial + (int64_t)first * p.wide + c;
#pragma unroll 8
    for (int s = warp; s < slabs; s += kWarps) v += from[(int64_t)s * p.wide];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= p.wide) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += part[w][lane];
  p.dbias[(int64_t)g * p.wide + c] = v;
}

}  // namespace

int64_t linear_grad_slabs(int64_t M, int groups) { return (M + kSlabRows - 1) / kSlabRows + groups; }

cudaError_t launch_linear_dz(const LinearGradArgs& args, cudaStream_t s) {
  LinearGradArgs p = args;
  if (p.partial && !p.counts && p.M <= kSlabRows) p.partial = p.dbias;  // one slab: its sums are the bias's
  const dim3 grid((unsigned)linear_grad_slabs(p.M, p.counts ? p.G : 0), (p.N + 255) / 256);
  auto go = [&](auto bf16, auto f16) {
    return launch_kernel(p.type == kTypeBf16 ? bf16 : f16, grid, dim3(kWarps * 32), 0, s, true, p);
  };
#define DZ(act) go(linear_dz_kernel<act, kTypeBf16>, linear_dz_kernel<act, kTypeF16>)
  const cudaError_t e = p.act == kActRelu       ? DZ(kActRelu)
                        : p.act == kActSilu     ? DZ(kActSilu)
                        : p.act == kActGelu     ? DZ(kActGelu)
                        : p.act == kActGeluTanh ? DZ(kActGeluTanh)
                        : p.act == kActSwiglu   ? DZ(kActSwiglu)
                                                : DZ(kActNone);
#undef DZ
  if (e != cudaSuccess || !p.partial || p.partial == p.dbias) return e;
  return launch_kernel(linear_dbias_kernel, dim3((p.wide + 31) / 32, p.G), dim3(kWarps * 32), 0, s, true, p);
}

}  // namespace nvfp4
