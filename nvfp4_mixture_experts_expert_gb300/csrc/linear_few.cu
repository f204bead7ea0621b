// 16-bit linear for few rows of activations, of one matrix or of each expert (see
// nvfp4_linear, nvfp4_linear_shape):
//
//   out[m][n] = act(sum_k x[m][k] * w[n][k] + bias[n]) + residual[m][n]
//
// A block computes 16 rows of w (SwiGLU: eight of the gate and their eight of the
// up half) against up to kLinearFewRows rows of x at a time.  w is the M operand of
// mma.sync.m16n8k16: the K order inside a block of 64 is free as long as both
// operands use the same, so a lane holds 32 consecutive bytes of its rows (the
// four lanes of a quad together one 128-byte line) and nothing is staged.  The
// block's warps split K; their sums are added in a fixed order.
//
// Bound: reading w.  Launches are chained, and a block has its part of w fetched
// into L2 before it waits for the kernel before (not with experts: which of them
// have rows is that kernel's result).  1 x 4096 x 4096 takes 7.1 us in a row of calls
// with different w (4.7 TB/s; floor 4.9; 0.6 more without the fetch): launch, first loads
// and the join of 16 warps are ~2 of them.  One token of six experts of 4096 x 4096: 40 us
// (5.0 TB/s; floor 30).  Built and not faster: w and x through a ring of bulk copies, one
// CTA a SM (twice the time; two CTAs 1.3 times).
#include <cuda_runtime.h>

#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

// Warps of a block, and blocks a SM: one matrix has few blocks, of which each should
// have all of its K in flight (1 x 4096 x 4096 with eight warps 1.5 times as long), the
// experts together have many, which overlap one's end with the next's beginning (six
// experts' 4096 x 4096 40 us instead of 44).  Five blocks of eight warps leave 48 registers,
// of which the kernel spills a little (84 bytes of stores, 52 of loads a thread).
__host__ __device__ constexpr int warps_of(bool experts) { return experts ? 8 : 16; }
__host__ __device__ constexpr int blocks_of(bool experts) { return experts ? 5 : 2; }
constexpr int kRows = (int)kLinearFewRows;
static_assert(kRows == 8, "the N of one mma");

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes at p + off (16-byte granules past `end` read as zero).  Not by read-only loads:
// the kernel before may write them while this one is already there.
__device__ __forceinline__ void load32(const uint8_t* p, int off, int end, uint32_t (&v)[8]) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = off < end ? *reinterpret_cast<const uint4*>(p + off) : z;
  const uint4 b = off + 16 < end ? *reinterpret_cast<const uint4*>(p + off + 16) : z;
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The nth expert that has rows, -1: fewer have.  Every warp looks for itself.
__device__ __forceinline__ int group_with_rows(const LinearFewArgs& p, int nth) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.G; base += 32) {
    const uint32_t some = __ballot_sync(0xffffffffu, base + lane < p.G && p.counts[base + lane] > 0);
    if (nth < __popc(some)) return base + (int)__fns(some, 0, nth + 1);
    nth -= __popc(some);
  }
  return -1;
}

template <bool BF16, bool EXPERTS>
__global__ void __launch_bounds__(32 * warps_of(EXPERTS), blocks_of(EXPERTS)) linear_few_kernel(const LinearFewArgs p) {
  constexpr int kWarps = warps_of(EXPERTS);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const bool pairs = p.ep.act == kActSwiglu;
  const int out_cols = pairs ? 8 : 16;
  const int n0 = blockIdx.x * out_cols;
  const int bytes = p.K * 2, kbs = (p.K + 63) / 64;
  __shared__ float4 part[kWarps][32];
  __shared__ float sums[kRows][16];
  const uint8_t* w0 = p.w + (int64_t)min(n0 + g, p.ep.N - 1) * bytes;
  const uint8_t* w1 = p.w + (int64_t)(pairs ? p.ep.N + min(n0 + g, p.ep.N - 1) : min(n0 + g + 8, p.ep.N - 1)) * bytes;
  if constexpr (!EXPERTS) {
    for (int kb = warp; kb < kbs; kb += kWarps) {
      const int off = kb * 128 + q * 32;
      if (off < bytes) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 + off));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 + off));
      }
    }
  }
  pdl_trigger();
  pdl_wait();
  const int group = EXPERTS ? group_with_rows(p, blockIdx.y) : 0;
  if (group < 0) return;
  const int rows = EXPERTS ? p.counts[group] : p.M;
  const int64_t row0 = EXPERTS ? p.offsets[group] : 0;
  w0 += (int64_t)group * p.ep.wide * bytes;
  w1 += (int64_t)group * p.ep.wide * bytes;
  for (int m0 = 0; m0 < rows; m0 += kRows) {
    const int here = min(kRows, rows - m0);
    const uint8_t* x = p.a + (row0 + m0 + min(g, here - 1)) * p.ld_a * 2;
    float acc[4] = {};
#pragma unroll 2
    for (int kb = warp; kb < kbs; kb += kWarps) {
      const int off = kb * 128 + q * 32;
      uint32_t a0[8], a1[8], b[8];
      load32(w0, off, bytes, a0);
      load32(w1, off, bytes, a1);
      load32(x, off, bytes, b);  // lanes past the last row repeat it: their sums are not stored
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma16<BF16>(acc, a0[2 * i], a1[2 * i], a0[2 * i + 1], a1[2 * i + 1], b[2 * i], b[2 * i + 1]);
    }
    part[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (threadIdx.x < kRows * 16) {
      const int r = threadIdx.x & 15, m = threadIdx.x >> 4;
      const int src = (r & 7) * 4 + m / 2, c = (r >> 3) * 2 + (m & 1);
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += reinterpret_cast<const float*>(&part[i][src])[c];
      sums[m][r] = v;
    }
    __syncthreads();
    const int per = out_cols / 8, m = threadIdx.x / per, c = threadIdx.x % per * 8, col = n0 + c;
    if (m < here && col < p.ep.N) {
      float z[8], u[8], b[8], bu[8], res[8];
      load_bias<kEpiAny>(p.ep, group, col, b, bu);
      load_residual(p.ep, row0 + m0 + m, col, res);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = sums[m][c + i], u[i] = sums[m][8 + i];
      finish<kEpiAny>(p.ep, row0 + m0 + m, col, z, u, b, bu, res);
    }
    __syncthreads();
  }
}

}  // namespace

// One matrix: two passes over w (the second from L2) against a 128-row tile: 16 x 4096 x
// 4096 10.7 us against 12.3 (8 rows 7.1 against 17; 17 rows 14.3 against 12.4).
// Experts: as many rows as experts, and at most four passes should all of them fall to
// one.  us here and (in brackets) on tiles, each row of another expert / all of one:
//   rows                       8                    32                     256
//   32 of 4096 x 4096         48 (57) / 11 (20)    173 (163) / 27 (19)
//   256 of 4096 x 4096        49 (67) / 13 (29)    176 (173) / 34 (29)    1328 (1260) / 222 (35)
//   256 of 768 x 2048 SwiGLU  15 (27) / 5 (18)      41 (48) / 13 (18)      268 (247) / 89 (24)
constexpr int64_t kMostRowsOfExperts = 32;
bool linear_is_few(int64_t M, int groups) {
  return groups ? M <= (groups < kMostRowsOfExperts ? groups : kMostRowsOfExperts) : M <= 2 * kLinearFewRows;
}

cudaError_t launch_linear_few(const LinearFewArgs& p, cudaStream_t s) {
  const int out_cols = p.ep.act == kActSwiglu ? 8 : 16;
  // at most as many experts as rows have any
  const dim3 grid((p.ep.N + out_cols - 1) / out_cols, p.M < p.G ? p.M : p.G);
  auto go = [&](auto bf16, auto f16, bool experts) {
    return launch_kernel(p.ep.type == kTypeBf16 ? bf16 : f16, grid, dim3(32 * warps_of(experts)), 0, s, true, p);
  };
  return p.counts ? go(linear_few_kernel<true, true>, linear_few_kernel<false, true>, true)
                  : go(linear_few_kernel<true, false>, linear_few_kernel<false, false>, false);
}

}  // namespace nvfp4
