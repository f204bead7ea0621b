// FP8 linear with block scales (see nvfp4_fp8_linear) for a decode batch of
// rows, on the 5th-generation tensor cores: w is the MMA's M operand and the
// rows of a, padded to NB, its N operand, so that no tile is mostly padding,
// and K is split over the CTAs of a cluster, so that a projection of 4096 x 4096
// keeps 128 SMs reading w.
//
//   part_r[m][n] = sum over the K-blocks c of CTA r of (sa[m][c] * sw[n / 128][c]) * sum_{k in c} w[n][k] a[m][k]
//   out[m][n]    = part_0[m][n] + part_1[m][n] + ...       (FP32, in this order)
//
// A CTA owns 128 rows of w (one scale block) and a range of K-blocks, 6 warps:
//   warp 0     TMA: per K-block 128 x 128 of w and NB x 128 of a into a ring
//   warp 1     MMA issuer: each K-block into a TMEM accumulator of its own
//   warps 2-5  sums in registers, a row of w per thread: sums += scale * accumulator
// The partial sums then pass through shared memory and every CTA of the
// cluster adds up its share of the rows of a.  Every wait is bounded and
// reports in the library's status word.
//
// Bound: reading w, behind a fixed part of ~3 us (launch, first copies, the
// join through the cluster).  16 x 4096 x 4096 over 128 CTAs: 5.9 us in a row of
// calls with different w, floor 2.5; 32 rows 6.5; 16 x 512 x 512 2.8.  What
// counted: launches chained, with w's first blocks fetched into L2 before the
// wait for the kernel before (0.8 us), and the join with two rows' loads in
// flight a warp instead of one value a thread (1.5 us at 32 rows).  With 64 rows
// of a the same kernel took 8.0 us at 4096 x 4096, 13.6 at 6144 x 6144 and 4.6 at
// 512 x 512 against 8.9, 12.0 and 3.2 for fp8_gemm.cu, which has them from 33 on.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8_mma.cuh"
#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kTileN = 128;  // rows of w: the MMA's M
constexpr int kBK = 128;
constexpr int kEpiWarp0 = 2;
constexpr int kThreads = 32 * (kEpiWarp0 + 4);
constexpr int kBufs = 4;               // TMEM accumulators
constexpr int kScaleBytes = 8192;      // scale products of up to kScaleBytes / (4 NB) K-blocks

template <int NB>
struct SplitCfg {
  static constexpr int W_BYTES = kTileN * kBK;
  static constexpr int STAGE_BYTES = W_BYTES + NB * kBK;
  static constexpr int STAGES = NB == 16 ? 6 : 5;
  static constexpr int TMEM_COLS = kBufs * NB;
  static constexpr int CHUNK = kScaleBytes / (4 * NB);  // K-blocks whose scales are held at a time
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + kScaleBytes + 8 * (2 * STAGES + kBufs) + 16;
  static_assert(SMEM <= 232448 && NB * kTileN * 4 <= STAGES * STAGE_BYTES, "the partial sums reuse the ring");
  static_assert(STAGES >= kBufs, "a stage's barrier may not complete twice before it has been seen once");
};

__device__ __forceinline__ void prefetch_tile_l2(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void ld_shared_2x64(uint32_t at, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at) : "memory");
}
// The four warps of the sums.
__device__ __forceinline__ void sums_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

struct SplitSmem {
  uint32_t stages, scales, full, done, acc_empty;
  uint32_t* tmem_slot;
  int* abort_flag;
};
template <int NB>
__device__ __forceinline__ SplitSmem carve(uint8_t* raw) {
  using C = SplitCfg<NB>;
  SplitSmem s;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.stages = smem_u32(base);
  s.scales = s.stages + C::STAGES * C::STAGE_BYTES;
  s.full = s.scales + kScaleBytes;
  s.done = s.full + 8 * C::STAGES;
  s.acc_empty = s.done + 8 * C::STAGES;
  s.tmem_slot = reinterpret_cast<uint32_t*>(base + (s.acc_empty + 8 * kBufs - s.stages));
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  return s;
}

template <int NB>
__device__ void load_loop(const Fp8SplitArgs& p, const SplitSmem& L, int n0, int kb0, int kb1) {
  using C = SplitCfg<NB>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0;
  int issued = 0;
  if (p.stall) kb1 = kb0 + 1;
  for (int kb = kb0; kb < kb1; ++kb) {
    if (!warp_wait(L.done + 8 * stage, phase ^ 1u, abort, p.status)) break;
    if (leader) {
      const uint32_t at = L.stages + stage * C::STAGE_BYTES, bar = L.full + 8 * stage;
      mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
      tma_load_2d(at, &p.map_w, kb * kBK, n0, bar);
      tma_load_2d(at + C::W_BYTES, &p.map_a, kb * kBK, 0, bar);
    }
    __syncwarp();
    ++issued;
    if (++stage == C::STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // The copies land before the warp leaves, also where another role gives up later.
  if (lane == 0) {
    for (int b = max(issued - C::STAGES, 0); b < issued; ++b) {
      volatile int no_abort = 0;
      wait_bounded(L.full + 8 * (b % C::STAGES), (b / C::STAGES) & 1, &no_abort, nullptr, kDrainNs);
    }
  }
  __syncwarp();
}

template <int NB>
__device__ void mma_loop(const Fp8SplitArgs& p, const SplitSmem& L, uint32_t tmem, int blocks) {
  using C = SplitCfg<NB>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  constexpr uint32_t idesc = idesc_e4m3(NB);
  const uint64_t w0 = smem_desc(L.stages, 16, 1024, 2);
  const uint64_t a0 = smem_desc(L.stages + C::W_BYTES, 16, 1024, 2);
  uint32_t stage = 0, phase = 0;
  int b = 0;
  for (; b < blocks; ++b) {
    if (!warp_wait(L.full + 8 * stage, phase, abort, p.status) ||
        !warp_wait(L.acc_empty + 8 * (b % kBufs), ((b / kBufs) & 1) ^ 1, abort, p.status))
      break;
    tc_fence_after();
    if (leader) {
      const uint64_t wd = w0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
      const uint64_t ad = a0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) tc_mma_f8(tmem + b % kBufs * NB, wd + 2 * i, ad + 2 * i, idesc, i != 0);
      tc_commit(L.done + 8 * stage);
    }
    __syncwarp();
    if (++stage == C::STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // The products end before the warp leaves and TMEM is freed, also where another role gives up later.
  if (lane == 0 && b > 0) {
    volatile int no_abort = 0;
    wait_bounded(L.done + 8 * ((b - 1) % C::STAGES), ((b - 1) / C::STAGES) & 1, &no_abort, nullptr, kDrainNs);
  }
  __syncwarp();
}

template <bool F32>
__device__ __forceinline__ void store(const Fp8SplitArgs& p, int m, int n, float v) {
  if (m >= p.M || n >= p.N) return;
  if (F32)
    static_cast<float*>(p.out)[(int64_t)m * p.ld_out + n] = v;
  else
    static_cast<uint16_t*>(p.out)[(int64_t)m * p.ld_out + n] = (uint16_t)pack_bf16x2(v, v);
}

template <int NB, bool F32>
__device__ void sum_loop(const Fp8SplitArgs& p, const SplitSmem& L, uint32_t tmem, int n0, int kb0, int kb1) {
  using C = SplitCfg<NB>;
  volatile int* abort = L.abort_flag;
  const int tid = threadIdx.x - 32 * kEpiWarp0, lane = tid & 31, quarter = (threadIdx.x >> 5) & 3;
  const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16);
  const int row = quarter * 32 + lane;  // of the tile: TMEM's lane
  const float* sw = p.w_scale + (int64_t)(n0 / 128) * p.kbs;
  uint64_t acc[NB / 2];
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) acc[i] = 0ull;
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  int b = 0;
  for (int c0 = kb0; c0 < kb1; c0 += C::CHUNK) {
    const int count = min(C::CHUNK, kb1 - c0);
    if (c0 > kb0) sums_sync();  // the products before have been read
#pragma unroll 4
    for (int i = tid; i < NB * count; i += 128) {
      const int m = i % NB, k = c0 + i / NB;
      st_shared_f32(L.scales + i * 4, m < p.M ? __ldg(p.a_scale + (int64_t)m * p.kbs + k) * __ldg(sw + k) : 0.f);
    }
    sums_sync();
    for (int k = 0; k < count && ok; ++k, ++b) {
      ok = warp_wait(L.done + 8 * stage, phase, abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = t0 + b % kBufs * NB, sc = L.scales + k * NB * 4;
      uint32_t d[NB];
      tmem_load_cols(at, d);
      tmem_load_wait();
#pragma unroll
      for (int i = 0; i < NB; ++i) asm volatile("" : "+r"(d[i]));  // no use of d moves above the wait
      tc_fence_before();  // everything is in registers: the accumulator is free
      __syncwarp();
      arrive_if(lane == 0, L.acc_empty + 8 * (b % kBufs));
#pragma unroll
      for (int i = 0; i < NB / 2; i += 2) {
        uint64_t s0, s1;
        ld_shared_2x64(sc + 8 * i, s0, s1);
        acc[i] = f2_fma(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), s0, acc[i]);
        acc[i + 1] = f2_fma(f2_pack(__uint_as_float(d[2 * i + 2]), __uint_as_float(d[2 * i + 3])), s1, acc[i + 1]);
      }
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  // The ring is empty: every copy has landed and every product is complete.
  sums_sync();
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) {
    float x, y;
    f2_unpack(acc[i], x, y);
    if (p.split == 1) {
      store<F32>(p, 2 * i, n0 + row, x);
      store<F32>(p, 2 * i + 1, n0 + row, y);
    } else {
      st_shared_f32(L.stages + (2 * i * kTileN + row) * 4, x);
      st_shared_f32(L.stages + ((2 * i + 1) * kTileN + row) * 4, y);
    }
  }
}

// A warp adds up a row of a at a time, four columns a lane, two rows' loads in
// flight: a load from another CTA takes ~0.3 us.
template <bool F32>
__device__ void add_parts(const Fp8SplitArgs& p, const SplitSmem& L, int rows, int rank, int n0) {
  const int warp = (threadIdx.x >> 5) - kEpiWarp0, col = (threadIdx.x & 31) * 4, n = n0 + col;
  const int step = 4 * p.split;
  for (int m = rank + warp * p.split; m < rows; m += 2 * step) {
    uint4 v[2][kMaxSplit];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < p.split && m + j * step < rows)
          v[j][r] = ld_shared_cluster_v4(mapa_shared(L.stages + ((m + j * step) * kTileN + col) * 4, r));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t at = (int64_t)(m + j * step) * p.ld_out + n;
      if (m + j * step >= rows || n >= p.N) continue;
      float s[4] = {};
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < p.split) {
          s[0] += __uint_as_float(v[j][r].x);
          s[1] += __uint_as_float(v[j][r].y);
          s[2] += __uint_as_float(v[j][r].z);
          s[3] += __uint_as_float(v[j][r].w);
        }
      if (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(s[0], s[1], s[2], s[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
  }
}

template <int NB, bool F32>
__global__ void __launch_bounds__(kThreads, 1) fp8_split_kernel(const __grid_constant__ Fp8SplitArgs p) {
  using C = SplitCfg<NB>;
  extern __shared__ uint8_t smem_raw[];
  const SplitSmem L = carve<NB>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * kTileN;
  const int kb0 = (int)((int64_t)p.kbs * rank / p.split), kb1 = (int)((int64_t)p.kbs * (rank + 1) / p.split);
  if (threadIdx.x == 0) {
    // w on its way to L2 while the kernel before still runs; a may come from it
    for (int kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb) prefetch_tile_l2(&p.map_w, kb * kBK, n0);
    prefetch_tmap(&p.map_a);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(L.full + 8 * s, 1);
      mbar_init(L.done + 8 * s, 1);
    }
    for (int b = 0; b < kBufs; ++b) mbar_init(L.acc_empty + 8 * b, 4);
    *L.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(L.tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) load_loop<NB>(p, L, n0, kb0, kb1);
  if (warp == 1) mma_loop<NB>(p, L, tmem, kb1 - kb0);
  if (warp >= kEpiWarp0) sum_loop<NB, F32>(p, L, tmem, n0, kb0, kb1);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (p.split > 1) {
    cluster_sync_all();
    if (warp >= kEpiWarp0) add_parts<F32>(p, L, min(NB, p.M), rank, n0);
    __syncwarp();
    cluster_arrive_relaxed();  // the other CTAs' reads of this one's shared memory
    cluster_wait();
  }
}

template <int NB, bool F32>
cudaError_t launch(Fp8SplitArgs& p, int num_sms, cudaStream_t s) {
  constexpr size_t SMEM = SplitCfg<NB>::SMEM;
  static PerDevice<Clusters, cudaError_t> fit;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const Clusters* clusters = nullptr;
  e = fit.get(dev, &clusters, [](Clusters& c) {
    if (const cudaError_t e = cudaFuncSetAttribute(fp8_split_kernel<NB, F32>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM))
      return e;
    return max_clusters(fp8_split_kernel<NB, F32>, kThreads, SMEM, c);
  });
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + kTileN - 1) / kTileN;
  p.split = 1;  // the most CTAs that run at once, one a SM
  for (int c = 2; c <= kMaxSplit && c <= p.kbs; ++c)
    if (tiles * c <= num_sms && tiles <= clusters->most[c]) p.split = c;
  return launch_split<const Fp8SplitArgs>(fp8_split_kernel<NB, F32>, tiles * p.split, kThreads, SMEM, p.split, s, p);
}

}  // namespace

int fp8_split_nb(int64_t M) { return M <= 16 ? 16 : 32; }

cudaError_t launch_fp8_split(Fp8SplitArgs& p, bool f32, int num_sms, cudaStream_t s) {
  if (fp8_split_nb(p.M) == 16) return f32 ? launch<16, true>(p, num_sms, s) : launch<16, false>(p, num_sms, s);
  return f32 ? launch<32, true>(p, num_sms, s) : launch<32, false>(p, num_sms, s);
}

}  // namespace nvfp4
