// FP8 linear with block scales on the 5th-generation tensor cores (see
// nvfp4_fp8_linear):
//
//   out[m][n] = sum_c sa[m][c] * sw[n / 128][c] * sum_{k in block c} a[m][k] * w[n][k]
//
// The scales are FP32 and change every 128 of K, so the tensor core cannot
// keep one accumulator over K: each K-block is a product of its own
// (tcgen05.mma kind::f8f6f4, E4M3, FP32 accumulator in TMEM) and the epilogue
// warps add it, times sa * sw, to sums in registers while the tensor core
// works on the next block in another accumulator.  sa is per row, i.e. per
// TMEM lane and thread; a warp's columns lie in one 128-block of w, so a
// thread multiplies a whole block by one number.
//
// Persistent, one CTA per SM, tiles of 128 x BN, 12 warps:
//   warp 0      TMA: per K-block a 128 x 128 box of a and a BN x 128 box of w
//               (SWIZZLE_128B) into a ring; rows and columns past the matrices
//               read as zero
//   warp 1      TMEM allocator, MMA issuer (4 MMAs of K = 32 per block)
//   warps 4-11  epilogue: a TMEM lane quarter and half of the columns each
// Every wait is bounded (see ptx.cuh) and reports in the library's status word.
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 128;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kRegsLaunch = 168;  // per thread at launch: 65,536 registers over 384 threads, in steps of 8
constexpr int kRegsSmall = 56;    // warps 0-3
constexpr int kRegsEpi = 224;     // epilogue: up to 128 sums and 64 loaded values
static_assert(128 * (kRegsSmall + 2 * kRegsEpi) <= kThreads * kRegsLaunch,
              "the register split must fit the launch allocation");

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK;
  static constexpr int STAGE_BYTES = A_BYTES + BN * kBK;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int BUFS = BN == 256 ? 2 : 4;  // TMEM accumulators
  static constexpr int TMEM_COLS = BUFS * BN;
  static constexpr int COLS = BN / 2;             // columns of an epilogue warp
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 8 * (2 * STAGES + 2 * BUFS + 1) + 16;
};

// E4M3 x E4M3 -> FP32, K-major operands, M = 128.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_load_32(uint32_t taddr, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(taddr)
      : "memory");
}

template <int BN>
struct Smem {
  uint8_t* stages;
  uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
  uint32_t* tmem_slot;
  int* abort_flag;
};

template <int BN>
__device__ __forceinline__ Smem<BN> carve(uint8_t* raw) {
  using C = Cfg<BN>;
  Smem<BN> s;
  s.stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.full = reinterpret_cast<uint64_t*>(s.stages + C::STAGES * C::STAGE_BYTES);
  s.empty = s.full + C::STAGES;
  s.acc_full = s.empty + C::STAGES;
  s.acc_empty = s.acc_full + C::BUFS;
  s.drain = s.acc_empty + C::BUFS;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  return s;
}

// Tiles m-fastest: the CTAs at work share few column tiles of w and every row of a.
struct Tile {
  int m0, n0;
};
template <int BN>
__device__ __forceinline__ Tile tile_at(const Fp8GemmArgs& p, int it) {
  const int nt = it / p.m_tiles;
  return {(it - nt * p.m_tiles) * kBM, nt * BN};
}

template <int BN>
__device__ void load_loop(const Fp8GemmArgs& p, const Smem<BN>& L) {
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  int ok = 1;
  for (int it = blockIdx.x; it < p.tiles && ok && !*abort; it += gridDim.x) {
    const Tile t = tile_at<BN>(p, it);
    for (int kb = 0; kb < p.kbs; ++kb) {
      if (lane == 0) ok = wait_bounded_spin(smem_u32(&L.empty[stage]), phase ^ 1u, abort, p.status, p.timeout_ns);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (leader) {
        const uint32_t at = smem_u32(L.stages) + stage * C::STAGE_BYTES, bar = smem_u32(&L.full[stage]);
        mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
        tma_load_2d(at, &p.map_a, kb * kBK, t.m0, bar);
        tma_load_2d(at + C::A_BYTES, &p.map_w, kb * kBK, t.n0, bar);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (lane == 0 && (*abort || !ok)) {  // copies in flight land before the CTA exits
    for (int s = 0; s < C::STAGES; ++s)
      if (issued & (1u << s)) {
        volatile int no_abort = 0;
        wait_bounded(smem_u32(&L.full[s]), (issued_parity >> s) & 1u, &no_abort, nullptr, p.timeout_ns);
      }
  }
  __syncwarp();
}

template <int BN>
__device__ void mma_loop(const Fp8GemmArgs& p, const Smem<BN>& L, uint32_t tmem) {
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  constexpr uint32_t idesc = idesc_e4m3(BN);
  const uint64_t a0 = smem_desc(smem_u32(L.stages), 16, 1024, 2);
  const uint64_t b0 = smem_desc(smem_u32(L.stages) + C::A_BYTES, 16, 1024, 2);
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
  bool issued = false;
  int ok = 1;
  for (int it = blockIdx.x; it < p.tiles && ok && !*abort; it += gridDim.x) {
    for (int kb = 0; kb < p.kbs; ++kb) {
      if (lane == 0) {
        ok = wait_bounded_spin(smem_u32(&L.acc_empty[buf]), buf_phase ^ 1u, abort, p.status, p.timeout_ns);
        if (ok) ok = wait_bounded_spin(smem_u32(&L.full[stage]), phase, abort, p.status, p.timeout_ns);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        const uint64_t ad = a0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
        const uint64_t bd = b0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) tc_mma_f8(tmem + buf * BN, ad + 2 * i, bd + 2 * i, idesc, i != 0);
        tc_commit(smem_u32(&L.empty[stage]));
        tc_commit(smem_u32(&L.acc_full[buf]));
      }
      __syncwarp();
      issued = true;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      if (++buf == C::BUFS) {
        buf = 0;
        buf_phase ^= 1u;
      }
    }
  }
  if (*abort && issued) {  // every MMA issued finishes before TMEM is freed
    if (leader) tc_commit(smem_u32(L.drain));
    __syncwarp();
    if (lane == 0) {
      volatile int no_abort = 0;
      wait_bounded(smem_u32(L.drain), 0, &no_abort, nullptr, p.timeout_ns);
    }
    __syncwarp();
  }
}

// acc += s * d for 32 columns.
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&d)[32], uint64_t s2) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    acc[i] = f2_fma(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), s2, acc[i]);
}

template <int BN>
__device__ void epilogue_loop(const Fp8GemmArgs& p, const Smem<BN>& L, uint32_t tmem) {
  using C = Cfg<BN>;
  constexpr int CHUNKS = C::COLS / 32;
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::COLS;
  uint32_t buf = 0, buf_phase = 0;
  int ok = 1;
  for (int it = blockIdx.x; it < p.tiles && ok; it += gridDim.x) {
    const Tile t = tile_at<BN>(p, it);
    const int m = t.m0 + quarter * 32 + lane, n0 = t.n0 + half * C::COLS;
    const bool row = m < p.M, live = n0 < p.N;
    const float* sa = p.a_scale + (int64_t)(row ? m : 0) * p.kbs;
    const float* sw = p.w_scale + (int64_t)(live ? n0 / 128 : 0) * p.kbs;
    // the block scales are loaded two blocks ahead
    auto scale_at = [&](int kb) { return kb < p.kbs ? __ldg(sa + kb) * __ldg(sw + kb) : 0.f; };
    float s0 = scale_at(0), s1 = scale_at(1);
    uint64_t acc[C::COLS / 2];
#pragma unroll
    for (int i = 0; i < C::COLS / 2; ++i) acc[i] = 0ull;
    for (int kb = 0; kb < p.kbs; ++kb) {
      const float s2 = scale_at(kb + 2);
      if (lane == 0) ok = wait_bounded_spin(smem_u32(&L.acc_full[buf]), buf_phase, abort, p.status, p.timeout_ns);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = t0 + buf * BN;
      const uint64_t ss = f2_pack(s0, s0);
      uint32_t d[2][32];
      tmem_load_32(at, d[0]);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        tmem_load_wait();
        if (c + 1 < CHUNKS) {
          tmem_load_32(at + 32 * (c + 1), d[(c + 1) & 1]);
        } else {  // everything is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&L.acc_empty[buf]));
        }
        add_scaled(acc + 16 * c, d[c & 1], ss);
      }
      s0 = s1;
      s1 = s2;
      if (++buf == C::BUFS) {
        buf = 0;
        buf_phase ^= 1u;
      }
    }
    if (!ok) break;
    if (!row) continue;
    const int cols = min(C::COLS, p.N - n0);  // a multiple of 8
    if (p.out_f32) {
      float* to = static_cast<float*>(p.out) + (int64_t)m * p.ld_out + n0;
#pragma unroll
      for (int i = 0; i < C::COLS / 8; ++i)
        if (8 * i < cols) {
          uint32_t v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            f2_unpack(acc[4 * i + j], x, y);
            v[2 * j] = __float_as_uint(x);
            v[2 * j + 1] = __float_as_uint(y);
          }
          reinterpret_cast<uint4*>(to + 8 * i)[0] = make_uint4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<uint4*>(to + 8 * i)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
    } else {
      uint16_t* to = static_cast<uint16_t*>(p.out) + (int64_t)m * p.ld_out + n0;
#pragma unroll
      for (int i = 0; i < C::COLS / 8; ++i)
        if (8 * i < cols) {
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            f2_unpack(acc[4 * i + j], x, y);
            v[j] = pack_bf16x2(x, y);
          }
          *reinterpret_cast<uint4*>(to + 8 * i) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmArgs p) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const Smem<BN> L = carve<BN>(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&L.full[s]), 1);
      mbar_init(smem_u32(&L.empty[s]), 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(smem_u32(&L.acc_full[b]), 1);
      mbar_init(smem_u32(&L.acc_empty[b]), kEpiWarps);
    }
    mbar_init(smem_u32(L.drain), 1);
    *L.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.map_a);
    prefetch_tmap(&p.map_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(L.tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  if (warp < kEpiWarp0) {
    regs_dec<kRegsSmall>();
    if (warp == 0) load_loop<BN>(p, L);
    if (warp == 1) mma_loop<BN>(p, L, tmem);
  } else {
    regs_inc<kRegsEpi>();
    epilogue_loop<BN>(p, L, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN>
cudaError_t launch(Fp8GemmArgs& p, int num_sms, cudaStream_t s) {
  static int configured = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured != dev) {
    // setmaxnreg.inc waits for what the other warps give back: launch only with the allocation it is sized for
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, fp8_gemm_kernel<BN>)) != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(fp8_gemm_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN>::SMEM);
    if (e != cudaSuccess) return e;
    configured = dev;
  }
  p.m_tiles = (int)((p.M + kBM - 1) / kBM);
  p.tiles = p.m_tiles * ((p.N + BN - 1) / BN);
  return launch_kernel(fp8_gemm_kernel<BN>, dim3(p.tiles < num_sms ? p.tiles : num_sms), dim3(kThreads),
                       Cfg<BN>::SMEM, s, false, p);
}

}  // namespace

// Columns of a tile: the widest whose tiles fill the SMs.
int fp8_gemm_bn(int64_t M, int64_t N, int num_sms) {
  const int64_t mt = (M + kBM - 1) / kBM;
  if (mt * ((N + 255) / 256) >= num_sms) return 256;
  if (mt * ((N + 127) / 128) >= num_sms) return 128;
  return 64;
}

cudaError_t launch_fp8_gemm(Fp8GemmArgs& p, int bn, int num_sms, cudaStream_t s) {
  return bn == 256 ? launch<256>(p, num_sms, s) : bn == 128 ? launch<128>(p, num_sms, s) : launch<64>(p, num_sms, s);
}

}  // namespace nvfp4
