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
// Persistent, one CTA per SM, tiles of 128 x BN; where a problem has few tiles, K
// is split over the CTAs of a cluster, which add their sums through shared memory
// (fp8_gemm_plan).  12 warps:
//   warp 0      TMA: per K-block a 128 x 128 box of a and a BN x 128 box of w
//               (SWIZZLE_128B) into a ring; rows and columns past the matrices
//               read as zero
//   warps 1, 2  MMA issuers (4 MMAs of K = 32 per block); warp 1 allocates TMEM
//   warp 3      a's scales, transposed into shared memory
//   warps 4-11  epilogue: a TMEM lane quarter and half of the columns each
// Every wait is bounded and reports in the library's status word.
//
// Measured (8192 x 4096 x 4096, bf16 out): 115 to 118 us in a row of calls over
// changing inputs, 2.3 to 2.4 PFLOP/s, 0.61 of twice the measured bf16 rate (the
// power cap counts: 109 us in short runs, the figure that those below stand
// against).  A K-block of a 128 x 256 tile takes ~900 cycles where its MMAs take 512:
// the issuers wait for accumulators, of which TMEM holds two, and an accumulator's
// way round (MMA, commit, the epilogue's wait of ~120 cycles and read of ~400,
// arrival, issue ~200) is 1,700.  Built and not faster: CTA pairs with 256 x 256
// tiles, which copy a third less a block (115 us), also with accumulators by column
// halves (115); w's scales through shared memory as a's are (109 to 112); an
// epilogue that enters the next block before it adds up the last columns of this
// one (129); column counts between (224, 192, 160, 96: two scales a warp; 2048 x
// 6144 x 3584 51 us with 224 against 49).
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "fp8_mma.cuh"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 128;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kMmaWarps = 2;  // warps 1 and 2
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kRegsLaunch = 168;  // per thread at launch: 65,536 registers over 384 threads, in steps of 8
constexpr int kRegsSmall = 56;    // warps 0-3
constexpr int kRegsEpi = 224;     // epilogue: up to 128 sums and 64 loaded values
static_assert(128 * (kRegsSmall + 2 * kRegsEpi) <= kThreads * kRegsLaunch,
              "the register split must fit the launch allocation");

constexpr int kStagingBytes = 32 * 64;  // an epilogue warp's output buffer
// a's scales pass through shared memory transposed, kScaleKb blocks of 128 rows
// a slot: read from global memory by the epilogue, a row per lane, each block's
// loads would touch 32 lines (256 cycles of the load unit over the 8 warps).
constexpr int kScaleKb = 8;
constexpr int kScaleSlots = 3;
constexpr int kScalePitch = kBM + 4;  // floats; the transposing stores then hit 32 banks
constexpr int kScaleSlotBytes = kScaleKb * kScalePitch * 4;

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK;
  static constexpr int STAGE_BYTES = A_BYTES + BN * kBK;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int BUFS = BN == 256 ? 2 : 4;  // TMEM accumulators
  static constexpr int TMEM_COLS = BUFS * BN;
  static constexpr int COLS = BN / 2;             // columns of an epilogue warp
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + kEpiWarps * kStagingBytes +
                                 kScaleSlots * kScaleSlotBytes + 8 * (2 * STAGES + BUFS + 2 * kScaleSlots) + 16;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert(STAGES % kMmaWarps == 0 && BUFS % kMmaWarps == 0, "each MMA warp has slots of its own");
  static_assert(STAGES >= BUFS, "a stage's barrier may not complete twice before the epilogue has seen it once");
};

// Shared-memory addresses: the ring, the output buffers, the barriers (full[STAGES]: a block's
// operands have landed; done[STAGES]: its product is complete, which frees the
// ring slot and hands the accumulator to the epilogue; acc_empty[BUFS]: the
// epilogue has read an accumulator; sc_full, sc_empty[kScaleSlots]).
template <int BN>
struct Smem {
  uint32_t stages, staging, scales, full, done, acc_empty, sc_full, sc_empty;
  uint32_t* tmem_slot;
  int* abort_flag;
};

template <int BN>
__device__ __forceinline__ Smem<BN> carve(uint8_t* raw) {
  using C = Cfg<BN>;
  Smem<BN> s;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.stages = smem_u32(base);
  s.staging = s.stages + C::STAGES * C::STAGE_BYTES;
  s.scales = s.staging + kEpiWarps * kStagingBytes;
  s.full = s.scales + kScaleSlots * kScaleSlotBytes;
  s.done = s.full + 8 * C::STAGES;
  s.acc_empty = s.done + 8 * C::STAGES;
  s.sc_full = s.acc_empty + 8 * C::BUFS;
  s.sc_empty = s.sc_full + 8 * kScaleSlots;
  s.tmem_slot = reinterpret_cast<uint32_t*>(base + (s.sc_empty + 8 * kScaleSlots - s.stages));
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

// This CTA's tiles (first, step) and K-blocks: all of them, or with SPLIT one
// range of one tile, whose other ranges the cluster's other CTAs have.
struct Work {
  int tile, step, kb0, kb1;
};
template <bool SPLIT>
__device__ __forceinline__ Work work_of(const Fp8GemmArgs& p) {
  if (!SPLIT) return {(int)blockIdx.x, (int)gridDim.x, 0, p.kbs};
  const int rank = blockIdx.x % p.split;
  return {(int)blockIdx.x / p.split, p.tiles, (int)((int64_t)p.kbs * rank / p.split),
          (int)((int64_t)p.kbs * (rank + 1) / p.split)};
}

template <int BN, bool SPLIT>
__device__ void load_loop(const Fp8GemmArgs& p, const Smem<BN>& L) {
  const Work g = work_of<SPLIT>(p);
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  const int kb1 = p.stall ? g.kb0 + 1 : g.kb1;
  for (int it = g.tile; it < p.tiles && ok && !*abort; it += g.step) {
    const Tile t = tile_at<BN>(p, it);
    for (int kb = g.kb0; kb < kb1; ++kb) {
      ok = warp_wait(L.done + 8 * stage, phase ^ 1u, abort, p.status);
      if (!ok) break;
      if (leader) {
        const uint32_t at = L.stages + stage * C::STAGE_BYTES, bar = L.full + 8 * stage;
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
  // The copies land before the warp leaves, also where another role gives up later.
  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s)
      if (issued & (1u << s)) {
        volatile int no_abort = 0;
        wait_bounded(L.full + 8 * s, (issued_parity >> s) & 1u, &no_abort, nullptr, kDrainNs);
      }
  }
  __syncwarp();
}

// Slot by slot: 128 rows x kScaleKb blocks, four rows of eight to a copy, up to
// kScaleSlots ahead.  Asynchronous, because behind the operand copies that the
// ring keeps in flight a load takes microseconds.
template <int BN, bool SPLIT>
__device__ void scale_loop(const Fp8GemmArgs& p, const Smem<BN>& L) {
  const Work g = work_of<SPLIT>(p);
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31, r0 = lane >> 3, k = lane & 7;
  uint32_t slot = 0, phase = 0;
  bool ok = true;
  for (int it = g.tile; it < p.tiles && ok; it += g.step) {
    const Tile t = tile_at<BN>(p, it);
    for (int c0 = g.kb0; c0 < g.kb1; c0 += kScaleKb) {
      ok = warp_wait(L.sc_empty + 8 * slot, phase ^ 1u, abort, p.status);
      if (!ok) break;
      const uint32_t to = L.scales + slot * kScaleSlotBytes + (k * kScalePitch + r0) * 4;
      // past the last row or block: some valid scale, for sums that nobody stores or uses
      const float* from = p.a_scale + min(c0 + k, p.kbs - 1);
#pragma unroll 8
      for (int i = 0; i < kBM / 4; ++i)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i * 16),
                     "l"(from + (int64_t)min(t.m0 + i * 4 + r0, p.M - 1) * p.kbs)
                     : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(L.sc_full + 8 * slot) : "memory");
      if (++slot == kScaleSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Two warps issue alternate blocks (different ring slots and accumulators, so
// their order does not matter): waiting for a block's barriers and issuing its
// four MMAs takes a warp ~400 cycles, the MMAs of a 128 x 128 block 256.  One
// elected lane issues; the loop runs on the whole warp so that descriptors,
// addresses and phases are warp-uniform.
template <int BN, bool SPLIT>
__device__ void mma_loop(const Fp8GemmArgs& p, const Smem<BN>& L, uint32_t tmem, int which) {
  const Work g = work_of<SPLIT>(p);
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  constexpr uint32_t idesc = idesc_e4m3(BN);
  const uint64_t a0 = smem_desc(L.stages, 16, 1024, 2);
  const uint64_t b0 = smem_desc(L.stages + C::A_BYTES, 16, 1024, 2);
  uint32_t stage = which, phase = 0, buf = which, buf_phase = 1;
  const int blocks = (g.kb1 - g.kb0) * ((p.tiles - g.tile + g.step - 1) / g.step);
  uint32_t last = 0, last_phase = 0;
  bool issued = false;
  for (int b = which; b < blocks; b += kMmaWarps) {
    if (!warp_wait(L.full + 8 * stage, phase, abort, p.status) ||
        !warp_wait(L.acc_empty + 8 * buf, buf_phase, abort, p.status))
      break;
    tc_fence_after();
    if (leader) {
      const uint64_t ad = a0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
      const uint64_t bd = b0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
      const uint32_t d = tmem + buf * BN;
#pragma unroll
      for (int i = 0; i < 4; ++i) tc_mma_f8(d, ad + 2 * i, bd + 2 * i, idesc, i != 0);
      tc_commit(L.done + 8 * stage);
    }
    __syncwarp();
    issued = true;
    last = stage;
    last_phase = phase;
    if ((stage += kMmaWarps) >= C::STAGES) {
      stage -= C::STAGES;
      phase ^= 1u;
    }
    if ((buf += kMmaWarps) >= C::BUFS) {
      buf -= C::BUFS;
      buf_phase ^= 1u;
    }
  }
  // The products end before the warp leaves and TMEM is freed, also where another role gives up later.
  if (lane == 0 && issued) {
    volatile int no_abort = 0;
    wait_bounded(L.done + 8 * last, last_phase, &no_abort, nullptr, kDrainNs);
  }
  __syncwarp();
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// acc += s * d.
template <int W>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&d)[W], uint64_t s2) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i)
    acc[i] = f2_fma(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), s2, acc[i]);
}

// A block costs a warp pair of one SM quarter 64 packed multiply-adds a thread
// (256 cycles of the FP32 pipe for a 128 x 256 tile) and its TMEM reads (~150
// cycles for all eight warps); measured alone, both together take ~340, of the
// 512 that the block's MMAs take.  The rows' scales are loaded by warp 3; the
// columns' (one number a warp) one block ahead, and multiplied when used: a
// product any earlier would wait for the load.
template <int BN, bool F32, bool SPLIT>
__device__ void epilogue_loop(const Fp8GemmArgs& p, const Smem<BN>& L, uint32_t tmem) {
  const Work g = work_of<SPLIT>(p);
  using C = Cfg<BN>;
  constexpr int W = BN == 256 ? 16 : 32, CHUNKS = C::COLS / W;  // measured: 112 / 142 us at 256, 130 / 122 at 128
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::COLS;
  const uint32_t staging = L.staging + (warp - kEpiWarp0) * kStagingBytes;
  const uint32_t my_scales = L.scales + (quarter * 32 + lane) * 4;
  uint32_t stage = 0, phase = 0, buf = 0, sc = 0, sc_phase = 0;
  bool ok = true;
  for (int it = g.tile; it < p.tiles && ok; it += g.step) {
    const Tile t = tile_at<BN>(p, it);
    const int n0 = t.n0 + half * C::COLS;
    const float* sw = p.w_scale + (int64_t)(n0 < p.N ? n0 / 128 : 0) * p.kbs;
    float sw0 = __ldg(sw + g.kb0);
    uint64_t acc[C::COLS / 2];
#pragma unroll
    for (int i = 0; i < C::COLS / 2; ++i) acc[i] = 0ull;
    for (int kb = g.kb0; kb < g.kb1; ++kb) {
      const float sw1 = kb + 1 < g.kb1 ? __ldg(sw + kb + 1) : 0.f;
      const int sk = (kb - g.kb0) % kScaleKb;
      if (sk == 0) {
        ok = warp_wait(L.sc_full + 8 * sc, sc_phase, abort, p.status);
        if (!ok) break;
      }
      const float sa0 = ld_shared_f32(my_scales + sc * kScaleSlotBytes + sk * (kScalePitch * 4));
      ok = warp_wait(L.done + 8 * stage, phase, abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = t0 + buf * BN;
      const float s0 = sa0 * sw0;
      const uint64_t ss = f2_pack(s0, s0);
      // 256 columns: the next 16 on their way while these are added (2048 x 6144 x 3584 in 46.0 us instead of
      // 48.4; at 128 and 64 columns it costs up to 3 %)
      constexpr int AHEAD = BN == 256 ? 2 : 1;
      uint32_t d[AHEAD][W];
      tmem_load_cols(at, d[0]);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        uint32_t(&now)[W] = d[c % AHEAD];
        if (AHEAD == 1 && c > 0) tmem_load_cols(at + W * c, now);
        tmem_load_wait();
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+r"(now[i]));  // no use of it moves above the wait
        if (AHEAD == 2 && c + 1 < CHUNKS) tmem_load_cols(at + W * (c + 1), d[(c + 1) % AHEAD]);
        if (c + 1 == CHUNKS) {  // everything is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          arrive_if(lane == 0, L.acc_empty + 8 * buf);
        }
        add_scaled(acc + W / 2 * c, now, ss);
      }
      sw0 = sw1;
      if (sk == kScaleKb - 1 || kb + 1 == g.kb1) {
        __syncwarp();
        arrive_if(lane == 0, L.sc_empty + 8 * sc);
        if (++sc == kScaleSlots) {
          sc = 0;
          sc_phase ^= 1u;
        }
      }
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      if (++buf == C::BUFS) buf = 0;
    }
    if (!ok) break;
    if constexpr (SPLIT) {  // the range's sums, a row of the tile per thread, for the join
      const uint32_t to = L.stages + ((quarter * 32 + lane) * (BN + 4) + half * C::COLS) * 4;
#pragma unroll
      for (int i = 0; i < C::COLS / 4; ++i) {
        float v[4];
        f2_unpack(acc[2 * i], v[0], v[1]);
        f2_unpack(acc[2 * i + 1], v[2], v[3]);
        st_shared_v4(to + 16 * i, {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      }
      continue;
    }
    // 32 rows x 64 bytes at a time through the warp's staging buffer
    constexpr int PIECE = F32 ? 16 : 32;  // columns
#pragma unroll
    for (int c = 0; c < C::COLS / PIECE; ++c) {
      if (lane == 0) bulk_wait_read_all();  // the copy before has left the buffer
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 16 bytes each, at their place in the 64-byte swizzle
        constexpr int PER = F32 ? 2 : 4;  // pairs of sums
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          float x, y;
          f2_unpack(acc[c * PIECE / 2 + i * PER + j], x, y);
          if (F32) {
            v[2 * j] = __float_as_uint(x);
            v[2 * j + 1] = __float_as_uint(y);
          } else {
            v[j] = pack_bf16x2(x, y);
          }
        }
        st_shared_v4(staging + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int x = n0 + c * PIECE, y = t.m0 + quarter * 32;
        if (x < p.N && y < p.M) tma_store_2d(&p.map_out, staging, x, y);  // clipped to the matrix
        bulk_commit();
      }
    }
  }
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

// The cluster's CTAs add up the ranges' sums in K order, each its share of the
// tile's rows: four columns a lane, two rows' loads in flight.
template <int BN, bool F32>
__device__ void join_ranges(const Fp8GemmArgs& p, const Smem<BN>& L) {
  constexpr int PER = BN / 4, ROWS = 32 / PER;  // lanes a row, rows a warp
  static_assert(PER <= 32 && 32 % PER == 0, "a warp reads whole rows");
  const Tile t = tile_at<BN>(p, work_of<true>(p).tile);
  const int warp = (threadIdx.x >> 5) - kEpiWarp0, lane = threadIdx.x & 31, rank = blockIdx.x % p.split;
  const int col = lane % PER * 4, n = t.n0 + col;
  const int r0 = kBM * rank / p.split, r1 = min(kBM * (rank + 1) / p.split, p.M - t.m0);
  for (int r = r0 + warp * ROWS + lane / PER; r < r1; r += 2 * kEpiWarps * ROWS) {
    uint4 v[2][kMaxSplit];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = r + j * kEpiWarps * ROWS;
#pragma unroll
      for (int i = 0; i < kMaxSplit; ++i)
        if (i < p.split && row < r1) v[j][i] = ld_shared_cluster_v4(mapa_shared(L.stages + (row * (BN + 4) + col) * 4, i));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = r + j * kEpiWarps * ROWS;
      if (row >= r1 || n >= p.N) continue;
      float s[4] = {};
#pragma unroll
      for (int i = 0; i < kMaxSplit; ++i)
        if (i < p.split) {
          s[0] += __uint_as_float(v[j][i].x);
          s[1] += __uint_as_float(v[j][i].y);
          s[2] += __uint_as_float(v[j][i].z);
          s[3] += __uint_as_float(v[j][i].w);
        }
      const int64_t at = (int64_t)(t.m0 + row) * p.ld_out + n;
      if (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(s[0], s[1], s[2], s[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
  }
}

template <int BN, bool F32, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmArgs p) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const Smem<BN> L = carve<BN>(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(L.full + 8 * s, 1);
      mbar_init(L.done + 8 * s, 1);
    }
    for (int b = 0; b < C::BUFS; ++b) mbar_init(L.acc_empty + 8 * b, kEpiWarps);
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(L.sc_full + 8 * i, 32);
      mbar_init(L.sc_empty + 8 * i, kEpiWarps);
    }
    *L.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.map_a);
    prefetch_tmap(&p.map_w);
    prefetch_tmap(&p.map_out);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(L.tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  pdl_wait();
  if (warp < kEpiWarp0) {
    regs_dec<kRegsSmall>();
    if (warp == 0) load_loop<BN, SPLIT>(p, L);
    if (warp == 1 || warp == 2) mma_loop<BN, SPLIT>(p, L, tmem, warp - 1);
    if (warp == 3) scale_loop<BN, SPLIT>(p, L);
    if constexpr (SPLIT) {  // the two meetings of the join
      __syncwarp();
      cluster_sync_all();
      cluster_arrive_relaxed();
      cluster_wait();
    }
  } else {
    regs_inc<kRegsEpi>();
    epilogue_loop<BN, F32, SPLIT>(p, L, tmem);
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync_all();
      join_ranges<BN, F32>(p, L);
      __syncwarp();
      cluster_arrive_relaxed();  // the other CTAs' reads of this one's shared memory
      cluster_wait();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, bool F32, bool SPLIT>
cudaError_t configure() {
  static PerDevice<char, cudaError_t> done;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  const char* none = nullptr;
  return done.get(dev, &none, [](char&) {
    // setmaxnreg.inc waits for what the other warps give back: launch only with the allocation it is sized for
    cudaFuncAttributes fa;
    if (const cudaError_t e = cudaFuncGetAttributes(&fa, fp8_gemm_kernel<BN, F32, SPLIT>)) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(fp8_gemm_kernel<BN, F32, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Cfg<BN>::SMEM);
  });
}
template <int BN, bool F32>
cudaError_t launch(Fp8GemmArgs& p, int num_sms, cudaStream_t s) {
  p.m_tiles = (int)((p.M + kBM - 1) / kBM);
  p.tiles = p.m_tiles * ((p.N + BN - 1) / BN);
  cudaError_t e;
  if constexpr (BN < 256) {
    if (p.split > 1) {
      if ((e = configure<BN, F32, true>()) != cudaSuccess) return e;
      return launch_split<const Fp8GemmArgs>(fp8_gemm_kernel<BN, F32, true>, p.tiles * p.split, kThreads,
                                             Cfg<BN>::SMEM, p.split, s, p);
    }
  }
  if ((e = configure<BN, F32, false>()) != cudaSuccess) return e;
  return launch_kernel(fp8_gemm_kernel<BN, F32, false>, dim3(p.tiles < num_sms ? p.tiles : num_sms), dim3(kThreads),
                       Cfg<BN>::SMEM, s, true, p);
}
template <int BN>
cudaError_t launch_out(Fp8GemmArgs& p, bool f32, int num_sms, cudaStream_t s) {
  return f32 ? launch<BN, true>(p, num_sms, s) : launch<BN, false>(p, num_sms, s);
}

}  // namespace

// The plan whose K-blocks take least time: columns of a tile, by its rounds of
// tiles over the SMs, and where there is one round with SMs to spare, CTAs that
// share a tile's K.  A K-block of a tile measured 503, 279 and 199 ns at 256, 128
// and 64 columns (8192 x 4096 x 4096, at the time: 113, 125 and 172 us), so 64 pays when 256
// leaves most SMs without a tile (128 x 4096 x 4096: 8.5 against 16.2 us), and the
// join of a split K 3 and 2 us (300 x 1000 x 3600: 8.4 us with 128 columns and five
// CTAs a tile against 10.7 with 64 and one; 100 x 512 x 4096 5.7 against 8.4; 256 x
// 1000 x 1024, eight K-blocks, would lose: 5.3 against 4.3).
cudaError_t fp8_gemm_plan(Fp8GemmArgs& p, int num_sms) {
  static PerDevice<Clusters, cudaError_t> fit;  // one CTA a SM in all forms
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const Clusters* clusters = nullptr;
  e = fit.get(dev, &clusters, [](Clusters& c) {
    if (const cudaError_t e = configure<64, false, true>()) return e;
    return max_clusters(fp8_gemm_kernel<64, false, true>, kThreads, Cfg<64>::SMEM, c);
  });
  if (e != cudaSuccess) return e;
  constexpr int kBns[3] = {256, 128, 64}, kNs[3] = {503, 279, 199}, kJoinNs[3] = {0, 3000, 2000};
  const int64_t mt = (p.M + kBM - 1) / kBM;
  int64_t least = INT64_MAX;
  for (int i = 0; i < 3; ++i) {
    const int64_t tiles = mt * ((p.N + kBns[i] - 1) / kBns[i]);
    for (int c = 1; c <= (kBns[i] < 256 ? kMaxSplit : 1) && c <= p.kbs; ++c) {
      if (c > 1 && (tiles * c > num_sms || tiles > clusters->most[c])) continue;
      const int64_t ns = (tiles * c + num_sms - 1) / num_sms * ((p.kbs + c - 1) / c) * kNs[i] + (c > 1 ? kJoinNs[i] : 0);
      if (ns < least) least = ns, p.bn = kBns[i], p.split = c;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_fp8_gemm(Fp8GemmArgs& p, bool f32, int num_sms, cudaStream_t s) {
  return p.bn == 256   ? launch_out<256>(p, f32, num_sms, s)
         : p.bn == 128 ? launch_out<128>(p, f32, num_sms, s)
                       : launch_out<64>(p, f32, num_sms, s);
}

}  // namespace nvfp4
