// 16-bit matrix products on the 5th-generation tensor cores with bias, activation
// and residual in the epilogue, over one matrix or over groups of rows (see
// nvfp4_linear, nvfp4_expert_linear and their gradients):
//
//   out[m][n] = act(sum_k A[m][k] * B[n][k] + bias[n]) + residual[m][n]
//
// The three products of a linear are one kernel; what changes is which dimension
// of an operand is contiguous in memory, which the tensor core takes as it is:
//   forward    A = x  [rows][K]        B = w [G][wide][K]     both by their rows
//   dx         A = dz [rows][wide]     B = w, read along its columns (b_mn)
//   dw         A = dz, B = x, both read along their columns (a_mn, b_mn); the
//              rows are the contraction, a group's rows one product (by_k)
// An operand read by rows lies in the ring as rows of 64 elements (128 bytes,
// SWIZZLE_128B), one read along columns as chunks of 64 columns x 64 rows.
//
// Groups: an expert's rows offsets[g] .. + counts[g] are tiled by themselves, a
// tile's rows behind the group's last are computed and not stored.  With by_k, rows
// behind the group's last are set to zero in the ring before the product.
//
// Persistent, tiles of 128 x BN, FP32 accumulators in TMEM, two of them, so that a
// tile's epilogue runs beside the next one's products.  Where a problem has few
// tiles, K is split over the CTAs of a cluster, which add their sums through shared
// memory.  10 warps: 0 TMA, 1 MMA issue (and TMEM), 2 to 9 epilogue (a lane quarter
// and half of the columns each).  Every wait is bounded and reports in the
// library's status word.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8_mma.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kMaxGroups = 256;
constexpr int kStagingBytes = 32 * 32 * 4;  // an epilogue warp's: 32 rows x 32 FP32 columns
constexpr int kChunkBytes = 64 * 128;       // 64 columns x 64 rows of an operand read along columns

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + BN * kBK * 2;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 7;
  static constexpr int BUFS = 2;
  static constexpr int TMEM_COLS = BUFS * BN;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + kEpiWarps * kStagingBytes +
                                 8 * (2 * STAGES + 2 * BUFS) + 16 + 4 * (kMaxGroups + 4);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// Shared-memory addresses: ring, staging, barriers (full: a stage has landed;
// empty: its products are done; acc_full, acc_empty: an accumulator), tiles before
// each group.
struct Smem {
  uint32_t stages, staging, full, empty, acc_full, acc_empty;
  uint32_t* tmem_slot;
  int* abort_flag;
  int* first_tile;  // [G + 1], in m-tiles
};

template <int BN>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
  using C = Cfg<BN>;
  Smem s;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.stages = smem_u32(base);
  s.staging = s.stages + C::STAGES * C::STAGE_BYTES;
  s.full = s.staging + kEpiWarps * kStagingBytes;
  s.empty = s.full + 8 * C::STAGES;
  s.acc_full = s.empty + 8 * C::STAGES;
  s.acc_empty = s.acc_full + 8 * C::BUFS;
  s.tmem_slot = reinterpret_cast<uint32_t*>(base + (s.acc_empty + 8 * C::BUFS - s.stages));
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  s.first_tile = s.abort_flag + 1;
  return s;
}

// One tile: its group, where its operands start, how many of its rows exist, and
// its contraction (K-blocks kb0 .. kb1 of this CTA; k0: first row with by_k; k_end:
// length).
struct Tile {
  int g, m0, n0, rows, kb0, kb1, k0, k_end;
  int64_t out_row;
};

// Walks the tiles of a role in its order; tiles of a group are neighbours, the
// group's rows run fastest (the CTAs at work share few column tiles of B).
template <bool SPLIT>
struct Walk {
  const LinearArgs& p;
  const int* first_tile;
  int it, step, rank, g = 0;
  int out_cols;  // columns of the output that a tile covers
  __device__ Walk(const LinearArgs& p, const int* first_tile, int bn)
      : p(p), first_tile(first_tile), out_cols(p.ep.act == kActSwiglu ? bn / 2 : bn) {
    it = SPLIT ? blockIdx.x / p.split : blockIdx.x;
    rank = SPLIT ? blockIdx.x % p.split : 0;
    step = SPLIT ? 1 << 30 : gridDim.x;
  }
  __device__ bool next(Tile& t) {
    const int m_total = p.by_k ? p.G * p.m_tiles : first_tile[p.G];
    if (it >= m_total * p.n_tiles) return false;
    if (p.by_k) {
      const int per = p.m_tiles * p.n_tiles;
      g = it / per;
      const int r = it - g * per, n = r / p.m_tiles;
      t.m0 = (r - n * p.m_tiles) * kBM;
      t.n0 = n * out_cols;
      t.rows = min(kBM, p.M - t.m0);
      t.out_row = (int64_t)g * p.M + t.m0;
      t.k0 = p.counts ? p.offsets[g] : 0;
      t.k_end = p.counts ? p.counts[g] : p.K;
    } else {
      while (it >= first_tile[g + 1] * p.n_tiles) ++g;
      const int mt = first_tile[g + 1] - first_tile[g], r = it - first_tile[g] * p.n_tiles, n = r / mt;
      const int m = (r - n * mt) * kBM;
      t.m0 = m + (p.counts ? p.offsets[g] : 0);
      t.n0 = n * out_cols;
      t.rows = min(kBM, (p.counts ? p.counts[g] : p.M) - m);
      t.out_row = t.m0;
      t.k0 = 0;
      t.k_end = p.K;
    }
    t.g = g;
    const int kbs = (t.k_end + kBK - 1) / kBK;
    t.kb0 = SPLIT ? (int)((int64_t)kbs * rank / p.split) : 0;
    t.kb1 = SPLIT ? (int)((int64_t)kbs * (rank + 1) / p.split) : kbs;
    it += step;
    return true;
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// FP32 accumulators, both operands FP16 or both BF16, either read along columns.
__device__ __forceinline__ uint32_t idesc_f16(int type, int a_mn, int b_mn, int m, int n) {
  const uint32_t fmt = type == kTypeBf16 ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int BN, bool SPLIT>
__device__ void load_loop(const LinearArgs& p, const Smem& L) {
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  Walk<SPLIT> walk(p, L.first_tile, BN);
  Tile t;
  while (ok && !*abort && walk.next(t)) {
    const int kb1 = p.stall && t.kb1 > t.kb0 ? t.kb0 + 1 : t.kb1;
    for (int kb = t.kb0; kb < kb1; ++kb) {
      ok = warp_wait(L.empty + 8 * stage, phase ^ 1u, abort, p.status);
      if (!ok) break;
      if (leader) {
        const uint32_t a = L.stages + stage * C::STAGE_BYTES, b = a + C::A_BYTES, bar = L.full + 8 * stage;
        const int k = t.k0 + kb * kBK;
        mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
        if (p.a_mn) {
#pragma unroll
          for (int i = 0; i < kBM / 64; ++i) tma_load_2d(a + i * kChunkBytes, &p.map_a, t.m0 + 64 * i, k, bar);
        } else {
          tma_load_2d(a, &p.map_a, k, t.m0, bar);
        }
        if (p.b_mn) {
          const int g = p.by_k ? 0 : t.g;
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) tma_load_3d(b + i * kChunkBytes, &p.map_b, t.n0 + 64 * i, k, g, bar);
        } else {
          tma_load_3d(b, &p.map_b, k, t.n0, t.g, bar);
          tma_load_3d(b + BN * kBK, &p.map_b, k, t.n0 + p.second, t.g, bar);
        }
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

// Rows `from` .. 15 behind it, up to a multiple of 16, of `chunks` column chunks: zero.
__device__ __forceinline__ void zero_rows(uint32_t at, int chunks, int from, int lane) {
  const int to = (from + 15) & ~15, per = (to - from) * 8;  // 16-byte pieces of a chunk
  for (int i = lane; i < chunks * per; i += 32) {
    const int c = i / per, r = i - c * per;
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + c * kChunkBytes + from * 128 + r * 16), "r"(0)
                 : "memory");
  }
}

template <int BN, bool SPLIT>
__device__ void mma_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  const uint32_t idesc = idesc_f16(p.ep.type, p.a_mn, p.b_mn, kBM, BN);
  // by rows: 8-row groups 1024 bytes apart; along columns: the same for 8 of K, 64-column chunks kChunkBytes apart
  const uint64_t a0 = smem_desc(L.stages, p.a_mn ? kChunkBytes : 16, 1024, 2);
  const uint64_t b0 = smem_desc(L.stages + C::A_BYTES, p.b_mn ? kChunkBytes : 16, 1024, 2);
  const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;  // 16 of K
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1, last = 0, last_phase = 0;
  bool issued = false, ok = true;
  Walk<SPLIT> walk(p, L.first_tile, BN);
  Tile t;
  while (ok && walk.next(t)) {
    if (t.kb0 == t.kb1) continue;  // nothing to add up: the epilogue takes zeros
    ok = warp_wait(L.acc_empty + 8 * buf, buf_phase, abort, p.status);
    if (!ok) break;
    const uint32_t d = tmem + buf * BN;
    for (int kb = t.kb0; kb < t.kb1; ++kb) {
      ok = warp_wait(L.full + 8 * stage, phase, abort, p.status);
      if (!ok) break;
      const uint32_t at = L.stages + stage * C::STAGE_BYTES;
      int steps = kBK / 16;
      const int left = t.k_end - kb * kBK;
      if (p.by_k && p.counts && left < kBK) {  // the next group's rows follow
        steps = (left + 15) / 16;
        zero_rows(at, kBM / 64 + BN / 64, left, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (leader) {
        const uint64_t ad = a0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
        const uint64_t bd = b0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int i = 0; i < kBK / 16; ++i)
          if (i < steps) tc_mma_f16(d, ad + i * a_step, bd + i * b_step, idesc, kb != t.kb0 || i != 0);
        tc_commit(L.empty + 8 * stage);
        if (kb + 1 == t.kb1) tc_commit(L.acc_full + 8 * buf);
      }
      __syncwarp();
      issued = true;
      last = stage;
      last_phase = phase;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (++buf == C::BUFS) {
      buf = 0;
      buf_phase ^= 1u;
    }
  }
  // The products end before the warp leaves and TMEM is freed, also where another role gives up later.
  if (lane == 0 && issued) {
    volatile int no_abort = 0;
    wait_bounded(L.empty + 8 * last, last_phase, &no_abort, nullptr, kDrainNs);
  }
  __syncwarp();
}

__device__ __forceinline__ void st_shared_f4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// 32 rows x 32 columns, a row per lane, to eight columns of rows lane / 4 + 8 i,
// through the warp's staging buffer: 16-byte pieces at piece ^ (row & 7), which
// keeps both directions free of bank conflicts.  So four lanes store 64 bytes of a
// row side by side, and bias and residual are read the same way.
__device__ __forceinline__ void turn(uint32_t staging, int lane, const uint32_t (&v)[32], float (&f)[4][8]) {
  __syncwarp();  // the reads before are done
#pragma unroll
  for (int i = 0; i < 8; ++i)
    st_shared_f4(staging + lane * 128 + ((i ^ (lane & 7)) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), c = (lane & 3) * 2;
    const float4 a = ld_shared_f4(staging + r * 128 + ((c ^ (r & 7)) << 4));
    const float4 b = ld_shared_f4(staging + r * 128 + (((c + 1) ^ (r & 7)) << 4));
    f[i][0] = a.x, f[i][1] = a.y, f[i][2] = a.z, f[i][3] = a.w;
    f[i][4] = b.x, f[i][5] = b.y, f[i][6] = b.z, f[i][7] = b.w;
  }
}

template <int BN, bool SPLIT>
__device__ void epilogue_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN>;
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const bool pairs = p.ep.act == kActSwiglu;
  const int cols = pairs ? BN / 4 : BN / 2;  // output columns of this warp
  const uint32_t staging = L.staging + (warp - kEpiWarp0) * kStagingBytes;
  uint32_t buf = 0, phase = 0;
  Walk<SPLIT> walk(p, L.first_tile, BN);
  Tile t;
  while (walk.next(t)) {
    const bool some = t.kb0 != t.kb1;
    if (some && !warp_wait(L.acc_full + 8 * buf, phase, abort, p.status)) break;
    tc_fence_after();
    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + half * cols;
    if constexpr (SPLIT) {  // the range's sums, a row of the tile per thread, for the join
      const uint32_t to = L.stages + ((quarter * 32 + lane) * (BN + 4) + half * (BN / 2)) * 4;
#pragma unroll
      for (int c = 0; c < BN / 2; c += 32) {
        uint32_t v[32];
        if (some) {
          tmem_load_cols(tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + half * (BN / 2) + c, v);
          tmem_load_wait();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          asm volatile("" : "+r"(v[i]));
          if (!some) v[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_f4(to + c * 4 + 16 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      break;  // one tile
    }
    const int row0 = quarter * 32 + (lane >> 2);
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
      uint32_t v[32], w[32];
      if (some) {
        tmem_load_cols(from + c, v);
        if (pairs) tmem_load_cols(from + BN / 2 + c, w);
        tmem_load_wait();
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        asm volatile("" : "+r"(v[i]));  // no use moves above the wait
        asm volatile("" : "+r"(w[i]));
        if (!some) v[i] = w[i] = 0;
      }
      if (some && c + 32 >= cols) {  // everything is in registers: the accumulator is free
        tc_fence_before();
        __syncwarp();
        arrive_if(lane == 0, L.acc_empty + 8 * buf);
      }
      const int col = t.n0 + half * cols + c + (lane & 3) * 8;
      const bool in = col < p.N;
      float f[4][8], u[4][8], b[8], bu[8];
      if (in) load_bias(p.ep, t.g, col, b, bu);
      turn(staging, lane, v, f);
      if (pairs) turn(staging, lane, w, u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in && row0 + 8 * i < t.rows) finish8(p.ep, t.out_row + row0 + 8 * i, col, f[i], u[i], b, bu);
    }
    if (some && ++buf == C::BUFS) {
      buf = 0;
      phase ^= 1u;
    }
  }
  __syncwarp();
}

// The cluster's CTAs add up the ranges' sums in K order, each its share of the
// tile's rows, eight output columns a lane.
template <int BN>
__device__ void join_ranges(const LinearArgs& p, const Smem& L) {
  Walk<true> walk(p, L.first_tile, BN);
  Tile t;
  if (!walk.next(t)) return;
  const bool pairs = p.ep.act == kActSwiglu;
  const int per = walk.out_cols / 8, rank = walk.rank;
  const int tid = threadIdx.x - kEpiWarp0 * 32;
  const int r0 = kBM * rank / p.split, r1 = min(kBM * (rank + 1) / p.split, t.rows);
  for (int i = tid; i < (r1 - r0) * per; i += kEpiWarps * 32) {
    const int r = r0 + i / per, c = i % per * 8, col = t.n0 + c;
    if (col >= p.N) continue;
    float z[8] = {}, u[8] = {}, b[8], bu[8];
    load_bias(p.ep, t.g, col, b, bu);
    auto add = [&](float(&s)[8], int at) {
      uint4 v[2][kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < p.split) {
          const uint32_t a = mapa_shared(L.stages + (r * (BN + 4) + at) * 4, q);
          v[0][q] = ld_shared_cluster_v4(a);
          v[1][q] = ld_shared_cluster_v4(a + 16);
        }
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < p.split) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[4 * h] += __uint_as_float(v[h][q].x);
            s[4 * h + 1] += __uint_as_float(v[h][q].y);
            s[4 * h + 2] += __uint_as_float(v[h][q].z);
            s[4 * h + 3] += __uint_as_float(v[h][q].w);
          }
        }
    };
    add(z, c);
    if (pairs) add(u, BN / 2 + c);
    finish8(p.ep, t.out_row + r, col, z, u, b, bu);
  }
}

// first_tile[g]: m-tiles before group g.
__device__ void count_tiles(const LinearArgs& p, int* first_tile) {
  if (!p.counts) {
    if (threadIdx.x == 0) {
      first_tile[0] = 0;
      first_tile[1] = p.m_tiles;
    }
    return;
  }
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int sum = 0;
  for (int base = 0; base < p.G; base += 32) {
    const int c = base + lane < p.G ? (p.counts[base + lane] + kBM - 1) / kBM : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (base + lane < p.G) first_tile[base + lane] = sum + incl - c;
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) first_tile[p.G] = sum;
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) linear_gemm_kernel(const __grid_constant__ LinearArgs p) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const Smem L = carve<BN>(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(L.full + 8 * s, 1);
      mbar_init(L.empty + 8 * s, 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(L.acc_full + 8 * b, 1);
      mbar_init(L.acc_empty + 8 * b, kEpiWarps);
    }
    *L.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.map_a);
    prefetch_tmap(&p.map_b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(L.tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  count_tiles(p, L.first_tile);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  if (warp == 0) load_loop<BN, SPLIT>(p, L);
  if (warp == 1) mma_loop<BN, SPLIT>(p, L, tmem);
  if (warp >= kEpiWarp0) epilogue_loop<BN, SPLIT>(p, L, tmem);
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= kEpiWarp0) join_ranges<BN>(p, L);
    __syncwarp();
    cluster_arrive_relaxed();  // the other CTAs' reads of this one's shared memory
    cluster_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, bool SPLIT>
cudaError_t configure() {
  static PerDevice<char, cudaError_t> done;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  const char* none = nullptr;
  return done.get(dev, &none, [](char&) {
    return cudaFuncSetAttribute(linear_gemm_kernel<BN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Cfg<BN>::SMEM);
  });
}

template <int BN>
cudaError_t launch(LinearArgs& p, int num_sms, cudaStream_t s) {
  const int out_cols = p.ep.act == kActSwiglu ? BN / 2 : BN;
  p.m_tiles = (p.M + kBM - 1) / kBM;
  p.n_tiles = (p.N + out_cols - 1) / out_cols;
  p.second = p.ep.act == kActSwiglu ? p.N : BN / 2;
  cudaError_t e;
  if constexpr (BN < 256) {
    if (p.split > 1) {
      if ((e = configure<BN, true>()) != cudaSuccess) return e;
      return launch_split<const LinearArgs>(linear_gemm_kernel<BN, true>, p.m_tiles * p.n_tiles * p.split, kThreads,
                                            Cfg<BN>::SMEM, p.split, s, p);
    }
  }
  if ((e = configure<BN, false>()) != cudaSuccess) return e;
  // groups by rows: at most one tile more than the rows' for each
  const int64_t m = p.by_k ? (int64_t)p.G * p.m_tiles : p.counts ? (int64_t)p.m_tiles + p.G : p.m_tiles;
  const int64_t tiles = m * p.n_tiles;
  return launch_kernel(linear_gemm_kernel<BN, false>, dim3((unsigned)(tiles < num_sms ? tiles : num_sms)),
                       dim3(kThreads), Cfg<BN>::SMEM, s, true, p);
}

}  // namespace

// The plan whose K-blocks take least time, as for the FP8 linear: columns of a
// tile by its rounds of tiles over the SMs, and where there is one round with SMs to
// spare, CTAs that share a tile's K.
cudaError_t linear_gemm_plan(LinearArgs& p, int num_sms) {
  static PerDevice<Clusters, cudaError_t> fit;  // one CTA a SM in all forms
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const Clusters* clusters = nullptr;
  e = fit.get(dev, &clusters, [](Clusters& c) {
    if (const cudaError_t e = configure<128, true>()) return e;
    return max_clusters(linear_gemm_kernel<128, true>, kThreads, Cfg<128>::SMEM, c);
  });
  if (e != cudaSuccess) return e;
  constexpr int kBns[3] = {256, 128, 64}, kNs[3] = {330, 190, 140}, kJoinNs[3] = {0, 3000, 2000};
  const bool pairs = p.ep.act == kActSwiglu;
  const int64_t k = p.counts && p.by_k ? (p.K + p.G - 1) / p.G : p.K;  // of a group, on average
  const int64_t kbs = (k + kBK - 1) / kBK;
  // rows of groups: half a tile more for each
  const int64_t mt = p.by_k ? (int64_t)p.G * ((p.M + kBM - 1) / kBM)
                            : (p.M + kBM - 1) / kBM + (p.counts ? (p.G + 1) / 2 : 0);
  int64_t least = INT64_MAX;
  for (int i = 0; i < (pairs ? 2 : 3); ++i) {
    const int out_cols = pairs ? kBns[i] / 2 : kBns[i];
    const int64_t tiles = mt * ((p.N + out_cols - 1) / out_cols);
    for (int c = 1; c <= (kBns[i] < 256 && !p.counts ? kMaxSplit : 1) && c <= kbs; ++c) {
      if (c > 1 && (tiles * c > num_sms || tiles > clusters->most[c])) continue;
      const int64_t ns = (tiles * c + num_sms - 1) / num_sms * ((kbs + c - 1) / c) * kNs[i] + (c > 1 ? kJoinNs[i] : 0);
      if (ns < least) least = ns, p.bn = kBns[i], p.split = c;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_linear_gemm(LinearArgs& p, int num_sms, cudaStream_t s) {
  return p.bn == 256   ? launch<256>(p, num_sms, s)
         : p.bn == 128 ? launch<128>(p, num_sms, s)
                       : launch<64>(p, num_sms, s);
}

}  // namespace nvfp4
