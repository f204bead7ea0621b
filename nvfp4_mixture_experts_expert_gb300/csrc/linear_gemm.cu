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
constexpr int kChunk = kEpilogueColumns;  // columns that an epilogue thread holds at a time
constexpr int kBiasBytes = 2 * 128 * 4;  // an epilogue warp's: the bias of up to 128 columns, SwiGLU of both halves
constexpr int kChunkBytes = 64 * 128;       // 64 columns x 64 rows of an operand read along columns

template <int BN, bool PAIR>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK * 2;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // of B that this CTA holds
  static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * kBK * 2;
  static constexpr int STAGES = PAIR ? 6 : BN == 256 ? 4 : BN == 128 ? 6 : 7;
  static constexpr int UNIT_ROWS = PAIR ? 2 * kBM : kBM;  // of a tile
  static constexpr int BUFS = 2;
  static constexpr int TMEM_COLS = BUFS * BN;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + kEpiWarps * kBiasBytes +
                                 8 * (3 * STAGES + 2 * BUFS) + 16 + 4 * (kMaxGroups + 4);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// Shared-memory addresses: ring, bias, barriers (full: a stage has landed;
// empty: its products are done; peer_full: the other CTA's stage has landed;
// acc_full, acc_empty: an accumulator), tiles before each group.
struct Smem {
  uint32_t stages, bias, full, empty, peer_full, acc_full, acc_empty;
  uint32_t* tmem_slot;
  int* abort_flag;
  int* first_tile;  // [G + 1], in m-tiles
};

template <int BN, bool PAIR>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
  using C = Cfg<BN, PAIR>;
  Smem s;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.stages = smem_u32(base);
  s.bias = s.stages + C::STAGES * C::STAGE_BYTES;
  s.full = s.bias + kEpiWarps * kBiasBytes;
  s.empty = s.full + 8 * C::STAGES;
  s.peer_full = s.empty + 8 * C::STAGES;
  s.acc_full = s.peer_full + 8 * C::STAGES;
  s.acc_empty = s.acc_full + 8 * C::BUFS;
  s.tmem_slot = reinterpret_cast<uint32_t*>(base + (s.acc_empty + 8 * C::BUFS - s.stages));
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  s.first_tile = s.abort_flag + 1;
  return s;
}

// This CTA's part of a tile: its group, where its operands start, how many of its
// rows exist (in a pair's second half none, or less, may), and its contraction (K-blocks kb0 .. kb1 of this CTA; k0: first row with by_k; k_end:
// length).
struct Tile {
  int g, m0, n0, rows, kb0, kb1, k0, k_end;
  int64_t out_row;
};

// Walks the tiles of a role in its order; tiles of a group are neighbours, the
// group's rows run fastest (the CTAs at work share few column tiles of B).
template <bool SPLIT, bool PAIR>
struct Walk {
  static constexpr int UNIT = PAIR ? 2 * kBM : kBM;
  const LinearArgs& p;
  const int* first_tile;
  int it, step, rank, g = 0;
  int out_cols;  // columns of the output that a tile covers
  __device__ Walk(const LinearArgs& p, const int* first_tile, int bn)
      : p(p), first_tile(first_tile), out_cols(p.ep.act == kActSwiglu ? bn / 2 : bn) {
    it = SPLIT ? blockIdx.x / p.split : PAIR ? blockIdx.x / 2 : blockIdx.x;
    rank = SPLIT ? blockIdx.x % p.split : PAIR ? blockIdx.x % 2 : 0;
    step = SPLIT ? 1 << 30 : PAIR ? gridDim.x / 2 : gridDim.x;
  }
  __device__ bool next(Tile& t) {
    const int m_total = p.by_k ? p.G * p.m_tiles : first_tile[p.G];
    if (it >= m_total * p.n_tiles) return false;
    if (p.by_k) {
      const int per = p.m_tiles * p.n_tiles;
      g = it / per;
      const int r = it - g * per, n = r / p.m_tiles;
      t.m0 = (r - n * p.m_tiles) * UNIT + (PAIR ? rank * kBM : 0);
      t.n0 = n * out_cols;
      t.rows = min(kBM, p.M - t.m0);
      t.out_row = (int64_t)g * p.M + t.m0;
      t.k0 = p.counts ? p.offsets[g] : 0;
      t.k_end = p.counts ? p.counts[g] : p.K;
    } else {
      while (it >= first_tile[g + 1] * p.n_tiles) ++g;
      const int mt = first_tile[g + 1] - first_tile[g], r = it - first_tile[g] * p.n_tiles, n = r / mt;
      const int m = (r - n * mt) * UNIT + (PAIR ? rank * kBM : 0);
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

template <bool PAIR>
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
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

template <int BN, bool SPLIT, bool PAIR>
__device__ void load_loop(const LinearArgs& p, const Smem& L) {
  using C = Cfg<BN, PAIR>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  Walk<SPLIT, PAIR> walk(p, L.first_tile, BN);
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
          const int g = p.by_k ? 0 : t.g, n0 = t.n0 + (PAIR ? walk.rank * C::B_ROWS : 0);
#pragma unroll
          for (int i = 0; i < C::B_ROWS / 64; ++i) tma_load_3d(b + i * kChunkBytes, &p.map_b, n0 + 64 * i, k, g, bar);
        } else if (PAIR) {
          tma_load_3d(b, &p.map_b, k, t.n0 + walk.rank * p.second, t.g, bar);
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

// With by_k: a group's last K-block, behind which the next group's rows follow.
// Sets them to zero in this CTA's operands; returns the steps of 16 that count.
template <int BN, bool PAIR>
__device__ __forceinline__ int end_of_group(const LinearArgs& p, uint32_t at, int left, int lane) {
  if (!p.by_k || !p.counts || left >= kBK) return kBK / 16;
  zero_rows(at, kBM / 64 + Cfg<BN, PAIR>::B_ROWS / 64, left, lane);
  fence_proxy_async_smem();
  __syncwarp();
  return (left + 15) / 16;
}

template <int BN, bool SPLIT, bool PAIR>
__device__ void mma_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN, PAIR>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  const uint32_t idesc = idesc_f16(p.ep.type, p.a_mn, p.b_mn, C::UNIT_ROWS, BN);
  // by rows: 8-row groups 1024 bytes apart; along columns: the same for 8 of K, 64-column chunks kChunkBytes apart
  const uint64_t a0 = smem_desc(L.stages, p.a_mn ? kChunkBytes : 16, 1024, 2);
  const uint64_t b0 = smem_desc(L.stages + C::A_BYTES, p.b_mn ? kChunkBytes : 16, 1024, 2);
  const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;  // 16 of K
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1, last = 0, last_phase = 0;
  bool issued = false, ok = true;
  Walk<SPLIT, PAIR> walk(p, L.first_tile, BN);
  Tile t;
  while (ok && walk.next(t)) {
    if (t.kb0 == t.kb1) continue;  // nothing to add up: the epilogue takes zeros
    ok = warp_wait(L.acc_empty + 8 * buf, buf_phase, abort, p.status);
    if (!ok) break;
    const uint32_t d = tmem + buf * BN;
    for (int kb = t.kb0; kb < t.kb1; ++kb) {
      ok = warp_wait(L.full + 8 * stage, phase, abort, p.status);
      if (!ok) break;
      const int left = t.k_end - kb * kBK;
      const int steps = end_of_group<BN, PAIR>(p, L.stages + stage * C::STAGE_BYTES, left, lane);
      if constexpr (PAIR) {
        ok = warp_wait(L.peer_full + 8 * stage, phase, abort, p.status);
        if (!ok) break;
        if (steps < kBK / 16 || left < kBK) asm volatile("fence.acq_rel.cluster;" ::: "memory");
      }
      tc_fence_after();
      if (leader) {
        const uint64_t ad = a0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
        const uint64_t bd = b0 + (uint64_t)stage * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int i = 0; i < kBK / 16; ++i)
          if (i < steps) tc_mma_f16<PAIR>(d, ad + i * a_step, bd + i * b_step, idesc, kb != t.kb0 || i != 0);
        if constexpr (PAIR) {
          tc_commit_pair_mc(L.empty + 8 * stage, 3);
          if (kb + 1 == t.kb1) tc_commit_pair_mc(L.acc_full + 8 * buf, 3);
        } else {
          tc_commit(L.empty + 8 * stage);
          if (kb + 1 == t.kb1) tc_commit(L.acc_full + 8 * buf);
        }
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

// The second CTA of a pair tells the first, which issues the products, that its
// operands of a stage have landed (and end where the group ends).
template <int BN>
__device__ void relay_loop(const LinearArgs& p, const Smem& L) {
  using C = Cfg<BN, true>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  uint32_t stage = 0, phase = 0;
  Walk<false, true> walk(p, L.first_tile, BN);
  Tile t;
  bool ok = true;
  while (ok && walk.next(t)) {
    for (int kb = t.kb0; kb < t.kb1; ++kb) {
      ok = warp_wait(L.full + 8 * stage, phase, abort, p.status);
      if (!ok) break;
      const int left = t.k_end - kb * kBK;
      const int steps = end_of_group<BN, true>(p, L.stages + stage * C::STAGE_BYTES, left, lane);
      if (lane == 0) {
        const uint32_t bar = mapa_shared(L.peer_full + 8 * stage, 0);
        if (steps < kBK / 16 || left < kBK)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
        else
          mbar_arrive_remote(bar);
      }
      __syncwarp();
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

__device__ __forceinline__ void st_shared_f4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// The bias of the warp's columns col .. col + n - 1 (and, for SwiGLU, of their up
// columns) into shared memory as FP32, zeros past the last column.
__device__ __forceinline__ void stage_bias(const LinearEpilogue& p, uint32_t to, int g, int col, int n, int lane) {
  __syncwarp();  // the reads of the tile before are done
  if (4 * lane < n) {
    const int c = col + 4 * lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && p.act != kActSwiglu) break;
      uint32_t f[4] = {};
      const int64_t at = (int64_t)g * p.wide + h * p.N + c;
      if (c < p.N) {
        if (p.bias_type == kTypeF32) {
          const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p.bias) + at);
          f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.bias) + at);
          float a, b;
          unpack2(p.bias_type, v.x, a, b), f[0] = __float_as_uint(a), f[1] = __float_as_uint(b);
          unpack2(p.bias_type, v.y, a, b), f[2] = __float_as_uint(a), f[3] = __float_as_uint(b);
        }
      }
      st_shared_f4(to + h * 512 + lane * 16, f[0], f[1], f[2], f[3]);
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void add_bias(uint32_t at, float (&z)[kChunk]) {
#pragma unroll
  for (int i = 0; i < kChunk / 4; ++i) {
    const float4 b = ld_shared_f4(at + 16 * i);
    z[4 * i] += b.x, z[4 * i + 1] += b.y, z[4 * i + 2] += b.z, z[4 * i + 3] += b.w;
  }
}

// Columns of the warp's rows, zeros where nothing was added up.
template <int W>
__device__ __forceinline__ void read_columns(bool some, uint32_t at, float (&f)[W]) {
  uint32_t v[W];
  if (some) {
    tmem_load_cols(at, v);
    tmem_load_wait();
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    asm volatile("" : "+r"(v[i]));  // no use moves above the wait
    f[i] = some ? __uint_as_float(v[i]) : 0.f;
  }
}

template <int BN, bool SPLIT, bool PAIR>
__device__ void epilogue_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN, PAIR>;
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const bool pairs = p.ep.act == kActSwiglu;
  const int cols = pairs ? BN / 4 : BN / 2;  // output columns of this warp
  const uint32_t bias = L.bias + (warp - kEpiWarp0) * kBiasBytes;
  // a pair's accumulators are free when both CTAs have read them: the first CTA's barrier counts
  const uint32_t acc_empty = PAIR && cluster_ctarank() ? mapa_shared(L.acc_empty, 0) : L.acc_empty;
  uint32_t buf = 0, phase = 0;
  Walk<SPLIT, PAIR> walk(p, L.first_tile, BN);
  Tile t;
  while (walk.next(t)) {
    const bool some = t.kb0 != t.kb1;
    if (!SPLIT && p.ep.bias) stage_bias(p.ep, bias, t.g, t.n0 + half * cols, cols, lane);
    if (some && !warp_wait(L.acc_full + 8 * buf, phase, abort, p.status)) break;
    tc_fence_after();
    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + half * cols;
    if constexpr (SPLIT) {  // the range's sums, a row of the tile per thread, for the join
      const uint32_t to = L.stages + ((quarter * 32 + lane) * (BN + 4) + half * (BN / 2)) * 4;
#pragma unroll
      for (int c = 0; c < BN / 2; c += 32) {
        float f[32];
        read_columns(some, tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + half * (BN / 2) + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_f4(to + c * 4 + 16 * i, __float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                       __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
      }
      break;  // one tile
    }
#pragma unroll 1
    for (int c = 0; c < cols; c += kChunk) {
      const int col = t.n0 + half * cols + c;
      uint32_t r[kChunk / 2];
      const bool mine = quarter * 32 + lane < t.rows && col < p.N;
      const int64_t row = t.out_row + quarter * 32 + lane;
      if (mine && p.ep.residual) load_row(p.ep.residual, row * p.ep.ld_residual + col, p.ep.residual_v8, p.N - col, r);
      float z[kChunk];
      read_columns(some, from + c, z);
      if (p.ep.bias) add_bias(bias + 4 * c, z);
      if (pairs) {
        float u[kChunk];
        read_columns(some, from + BN / 2 + c, u);
        if (p.ep.bias) add_bias(bias + 512 + 4 * c, u);
        if (mine && p.ep.preact) {
          store_row(p.ep.preact, row * p.ep.ld_preact + col, p.ep.type, p.ep.preact_v8, p.N - col, z);
          store_row(p.ep.preact, row * p.ep.ld_preact + p.N + col, p.ep.type, p.ep.preact_v8, p.N - col, u);
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) z[i] = swiglu(z[i], u[i], p.ep.gate_limit, p.ep.up_limit);
      } else {
        if (mine && p.ep.preact)
          store_row(p.ep.preact, row * p.ep.ld_preact + col, p.ep.type, p.ep.preact_v8, p.N - col, z);
        activate_all(p.ep.act, z);
      }
      if (some && c + kChunk >= cols) {  // everything is in registers: the accumulator is free
        tc_fence_before();
        __syncwarp();
        if (PAIR && acc_empty != L.acc_empty) {
          if (lane == 0) mbar_arrive_remote(acc_empty + 8 * buf);
        } else {
          arrive_if(lane == 0, L.acc_empty + 8 * buf);
        }
      }
      if (!mine) continue;
      if (p.ep.residual) {
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
          float a, b;
          unpack2(p.ep.type, r[i], a, b);
          z[2 * i] += a, z[2 * i + 1] += b;
        }
      }
      store_row(p.ep.out, row * p.ep.ld_out + col, p.ep.out_type, p.ep.out_v8, p.N - col, z);
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
  Walk<true, false> walk(p, L.first_tile, BN);
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
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v[kMaxSplit];
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < p.split) v[q] = ld_shared_cluster_v4(mapa_shared(L.stages + (r * (BN + 4) + at + 4 * h) * 4, q));
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < p.split) {
            s[4 * h] += __uint_as_float(v[q].x);
            s[4 * h + 1] += __uint_as_float(v[q].y);
            s[4 * h + 2] += __uint_as_float(v[q].z);
            s[4 * h + 3] += __uint_as_float(v[q].w);
          }
      }
    };
    add(z, c);
    if (pairs) add(u, BN / 2 + c);
    finish8(p.ep, t.out_row + r, col, z, u, b, bu);
  }
}

// first_tile[g]: m-tiles before group g.
template <int UNIT>
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
    const int c = base + lane < p.G ? (p.counts[base + lane] + UNIT - 1) / UNIT : 0;
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

template <int BN, bool SPLIT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) linear_gemm_kernel(const __grid_constant__ LinearArgs p) {
  using C = Cfg<BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  const Smem L = carve<BN, PAIR>(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(L.full + 8 * s, 1);
      mbar_init(L.empty + 8 * s, 1);
      mbar_init(L.peer_full + 8 * s, 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(L.acc_full + 8 * b, 1);
      mbar_init(L.acc_empty + 8 * b, PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    *L.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.map_a);
    prefetch_tmap(&p.map_b);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(L.tmem_slot), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(L.tmem_slot), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  pdl_wait();
  count_tiles<C::UNIT_ROWS>(p, L.first_tile);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers are initialised, their TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  if (warp == 0) load_loop<BN, SPLIT, PAIR>(p, L);
  if (warp == 1) {
    if (PAIR && cluster_ctarank() != 0)
      relay_loop<BN>(p, L);
    else
      mma_loop<BN, SPLIT, PAIR>(p, L, tmem);
  }
  if (warp >= kEpiWarp0) epilogue_loop<BN, SPLIT, PAIR>(p, L, tmem);
  __syncwarp();
  if constexpr (SPLIT) {
    cluster_sync_all();
    if (warp >= kEpiWarp0) join_ranges<BN>(p, L);
    __syncwarp();
    cluster_arrive_relaxed();  // the other CTAs' reads of this one's shared memory
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // neither frees TMEM or leaves while the other may still touch it
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, bool SPLIT, bool PAIR>
cudaError_t configure() {
  static PerDevice<char, cudaError_t> done;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  const char* none = nullptr;
  return done.get(dev, &none, [](char&) {
    return cudaFuncSetAttribute(linear_gemm_kernel<BN, SPLIT, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Cfg<BN, PAIR>::SMEM);
  });
}

template <int BN, bool PAIR>
cudaError_t launch(LinearArgs& p, int slots, cudaStream_t s) {
  using C = Cfg<BN, PAIR>;
  const int out_cols = p.ep.act == kActSwiglu ? BN / 2 : BN;
  p.m_tiles = (p.M + C::UNIT_ROWS - 1) / C::UNIT_ROWS;
  p.n_tiles = (p.N + out_cols - 1) / out_cols;
  p.second = p.ep.act == kActSwiglu ? p.N : BN / 2;
  cudaError_t e;
  if constexpr (BN < 256) {
    if (p.split > 1) {
      if ((e = configure<BN, true, false>()) != cudaSuccess) return e;
      return launch_split<const LinearArgs>(linear_gemm_kernel<BN, true, false>, p.m_tiles * p.n_tiles * p.split,
                                            kThreads, C::SMEM, p.split, s, p);
    }
  }
  if ((e = configure<BN, false, PAIR>()) != cudaSuccess) return e;
  // groups by rows: at most one tile more than the rows' for each
  const int64_t m = p.by_k ? (int64_t)p.G * p.m_tiles : p.counts ? (int64_t)p.m_tiles + p.G : p.m_tiles;
  const int64_t tiles = m * p.n_tiles;
  const int grid = (int)(tiles < slots ? tiles : slots);
  if (PAIR)
    return launch_split<const LinearArgs>(linear_gemm_kernel<BN, false, PAIR>, 2 * grid, kThreads, C::SMEM, 2, s, p);
  return launch_kernel(linear_gemm_kernel<BN, false, PAIR>, dim3(grid), dim3(kThreads), C::SMEM, s, true, p);
}

// Clusters of the split and of the pair form that the GPU holds at a time.
struct Fit {
  Clusters split, pair;
};
cudaError_t clusters_that_fit(const Fit** out) {
  static PerDevice<Fit, cudaError_t> fit;  // one CTA a SM in all forms
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  return fit.get(dev, out, [](Fit& f) {
    if (const cudaError_t e = configure<128, true, false>()) return e;
    if (const cudaError_t e = configure<256, false, true>()) return e;
    if (const cudaError_t e = max_clusters(linear_gemm_kernel<128, true, false>, kThreads, Cfg<128, false>::SMEM, f.split))
      return e;
    return max_clusters(linear_gemm_kernel<256, false, true>, kThreads, Cfg<256, true>::SMEM, f.pair);
  });
}

}  // namespace

// The plan whose K-blocks take least time, as for the FP8 linear: columns of a
// tile by its rounds of tiles over the SMs, and where there is one round with SMs to
// spare, CTAs that share a tile's K.
cudaError_t linear_gemm_plan(LinearArgs& p, int num_sms) {
  const Fit* fit = nullptr;
  const cudaError_t e = clusters_that_fit(&fit);
  if (e != cudaSuccess) return e;
  struct Form {
    int bn, pair, ns, tile_ns, join_ns;
  };
  constexpr Form kForms[4] = {{256, 1, 300, 1500, 0}, {256, 0, 330, 1500, 0}, {128, 0, 190, 1000, 3000}, {64, 0, 140, 800, 2000}};
  const bool pairs = p.ep.act == kActSwiglu;
  const int64_t k = p.counts && p.by_k ? (p.K + p.G - 1) / p.G : p.K;  // of a group, on average
  const int64_t kbs = (k + kBK - 1) / kBK;
  int64_t least = INT64_MAX;
  for (const Form& f : kForms) {
    const int rows = f.pair ? 2 * kBM : kBM, out_cols = pairs ? f.bn / 2 : f.bn;
    const int64_t slots = f.pair ? fit->pair.most[2] : num_sms;
    if (slots == 0) continue;
    // rows of groups: half a tile more for each
    const int64_t mt = p.by_k ? (int64_t)p.G * ((p.M + rows - 1) / rows)
                              : (p.M + rows - 1) / rows + (p.counts ? (p.G + 1) / 2 : 0);
    const int64_t tiles = mt * ((p.N + out_cols - 1) / out_cols);
    for (int c = 1; c <= (f.bn < 256 && !p.counts ? kMaxSplit : 1) && c <= kbs; ++c) {
      if (c > 1 && (tiles * c > num_sms || tiles > fit->split.most[c])) continue;
      const int64_t ns = (tiles * c + slots - 1) / slots * ((kbs + c - 1) / c * f.ns + f.tile_ns) + (c > 1 ? f.join_ns : 0);
      if (ns < least) least = ns, p.bn = f.bn, p.pair = f.pair, p.split = c;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_linear_gemm(LinearArgs& p, int num_sms, cudaStream_t s) {
  if (p.pair) {
    const Fit* fit = nullptr;
    const cudaError_t e = clusters_that_fit(&fit);
    return e != cudaSuccess ? e : launch<256, true>(p, fit->pair.most[2], s);
  }
  return p.bn == 256   ? launch<256, false>(p, num_sms, s)
         : p.bn == 128 ? launch<128, false>(p, num_sms, s)
                       : launch<64, false>(p, num_sms, s);
}

}  // namespace nvfp4
