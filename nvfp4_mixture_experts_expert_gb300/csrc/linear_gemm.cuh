// 16-bit matrix products on the 5th-generation tensor cores with bias, activation
// and residual in the epilogue, over one matrix or over groups of rows (see
// nvfp4_linear and nvfp4_linear_grad):
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
// behind the group's last are set to zero in the ring before the product.  CTA pairs on
// groups by rows run turned (TURN): w is the M operand and the group's rows the N one,
// whose length an instruction takes in steps of 32 where M is always 256, so the tiles
// of a group share its rows evenly.  A lane of the accumulator is then an output column,
// and the epilogue turns it through shared memory.  32 groups of 300 rows, 4096 x 4096:
// 260 us instead of 315, 48 skewed ones of 1024 on average 932 instead of 970.
//
// Persistent, tiles of 128 x BN, FP32 accumulators in TMEM, two of them, so that a
// tile's epilogue runs beside the next one's products.  Large problems run as CTA
// pairs (cta_group::2): 256 x 256 tiles, each CTA with its 128 rows of A and half of B,
// both CTAs' copies counted on the issuing CTA's barrier.  Where a problem has few
// tiles, K is split over the CTAs of a cluster, which add their sums through shared
// memory.  10 warps: 0 TMA, 1 MMA issue (and TMEM), 2 to 9 epilogue (a lane quarter
// and half of the columns each).  Every wait is bounded and reports in the
// library's status word.
//
// Bound: the tensor pipe, then power.  8192 x 4096 x 4096 takes 144 us in a short row
// of calls (1.91 PFLOP/s; tensor pipe 91 % busy; torch.mm 140) and 164 over seconds
// (torch.mm 158), with bias and residual 152 and 174.  What made the difference, from 234 us:
//   - pairs (163 us): a CTA alone copies 48 KB and its MMAs read 48 KB of shared memory a
//     K-block, which is more than the 512 cycles of its products carry (385 ns a block
//     instead of 310);
//   - the next stage's barrier asked while this stage's products are issued (152), the
//     second CTA's copies counted directly instead of relayed by a warp (148), a wait that
//     sleeps in the epilogue;
//   - tiles in bands (144);
//   - an epilogue thread that keeps a row's 16 or 32 columns and stores whole 32-byte
//     sectors; spilled registers cost most where an output is large (8192 x 8192 x 64:
//     174 us with them, 38 without; 4 TB/s of writes, what a fill of memory reaches).  Left
//     are 20 bytes of stores and 44 of loads a thread in the pairs without an activation.
// Built and not faster: the output through shared memory and bulk copies (42 to 49 us
// there), two K-blocks a stage for pairs, the producer asking ahead as well.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8_mma.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace linear_gemm {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kMaxGroups = 256;
constexpr int kBiasBytes = 2 * 128 * 4;    // an epilogue warp's: the bias of up to 128 columns, SwiGLU of both halves
constexpr int kTurnTokens = 16;            // tokens that a warp turns at a time, 32 columns of each:
constexpr int kTurnPitch = 36;             // floats a token, so that eight lanes' 16 bytes meet no bank twice
constexpr int kTurnBytes = kTurnTokens * kTurnPitch * 4;
constexpr int kChunkBytes = 64 * 128;      // 64 columns x 64 rows of an operand read along columns

template <int BN, bool PAIR, bool TURN = false>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK * 2;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // of B that this CTA holds
  static constexpr int BLOCK_BYTES = A_BYTES + B_ROWS * kBK * 2;  // a K-block's operands
  // K-blocks of a ring stage: with two, a small tile's stage takes longer than its waits
  // and issue (128 columns 250 ns a block instead of 275, 64 190 instead of 245); pairs lose
  static constexpr int BLOCKS = BN == 256 ? 1 : 2;
  static constexpr int STAGE_BYTES = BLOCKS * BLOCK_BYTES;
  static constexpr int STAGES = PAIR ? 6 : BN == 64 ? 4 : BN == 128 ? 3 : 4;
  static constexpr int UNIT_ROWS = PAIR ? 2 * kBM : kBM;  // of a tile
  static constexpr int BUFS = 2;
  static constexpr int TMEM_COLS = BUFS * BN;
  static constexpr int EPI_BYTES = TURN ? kTurnBytes : kBiasBytes;  // of an epilogue warp
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + kEpiWarps * EPI_BYTES +
                                 8 * (2 * STAGES + 2 * BUFS) + 16 + 4 * (3 * kMaxGroups + 4);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// Shared-memory addresses: ring, bias, barriers (full: a stage has landed;
// empty: its products are done; acc_full, acc_empty: an accumulator), the groups'
// tables.
struct Smem {
  uint32_t stages, bias, full, empty, acc_full, acc_empty;
  uint32_t* tmem_slot;
  int* abort_flag;
  int* first_tile;  // [G + 1], in m-tiles
  int *first_row, *rows;  // [G], of the groups: read by every role for every tile
};

template <int BN, bool PAIR, bool TURN>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
  using C = Cfg<BN, PAIR, TURN>;
  Smem s;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.stages = smem_u32(base);
  s.bias = s.stages + C::STAGES * C::STAGE_BYTES;
  s.full = s.bias + kEpiWarps * C::EPI_BYTES;
  s.empty = s.full + 8 * C::STAGES;
  s.acc_full = s.empty + 8 * C::STAGES;
  s.acc_empty = s.acc_full + 8 * C::BUFS;
  s.tmem_slot = reinterpret_cast<uint32_t*>(base + (s.acc_empty + 8 * C::BUFS - s.stages));
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  s.first_tile = s.abort_flag + 1;
  s.first_row = s.first_tile + kMaxGroups + 1;
  s.rows = s.first_row + kMaxGroups;
  return s;
}

// This CTA's part of a tile: its group, where its operands start, how many of its
// rows exist (none, or less, where a pair's second half begins behind them), and its
// contraction (K-blocks kb0 .. kb1 of this CTA; k0: first row with by_k; k_end: length).
struct Tile {
  int g, m0, n0, rows, kb0, kb1, k0, k_end;
  int tokens;  // TURN: that the tile's products cover
  int64_t out_row;
};

// Walks the tiles of a role in its order; tiles of a group are neighbours.  Within it
// bands of p.band m-tiles, in each of which m runs fastest: the CTAs at work then read
// about as many rows of A as of B (8192 x 4096 x 4096 read 470 MB of memory with one
// band, of 168 that the product needs).
template <bool SPLIT, bool PAIR, bool SWIGLU, bool TURN = false>
struct Walk {
  static constexpr int UNIT = PAIR ? 2 * kBM : kBM;
  const LinearArgs& p;
  const Smem& L;
  int it, step, rank, g = 0;
  int out_cols;  // columns of the output that a tile covers
  __device__ Walk(const LinearArgs& p, const Smem& L, int bn)
      : p(p), L(L), out_cols(SWIGLU ? bn / 2 : bn) {
    it = SPLIT ? blockIdx.x / p.split : PAIR ? blockIdx.x / 2 : blockIdx.x;
    rank = SPLIT ? blockIdx.x % p.split : PAIR ? blockIdx.x % 2 : 0;
    step = SPLIT ? 1 << 30 : PAIR ? gridDim.x / 2 : gridDim.x;
  }
  // Tile r of `mt` rows of tiles: its row and column.
  __device__ __forceinline__ void place(int r, int mt, int& m, int& n) const {
    const int band = r / (p.band * p.n_tiles), first = band * p.band, size = min(p.band, mt - first);
    r -= first * p.n_tiles;
    n = r / size;
    m = first + r - n * size;
  }
  __device__ bool next(Tile& t) {
    const int m_total = p.by_k ? p.G * p.m_tiles : L.first_tile[p.G];
    if (it >= m_total * p.n_tiles) return false;
    if (p.by_k) {
      const int per = p.m_tiles * p.n_tiles;
      g = it / per;
      int m, n;
      place(it - g * per, p.m_tiles, m, n);
      t.m0 = m * UNIT + (PAIR ? rank * kBM : 0);
      t.n0 = n * out_cols;
      t.rows = min(kBM, p.M - t.m0);
      t.out_row = (int64_t)g * p.M + t.m0;
      t.k0 = L.first_row[g];
      t.k_end = L.rows[g];
    } else {
      while (it >= L.first_tile[g + 1] * p.n_tiles) ++g;
      int m, n;
      place(it - L.first_tile[g] * p.n_tiles, L.first_tile[g + 1] - L.first_tile[g], m, n);
      if constexpr (TURN) {  // the group's tiles share its rows evenly, in steps of 32
        const int mt = L.first_tile[g + 1] - L.first_tile[g];
        t.tokens = (L.rows[g] + 32 * mt - 1) / (32 * mt) * 32;
        m *= t.tokens;
      } else {
        m = m * UNIT + (PAIR ? rank * kBM : 0);
      }
      t.m0 = m + L.first_row[g];
      t.n0 = n * out_cols;
      t.rows = min(TURN ? t.tokens : kBM, L.rows[g] - m);
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

// Boxes into this CTA's shared memory.  PAIR: the barrier is the first CTA's (a
// cluster address), which counts what lands in both.
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    tma_load_2d(dst, map, x, y, bar);
}
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                         uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
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

// The operands of the K-block from k on.
template <int BN, bool PAIR, bool SWIGLU, bool TURN>
__device__ __forceinline__ void load_block(const LinearArgs& p, const Tile& t, int rank, uint32_t a, int k,
                                           uint32_t bar) {
  using C = Cfg<BN, PAIR>;
  const uint32_t b = a + C::A_BYTES;
  if constexpr (TURN) {
    const int n0 = t.n0 + rank * (SWIGLU ? kBM / 2 : kBM);
    if (p.b_mn) {
#pragma unroll
      for (int i = 0; i < kBM / 64; ++i) load_box<PAIR>(a + i * kChunkBytes, &p.map_a, n0 + 64 * i, k, t.g, bar);
    } else if (SWIGLU) {  // 64 rows of the gate, and their 64 of the up half
      load_box<PAIR>(a, &p.map_a, k, n0, t.g, bar);
      load_box<PAIR>(a + kChunkBytes, &p.map_a, k, p.N + n0, t.g, bar);
    } else {
      load_box<PAIR>(a, &p.map_a, k, n0, t.g, bar);
    }
    load_box<PAIR>(b, &p.map_b, k, t.m0 + rank * (t.tokens / 2), bar);
    return;
  }
  if (p.a_mn) {
#pragma unroll
    for (int i = 0; i < kBM / 64; ++i) load_box<PAIR>(a + i * kChunkBytes, &p.map_a, t.m0 + 64 * i, k, bar);
  } else {
    load_box<PAIR>(a, &p.map_a, k, t.m0, bar);
  }
  if (p.b_mn) {
    const int g = p.by_k ? 0 : t.g, n0 = t.n0 + (PAIR ? rank * C::B_ROWS : 0);
#pragma unroll
    for (int i = 0; i < C::B_ROWS / 64; ++i) load_box<PAIR>(b + i * kChunkBytes, &p.map_b, n0 + 64 * i, k, g, bar);
  } else if (PAIR) {
    load_box<PAIR>(b, &p.map_b, k, t.n0 + rank * p.second, t.g, bar);
  } else {
    load_box<PAIR>(b, &p.map_b, k, t.n0, t.g, bar);
    if (SWIGLU) load_box<PAIR>(b + BN * kBK, &p.map_b, k, t.n0 + p.second, t.g, bar);
  }
}

template <int BN, bool SPLIT, bool PAIR, bool SWIGLU, bool TURN>
__device__ void load_loop(const LinearArgs& p, const Smem& L) {
  using C = Cfg<BN, PAIR, TURN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  Walk<SPLIT, PAIR, SWIGLU, TURN> walk(p, L, BN);
  const uint32_t full0 = PAIR ? mapa_shared(L.full, 0) : L.full;
  Tile t;
  while (ok && !*abort && walk.next(t)) {
    const int kb1 = p.stall && t.kb1 > t.kb0 ? t.kb0 + 1 : t.kb1;
    for (int kb = t.kb0; kb < kb1; kb += C::BLOCKS) {
      ok = warp_wait(L.empty + 8 * stage, phase ^ 1u, abort, p.status);
      if (!ok) break;
      if (leader) {
        const uint32_t bar = full0 + 8 * stage;
        const int blocks = min(C::BLOCKS, kb1 - kb);
        const uint32_t at = L.stages + stage * C::STAGE_BYTES;
        if (!PAIR || walk.rank == 0)
          mbar_arrive_expect_tx(L.full + 8 * stage, (PAIR ? 2 : 1) * blocks * C::BLOCK_BYTES);
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i)
          if (i < blocks)
            load_block<BN, PAIR, SWIGLU, TURN>(p, t, walk.rank, at + i * C::BLOCK_BYTES, t.k0 + (kb + i) * kBK, bar);
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
  // A pair's second CTA, whose barriers are the first's, has them consumed when both
  // meet at the end, or gives them time.
  if (PAIR && walk.rank != 0) {
    if (!ok || *abort) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s)
      if (issued & (1u << s)) {
        volatile int no_abort = 0;
        if (!wait_bounded(L.full + 8 * s, (issued_parity >> s) & 1u, &no_abort, nullptr, kDrainNs)) break;
      }
  }
  __syncwarp();
}

// A group's last K-block with by_k, behind which the next group's rows follow: sets
// them to zero up to a multiple of 16 (in both operands: what lies there may be
// infinite); returns the steps of 16 that count.
template <int BN>
__device__ __forceinline__ int end_of_group(uint32_t at, int left, int lane) {
  for (int r = left + (lane >> 3); r < ((left + 15) & ~15); r += 4) {
#pragma unroll
    for (int c = 0; c < kBM / 64 + BN / 64; ++c)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + c * kChunkBytes + r * 128 + (lane & 7) * 16),
                   "r"(0)
                   : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
  return (left + 15) / 16;
}

template <int BN, bool SPLIT, bool PAIR, bool SWIGLU, bool TURN>
__device__ void mma_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN, PAIR, TURN>;
  volatile int* abort = L.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  const int a_mn = TURN ? p.b_mn : p.a_mn, b_mn = TURN ? 0 : p.b_mn;
  uint32_t idesc = idesc_f16(p.ep.type, a_mn, b_mn, C::UNIT_ROWS, BN);
  // by rows: 8-row groups 1024 bytes apart; along columns: the same for 8 of K, 64-column chunks kChunkBytes apart
  const uint64_t a0 = smem_desc(L.stages, a_mn ? kChunkBytes : 16, 1024, 2);
  const uint64_t b0 = smem_desc(L.stages + C::A_BYTES, b_mn ? kChunkBytes : 16, 1024, 2);
  const uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;  // 16 of K
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1, last = 0, last_phase = 0;
  bool issued = false, ok = true, ready = false;
  const bool ends = !PAIR && p.by_k && p.counts;  // not planned as pairs
  Walk<SPLIT, PAIR, SWIGLU, TURN> walk(p, L, BN);
  Tile t;
  while (ok && walk.next(t)) {
    if (t.kb0 == t.kb1) continue;  // nothing to add up: the epilogue takes zeros
    ok = warp_wait(L.acc_empty + 8 * buf, buf_phase, abort, p.status);
    if (!ok) break;
    if constexpr (TURN) idesc = idesc_f16(p.ep.type, a_mn, b_mn, C::UNIT_ROWS, t.tokens);
    const uint32_t d = tmem + buf * BN;
    for (int kb = t.kb0; kb < t.kb1; kb += C::BLOCKS) {
      if (!ready) {
        ok = warp_wait(L.full + 8 * stage, phase, abort, p.status);
        if (!ok) break;
      }
      const int blocks = min(C::BLOCKS, t.kb1 - kb);
      int steps = kBK / 16;  // of the last block
      if (ends) {
        const int at = kb + blocks - 1, left = t.k_end - at * kBK;
        if (left < kBK)
          steps = end_of_group<BN>(L.stages + stage * C::STAGE_BYTES + (blocks - 1) * C::BLOCK_BYTES, left, lane);
      }
      tc_fence_after();
      const uint32_t now = stage;
      last = stage;
      last_phase = phase;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      // whether the next stage is there, asked while this one's products are issued
      const uint32_t next = mbar_test_wait(L.full + 8 * stage, phase);
      if (leader) {
        const uint64_t ad = a0 + (uint64_t)now * (C::STAGE_BYTES >> 4);
        const uint64_t bd = b0 + (uint64_t)now * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < C::BLOCKS; ++j)
          if (j < blocks) {
            const uint32_t block = j * (C::BLOCK_BYTES >> 4);
#pragma unroll
            for (int i = 0; i < kBK / 16; ++i)
              if (j + 1 < blocks || i < steps)
                tc_mma_f16<PAIR>(d, ad + block + i * a_step, bd + block + i * b_step, idesc,
                                 kb != t.kb0 || i != 0 || j != 0);
          }
        const bool done = kb + C::BLOCKS >= t.kb1;
        if constexpr (PAIR) {
          tc_commit_pair_mc(L.empty + 8 * now, 3);
          if (done) tc_commit_pair_mc(L.acc_full + 8 * buf, 3);
        } else {
          tc_commit(L.empty + 8 * now);
          if (done) tc_commit(L.acc_full + 8 * buf);
        }
      }
      ready = __all_sync(0xffffffffu, next);
      issued = true;
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
__device__ __forceinline__ void st_shared_u32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <int W>
__device__ __forceinline__ void get_cols(uint32_t at, float (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 v = ld_shared_f4(at + 4 * i);
    f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
  }
}

// The bias of the warp's columns col .. col + n - 1 (and, for SwiGLU, of their up
// columns) into shared memory as FP32, zeros past the last column.
template <bool SWIGLU>
__device__ __forceinline__ void stage_bias(const LinearEpilogue& p, uint32_t to, int g, int col, int n, int lane) {
  __syncwarp();  // the reads of the tile before are done
  if (4 * lane < n) {
    const int c = col + 4 * lane;
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
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
template <int W>
__device__ __forceinline__ void add_bias(uint32_t at, float (&z)[W]) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
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

template <int BN, bool SPLIT, bool PAIR, int EPI>
__device__ void epilogue_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN, PAIR>;
  constexpr bool SWIGLU = EPI == kEpiSwiglu;
  constexpr int COLS = SWIGLU ? BN / 4 : BN / 2;               // output columns of this warp
  constexpr int W = EPI == kEpiPlain && COLS >= 32 ? 32 : 16;  // held at a time
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const uint32_t bias = L.bias + (warp - kEpiWarp0) * kBiasBytes;
  const LinearEpilogue& ep = p.ep;
  const int type = ep.type, out_type = ep.out_type, out_size = out_type == kTypeF32 ? 4 : 2;
  // a pair's accumulators are free when both CTAs have read them: the first CTA's barrier counts
  const uint32_t acc_empty = PAIR && cluster_ctarank() ? mapa_shared(L.acc_empty, 0) : L.acc_empty;
  uint32_t buf = 0, phase = 0;
  Walk<SPLIT, PAIR, SWIGLU> walk(p, L, BN);
  Tile t;
  while (walk.next(t)) {
    const bool some = t.kb0 != t.kb1;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN;
    if constexpr (SPLIT) {  // the range's sums, a row of the tile per thread, for the join
      if (some && !warp_wait_asleep(L.acc_full + 8 * buf, phase, abort, p.status)) break;
      tc_fence_after();
      const uint32_t to = L.stages + ((quarter * 32 + lane) * (BN + 4) + half * (BN / 2)) * 4;
#pragma unroll
      for (int c = 0; c < BN / 2; c += 32) {
        float f[32];
        read_columns(some, lanes + half * (BN / 2) + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_f4(to + c * 4 + 16 * i, __float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                       __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
      }
      break;  // one tile
    }
    const int n0 = t.n0 + half * COLS;
    const int left = quarter * 32 + lane < t.rows ? p.N - n0 : 0;  // columns that this thread's row has from n0 on
    const int64_t row = t.out_row + quarter * 32 + lane;
    uint8_t* out = static_cast<uint8_t*>(ep.out) + (row * ep.ld_out + n0) * out_size;
    const uint8_t* res = static_cast<const uint8_t*>(ep.residual) + (row * ep.ld_residual + n0) * 2;
    uint8_t* pre = static_cast<uint8_t*>(ep.preact) + (row * ep.ld_preact + n0) * 2;
    // the residual's next two pieces are on their way: each alone would add its trip to memory
    uint32_t r0[W / 2], r1[W / 2];
    auto residual = [&](int c, uint32_t(&r)[W / 2]) {
      if (ep.residual && c < COLS && c < left) load_row(res + 2 * c, ep.residual_v8, left - c, r);
    };
    residual(0, r0);
    residual(W, r1);
    if (ep.bias) stage_bias<SWIGLU>(ep, bias, t.g, n0, COLS, lane);
    if (some && !warp_wait_asleep(L.acc_full + 8 * buf, phase, abort, p.status)) break;
    tc_fence_after();
    auto piece = [&](int c, uint32_t(&r)[W / 2]) {
      __syncwarp();
      float z[W], u[SWIGLU ? W : 1];
      read_columns(some, lanes + half * COLS + c, z);
      if constexpr (SWIGLU) read_columns(some, lanes + BN / 2 + half * COLS + c, u);
      if (some && c + W >= COLS) {  // everything is in registers: the accumulator is free
        tc_fence_before();
        __syncwarp();
        if (PAIR && acc_empty != L.acc_empty) {
          if (lane == 0) mbar_arrive_remote(acc_empty + 8 * buf);
        } else {
          arrive_if(lane == 0, L.acc_empty + 8 * buf);
        }
      }
      if (ep.bias) {
        add_bias(bias + 4 * c, z);
        if constexpr (SWIGLU) add_bias(bias + 512 + 4 * c, u);
      }
      if (c >= left) return;
      if (ep.preact) {
        store_row(pre + 2 * c, type, ep.preact_v8, left - c, z);
        if constexpr (SWIGLU) store_row(pre + 2 * (p.N + c), type, ep.preact_v8, left - c, u);
      }
      if constexpr (SWIGLU) {
#pragma unroll
        for (int i = 0; i < W; ++i) z[i] = swiglu(z[i], u[i], ep.gate_limit, ep.up_limit);
      }
      if constexpr (EPI == kEpiActivation) activate_all(ep.act, z);
      if (ep.residual) {
        add_row(type, r, z);
        residual(c + 2 * W, r);
      }
      store_row(out + c * out_size, out_type, ep.out_v8, left - c, z);
    };
    constexpr int PIECES = COLS / W;
#pragma unroll 1
    for (int c = 0; c < PIECES / 2 * 2 * W; c += 2 * W) {
      piece(c, r0);
      piece(c + W, r1);
    }
    if constexpr (PIECES % 2 != 0) piece(COLS - W, r0);
    if (some && ++buf == C::BUFS) {
      buf = 0;
      phase ^= 1u;
    }
  }
  __syncwarp();
}

// The W columns from col on of a token's row, turned, at `from` of shared memory (SwiGLU:
// the up's kTurnBytes behind).
template <int EPI, int W>
__device__ __forceinline__ void finish_turned(const LinearEpilogue& ep, int64_t row, int col, uint32_t from,
                                              const float (&b)[W / 8][8], const float (&bu)[W / 8][8]) {
  constexpr bool SWIGLU = EPI == kEpiSwiglu;
  const int left = ep.N - col, out_size = ep.out_type == kTypeF32 ? 4 : 2;
  float z[W], u[SWIGLU ? W : 1];
  uint32_t r[W / 2];
  if (ep.residual)
    load_row(static_cast<const uint8_t*>(ep.residual) + (row * ep.ld_residual + col) * 2, ep.residual_v8, left, r);
  get_cols(from, z);
  if constexpr (SWIGLU) get_cols(from + kTurnBytes, u);
  if (ep.bias) {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] += b[i / 8][i % 8];
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] += bu[i / 8][i % 8];
    }
  }
  if (ep.preact) {
    uint8_t* to = static_cast<uint8_t*>(ep.preact) + (row * ep.ld_preact + col) * 2;
    store_row(to, ep.type, ep.preact_v8, left, z);
    if constexpr (SWIGLU) store_row(to + 2 * ep.N, ep.type, ep.preact_v8, left, u);
  }
  if constexpr (SWIGLU) {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] = swiglu(z[i], u[i], ep.gate_limit, ep.up_limit);
  }
  if constexpr (EPI == kEpiActivation) activate_all(ep.act, z);
  if (ep.residual) add_row(ep.type, r, z);
  uint8_t* out = static_cast<uint8_t*>(ep.out) + (row * ep.ld_out + col) * out_size;
  store_row(out, ep.out_type, ep.out_v8, left, z);
}

// Whether both warps that share a barrier say so.
__device__ __forceinline__ bool both(bool ok, int barrier) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.and.pred p, %2, 64, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(barrier)
      : "memory");
  return r;
}

// The epilogue of a turned tile: an accumulator's lane is an output column, its columns
// are tokens.  A warp turns 16 tokens of its 32 lanes at a time through shared memory;
// then a lane has 16 columns of a token (SwiGLU, where two warps turn a gate's lanes and
// their up's: eight of each).
template <int BN, int EPI>
__device__ void turned_epilogue_loop(const LinearArgs& p, const Smem& L, uint32_t tmem) {
  using C = Cfg<BN, true, true>;
  constexpr bool SWIGLU = EPI == kEpiSwiglu;
  constexpr int W = SWIGLU ? 8 : 16;  // output columns of a lane
  volatile int* abort = L.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
  // SwiGLU: a gate's warp and its up's share what they turn
  const int with = SWIGLU ? quarter >> 1 : 0, first = half * 4 + (SWIGLU ? quarter % 2 * 2 : quarter);
  const int at = with * 32 + lane, token = at / (32 / W), my_col = at % (32 / W) * W;
  const uint32_t turn = L.bias + first * C::EPI_BYTES;
  const uint32_t to = turn + with * C::EPI_BYTES + lane * 4, from = turn + (token * kTurnPitch + my_col) * 4;
  auto meet = [&] {
    if constexpr (SWIGLU)
      asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + half * 2 + quarter % 2) : "memory");
    else
      __syncwarp();
  };
  const LinearEpilogue& ep = p.ep;
  const uint32_t acc_empty = cluster_ctarank() ? mapa_shared(L.acc_empty, 0) : L.acc_empty;
  uint32_t buf = 0, phase = 0;
  Walk<false, true, SWIGLU, true> walk(p, L, BN);
  Tile t;
  while (walk.next(t)) {
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN;
    const int col = t.n0 + (SWIGLU ? walk.rank * 64 + quarter % 2 * 32 : walk.rank * 128 + quarter * 32) + my_col;
    float b[W / 8][8], bu[W / 8][8];
#pragma unroll
    for (int i = 0; i < W / 8; ++i) load_bias<EPI>(ep, t.g, col + 8 * i, b[i], bu[i]);
    bool ok = warp_wait_asleep(L.acc_full + 8 * buf, phase, abort, p.status);
    if constexpr (SWIGLU) ok = both(ok, 1 + half * 2 + quarter % 2);  // neither waits for one that has left
    if (!ok) break;
    tc_fence_after();
    // the next tokens are on their way from the accumulator while these are stored
    uint32_t v[kTurnTokens];
    auto take = [&](int c) {
      if (c < t.rows) tmem_load_cols(lanes + c, v);
    };
    take(half * kTurnTokens);
    for (int c = half * kTurnTokens;; c += 2 * kTurnTokens) {
      __syncwarp();
      tmem_load_wait();
      if (c >= t.rows) break;
      meet();  // the reads of the tokens before are done
#pragma unroll
      for (int i = 0; i < kTurnTokens; ++i) {
        asm volatile("" : "+r"(v[i]));  // no use moves above the wait
        st_shared_u32(to + i * kTurnPitch * 4, v[i]);
      }
      meet();
      take(c + 2 * kTurnTokens);
      if (c + token < t.rows && col < p.N) finish_turned<EPI, W>(ep, t.out_row + c + token, col, from, b, bu);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (acc_empty != L.acc_empty)
        mbar_arrive_remote(acc_empty + 8 * buf);
      else
        mbar_arrive(acc_empty + 8 * buf);
    }
    if (++buf == C::BUFS) {
      buf = 0;
      phase ^= 1u;
    }
  }
  __syncwarp();
}

// The cluster's CTAs add up the ranges' sums in K order, each its share of the
// tile's rows, four columns a thread.  A thread's columns stay the same from row to row,
// so their bias is loaded once, and two rows' sums and residuals are in flight: what is
// loaded only when it is needed adds its trip to memory (300 x 1000 x 3600: the join 4.1
// us with eight columns and one row at a time, 3.5 so; by bulk copies to the owner of a
// row 2.9, but the call 12.2 instead of 11.0).
template <int BN, int EPI>
__device__ void join_ranges(const LinearArgs& p, const Smem& L) {
  constexpr bool SWIGLU = EPI == kEpiSwiglu;
  constexpr int PER = (SWIGLU ? BN / 2 : BN) / 4, STEP = kEpiWarps * 32 / PER;  // threads a row; rows a step
  static_assert(kEpiWarps * 32 % PER == 0, "whole rows a step");
  Walk<true, false, SWIGLU> walk(p, L, BN);
  Tile t;
  if (!walk.next(t)) return;
  const int tid = threadIdx.x - kEpiWarp0 * 32, c = tid % PER * 4, col = t.n0 + c;
  const int end = col < p.N ? min(kBM * (walk.rank + 1) / p.split, t.rows) : 0;
  float b[4], bu[4];
  load_bias<EPI>(p.ep, t.g, col, b, bu);
  for (int r0 = kBM * walk.rank / p.split + tid / PER; r0 < end; r0 += 2 * STEP) {
    float res[2][4], s[2][SWIGLU ? 2 : 1][4] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (r0 + j * STEP < end) load_residual(p.ep, t.out_row + r0 + j * STEP, col, res[j]);
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
      uint4 v[2][kMaxSplit];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = L.stages + ((r0 + j * STEP) * (BN + 4) + c + h * (BN / 2)) * 4;
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < p.split && r0 + j * STEP < end) v[j][q] = ld_shared_cluster_v4(mapa_shared(at, q));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < p.split) {
            s[j][h][0] += __uint_as_float(v[j][q].x);
            s[j][h][1] += __uint_as_float(v[j][q].y);
            s[j][h][2] += __uint_as_float(v[j][q].z);
            s[j][h][3] += __uint_as_float(v[j][q].w);
          }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (r0 + j * STEP < end)
        finish<EPI>(p.ep, t.out_row + r0 + j * STEP, col, s[j][0], s[j][SWIGLU], b, bu, res[j]);
  }
}

// The groups' tables: first rows, rows, and the m-tiles before each.
template <int UNIT>
__device__ void read_groups(const LinearArgs& p, const Smem& L) {
  if (!p.counts) {
    if (threadIdx.x == 0) {
      L.first_row[0] = 0;
      L.rows[0] = p.by_k ? p.K : p.M;
      L.first_tile[0] = 0;
      L.first_tile[1] = p.m_tiles;
    }
    return;
  }
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int sum = 0;
  for (int base = 0; base < p.G; base += 32) {
    const int g = base + lane, rows = g < p.G ? p.counts[g] : 0, c = (rows + UNIT - 1) / UNIT;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (g < p.G) {
      L.first_row[g] = p.offsets[g];
      L.rows[g] = rows;
      L.first_tile[g] = sum + incl - c;
    }
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) L.first_tile[p.G] = sum;
}

template <int BN, bool SPLIT, bool PAIR, int EPI, bool TURN = false>
__global__ void __launch_bounds__(kThreads, 1) linear_gemm_kernel(const __grid_constant__ LinearArgs p) {
  using C = Cfg<BN, PAIR, TURN>;
  extern __shared__ uint8_t smem_raw[];
  const Smem L = carve<BN, PAIR, TURN>(smem_raw);
  constexpr bool SWIGLU = EPI == kEpiSwiglu;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(L.full + 8 * s, 1);
      mbar_init(L.empty + 8 * s, 1);
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
  if (!p.beside) pdl_wait();
  if (p.before) pdl_trigger();
  read_groups<C::UNIT_ROWS>(p, L);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers are initialised, their TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *L.tmem_slot;
  if (warp == 0) load_loop<BN, SPLIT, PAIR, SWIGLU, TURN>(p, L);
  if (warp == 1 && (!PAIR || cluster_ctarank() == 0)) mma_loop<BN, SPLIT, PAIR, SWIGLU, TURN>(p, L, tmem);
  if (warp >= kEpiWarp0) {
    if constexpr (TURN)
      turned_epilogue_loop<BN, EPI>(p, L, tmem);
    else
      epilogue_loop<BN, SPLIT, PAIR, EPI>(p, L, tmem);
  }
  __syncwarp();
  if (p.beside) pdl_wait();  // this kernel's end is also the end of the one it ran beside
  if constexpr (SPLIT) {
    cluster_sync_all();
    if (warp >= kEpiWarp0) join_ranges<BN, EPI>(p, L);
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

template <int BN, bool SPLIT, bool PAIR, int EPI, bool TURN = false>
cudaError_t configure() {
  static PerDevice<char, cudaError_t> done;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  const char* none = nullptr;
  return done.get(dev, &none, [](char&) {
    return cudaFuncSetAttribute(linear_gemm_kernel<BN, SPLIT, PAIR, EPI, TURN>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN, PAIR, TURN>::SMEM);
  });
}

template <int BN, bool PAIR, int EPI, bool TURN = false>
cudaError_t launch(LinearArgs& p, int slots, cudaStream_t s) {
  using C = Cfg<BN, PAIR, TURN>;
  const int out_cols = EPI == kEpiSwiglu ? BN / 2 : BN;
  p.m_tiles = (p.M + C::UNIT_ROWS - 1) / C::UNIT_ROWS;
  p.n_tiles = (p.N + out_cols - 1) / out_cols;
  p.second = EPI == kEpiSwiglu ? p.N : BN / 2;
  // as many rows as columns at a time: band * UNIT_ROWS = slots / band * BN
  p.band = 1;
  while ((p.band + 1) * (p.band + 1) * C::UNIT_ROWS <= slots * BN) ++p.band;
  cudaError_t e;
  if constexpr (BN < 256) {
    if (p.split > 1) {
      if ((e = configure<BN, true, false, EPI>()) != cudaSuccess) return e;
      return launch_split<const LinearArgs>(linear_gemm_kernel<BN, true, false, EPI>, p.m_tiles * p.n_tiles * p.split,
                                            kThreads, C::SMEM, p.split, s, p);
    }
  }
  if ((e = configure<BN, false, PAIR, EPI, TURN>()) != cudaSuccess) return e;
  // groups by rows: at most one tile more than the rows' for each
  const int64_t m = p.by_k ? (int64_t)p.G * p.m_tiles : p.counts ? (int64_t)p.m_tiles + p.G : p.m_tiles;
  const int64_t tiles = m * p.n_tiles;
  const int grid = (int)(tiles < slots ? tiles : slots);
  if (PAIR)
    return launch_split<const LinearArgs>(linear_gemm_kernel<BN, false, PAIR, EPI, TURN>, 2 * grid, kThreads, C::SMEM,
                                          2, s, p);
  return launch_kernel(linear_gemm_kernel<BN, false, PAIR, EPI>, dim3(grid), dim3(kThreads), C::SMEM, s, true, p);
}

template <int EPI>
cudaError_t launch_form(LinearArgs& p, int slots, cudaStream_t s) {
  if (p.pair && p.turned) return launch<256, true, EPI, true>(p, slots, s);
  if (p.pair) return launch<256, true, EPI>(p, slots, s);
  return p.bn == 256   ? launch<256, false, EPI>(p, slots, s)
         : p.bn == 128 ? launch<128, false, EPI>(p, slots, s)
                       : launch<64, false, EPI>(p, slots, s);
}

}  // namespace linear_gemm

// The launch of a planned product; slots: CTAs, or pairs, that the GPU holds at a time.
cudaError_t launch_linear_plain(LinearArgs& p, int slots, cudaStream_t s);
cudaError_t launch_linear_activation(LinearArgs& p, int slots, cudaStream_t s);
cudaError_t launch_linear_swiglu(LinearArgs& p, int slots, cudaStream_t s);

}  // namespace nvfp4
