// The whole NVFP4 MoE FFN layer for at most 32 tokens.
//
//   ids, p = top-k of the FP32 logits (ties -> lower expert), softmax over the k
//   h_a    = silu(min(g, gate_limit)) * clamp(u, +-up_limit),  g, u = W13[e] x_t
//   out_t  = bf16( sum_j p_tj * W2[e_tj] h_tj ),  j ascending
//
// With so few tokens the layer is a stream of the chosen experts' weights, so
// the activations are not quantized: the product takes the weights' exact
// values.  E2M1 x E4M3 has at most 6 significant bits and lies in
// [2^-10, 2688], so code * block scale is exact in f16 and the weights go
// through mma.sync.m16n8k16 (f16 operands, FP32 accumulation) as the M operand,
// straight from their packed form: the K order inside a slab of 128 is free as
// long as both operands use the same one, so a lane takes 32 consecutive
// weights (16 bytes, two scale blocks) of its rows.  The tokens are the N
// operand, eight at a time: an expert with more of them is listed again for
// the next eight.  A slab of a token's activations is scaled by a power of two
// that puts its largest value at 2^14..2^15 (exact for bf16; 11 bits are kept
// of the FP32 h) and the sum is scaled back in FP32.
//
//
// The 128 x 4 scale tiles keep rows r, r + 32, r + 64, r + 96 in one 16-byte
// line, so the rows of an m16 tile are taken as whole lines: W13, 2 lines of
// gate rows and the same 2 of up rows (8 features; gate in accumulator rows
// 0-7, up in rows 8-15, so a lane holds both of its feature); W2, 4 lines.
//
// Two launches of one kernel, h between them; one CTA per SM, which takes an
// equal share of the (list entry, tile) pairs in order, so that it changes
// expert once or twice.  A tile is R m16 tiles (about 32 KB of packed weights)
// over all of K.  Its warps:
//   16 consumers     KG = 16 / R of them share an m16 tile and split K by slabs;
//                    their activations stay in registers while the entry lasts
//   warp 16          joins the KG sums in a fixed order; SwiGLU, or the weighted
//                    row; the last to add to an output tile sums the experts
//   warp 17          weights: one bulk copy a row into the ring, whose row pitch
//                    (64 mod 128 bytes) makes the consumers' reads conflict-free
//   warp 18          scales: the lines of the tile, 16 bytes a copy
// Every CTA routes for itself (a microsecond, no launch in between).  The second
// launch starts as CTAs of the first leave (programmatic dependent launch) and
// fills its rings before it waits for h, and the first asks for the second's
// first weights to be brought into L2, so HBM does not idle between the two.
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"
#include "route_key.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 16;  // consumers
constexpr int kThreads = 32 * (kWarps + 4);
constexpr int kRegsLaunch = 96;    // per thread; 61,440 of the SM's 65,536 registers
constexpr int kRegsConsumer = 104; // with four slabs a warp: 64 of them activations
constexpr int kRegsOther = 64;
static_assert(128 * (4 * kRegsConsumer + kRegsOther) <= kThreads * kRegsLaunch, "the register split must fit");
constexpr int kMaxStages = 16;
constexpr int kPartBufs = 3;       // tiles whose sums wait to be joined
constexpr int kPrefetch = 6;       // W2 tiles a CTA of the first launch brings into L2
constexpr int kGroup = 8;  // tokens of one list entry

// Routing tables: every (token, expert) assignment a = t * k + j, and the list
// of (expert, up to 8 of its assignments).
struct Route {
  int32_t n_list;
  int32_t pad[3];
  int32_t id[kFewAssignments];  // local expert, -1: not computed
  float weight[kFewAssignments];
  int32_t expert[kFewAssignments];
  int16_t member[kFewAssignments][kGroup];  // assignments of a list entry, -1 past the last
};

__device__ __forceinline__ float clamp_up(float v, float hi) { return v > hi ? hi : v; }  // NaN stays

// One warp per token: lane j < k gets the j-th choice.  An assignment of weight
// 0 (a -inf logit, a zero weight of the caller's) is not computed; a token with
// none left gets a zero row.  An expert named twice is computed once, with the
// sum of the two weights.
__device__ void route_one(const FewArgs& p, int t, int lane, int32_t* s_id, float* s_w, uint32_t* s_mask) {
  int id = -1;
  float w = 0.f;
  if (p.logits) {
    uint64_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < p.E ? route_key(__ldg(p.logits + (int64_t)t * p.E + e), e) : 0ull;
    }
    uint64_t mine = 0ull;
    for (int j = 0; j < p.k; ++j) {
      uint64_t best = key[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) best = key[i] > best ? key[i] : best;
      const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
      const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
      const uint64_t win = ((uint64_t)hi << 32) | lo;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key[i] == win) key[i] = 0ull;
      if (lane == j) mine = win;
    }
    const float top = key_value(__shfl_sync(0xffffffffu, mine, 0));
    float z = 0.f;
    if (lane < p.k) {
      const float l = key_value(mine);
      id = key_expert(mine);
      z = l == -INFINITY ? 0.f : l == top ? 1.f : expf(l - top);
    }
    float sum = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum == 0.f ? 0.f : z / sum;
  } else {
    if (lane < p.k) {
      const int64_t e = (int64_t)__ldg(p.ext_ids + t * p.k + lane) - p.start;
      if (e >= 0 && e < p.E) {
        id = (int)e;
        w = __ldg(p.ext_w + t * p.k + lane);
      }
    }
    float all = 0.f;
    int first = lane;
    for (int j = p.k - 1; j >= 0; --j) {
      const int oid = __shfl_sync(0xffffffffu, id, j);
      const float ow = __shfl_sync(0xffffffffu, w, j);
      if (id >= 0 && oid == id) {
        all = ow + all;
        first = j;
      }
    }
    if (first != lane) id = -1;
    w = all;
  }
  if (lane < p.k) {
    if (w == 0.f) id = -1;
    s_id[t * p.k + lane] = id;
    s_w[t * p.k + lane] = id < 0 ? 0.f : w;
    if (id >= 0) atomicOr(&s_mask[id], 1u << t);
  }
}

// Fills `r` with the block's threads.
__device__ void route_all(const FewArgs& p, Route* r) {
  __shared__ uint32_t s_mask[256];
  __shared__ int32_t s_first[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < 256; e += kThreads) s_mask[e] = 0u;
  for (int i = tid; i < kFewAssignments * kGroup; i += kThreads) (&r->member[0][0])[i] = -1;
  __syncthreads();
  for (int t = warp; t < p.T; t += kThreads / 32) route_one(p, t, lane, r->id, r->weight, s_mask);
  __syncthreads();
  if (warp == 0) {  // list entries of the experts, in expert order
    int n[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = (__popc(s_mask[lane * 8 + i]) + kGroup - 1) / kGroup;
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int at = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s_first[lane * 8 + i] = at;
      at += n[i];
    }
    if (lane == 31) r->n_list = incl;
  }
  __syncthreads();
  for (int a = tid; a < p.T * p.k; a += kThreads) {
    const int e = r->id[a], t = a / p.k;
    if (e < 0) continue;
    const int rank = __popc(s_mask[e] & ((1u << t) - 1u));
    const int v = s_first[e] + rank / kGroup;
    r->expert[v] = e;
    r->member[v][rank % kGroup] = (int16_t)a;
  }
}

// Eight E2M1 codes (one word) times a block scale: four f16 pairs, in order.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t s2, uint32_t (&r)[4]) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\n.reg .b32 t0, t1, t2, t3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 t0, b0;\ncvt.rn.f16x2.e2m1x2 t1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 t2, b2;\ncvt.rn.f16x2.e2m1x2 t3, b3;\n"
      "mul.rn.f16x2 %0, t0, %5;\nmul.rn.f16x2 %1, t1, %5;\nmul.rn.f16x2 %2, t2, %5;\nmul.rn.f16x2 %3, t3, %5;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w), "r"(s2));
}
// Two E4M3 scales -> each as an f16 pair of itself.
__device__ __forceinline__ void scale_pairs(uint32_t codes, uint32_t& s0, uint32_t& s1) {
  uint32_t h;
  asm("{\n.reg .b16 t;\ncvt.u16.u32 t, %1;\ncvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(h) : "r"(codes));
  s0 = __byte_perm(h, h, 0x1010);
  s1 = __byte_perm(h, h, 0x3232);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The lane's 32 weights of two rows (words in K order, the rows' two scales)
// times its 32 activations of one token, over the quad: 128 of K.  Two sums, so
// that a product does not wait for the one before it.
__device__ __forceinline__ void mma_slab(float (&c)[4], float (&d)[4], const uint4& w0, const uint4& w1, uint32_t sc0, uint32_t sc1,
                                         const uint32_t (&b)[16]) {
  uint32_t s[2][2];
  scale_pairs(sc0, s[0][0], s[0][1]);
  scale_pairs(sc1, s[1][0], s[1][1]);
  const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r0[4], r1[4];
    decode8(x0[i], s[0][i >> 1], r0);
    decode8(x1[i], s[1][i >> 1], r1);
    mma_f16(c, r0[0], r1[0], r0[1], r1[1], b[4 * i], b[4 * i + 1]);
    mma_f16(d, r0[2], r1[2], r0[3], r1[3], b[4 * i + 2], b[4 * i + 3]);
  }
}

// Power of two that takes a largest magnitude to [2^14, 2^15), and its inverse
// (magnitudes below 2^-112 stay smaller; inf and NaN go through).
__device__ __forceinline__ float slab_scale(float amax, float& inverse) {
  const int e = amax == 0.f ? 0 : 141 - (int)(__float_as_uint(amax) >> 23);
  const int s = e > 126 ? 126 : e;
  inverse = pow2f(-s);
  return pow2f(s);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float swiglu(float gate, float up, float gate_limit, float up_limit) {
  gate = clamp_up(gate, gate_limit);
  up = -clamp_up(-clamp_up(up, up_limit), up_limit);
  return gate / (1.f + expf(-gate)) * up;
}

// Where row g (and, in W2, row g + 8) of m16 tile `st` lies: feature (phase 0)
// or output column (phase 1).
template <int PHASE>
__device__ __forceinline__ int tile_row(int st, int g) {
  const int i = g >> 2, j = g & 3;
  return PHASE == 0 ? (st >> 4) * 128 + (st & 15) * 2 + i + 32 * j : (st >> 3) * 128 + (st & 7) * 4 + i + 32 * j;
}

// What a launch needs to know of its product (0: W13 x, 1: W2 h).
struct Phase {
  int K, R, KG;      // R m16 tiles a tile, KG = 16 / R warps along K
  int tiles;         // per list entry
  int pitch;         // bytes of a weight row in the ring
  int scale_off;     // of the tile's scales in a ring slot
  int stage_bytes, stages;
};

struct Ring {
  uint32_t slots, part;             // weights and scales of a tile; the warps' sums
  uint32_t full, scales, empty;     // a slot's weights, its scales have landed; it has been read
  uint32_t part_full, part_empty;
  volatile int* abort;
};

// The list entry and tile of unit u.
struct Unit {
  int v, tile;
};
__device__ __forceinline__ Unit unit_at(int u, int tiles) {
  const int v = u / tiles;
  return {v, u - v * tiles};
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// Global row of row m (0-15) of m16 tile st.
template <int PHASE>
__device__ __forceinline__ int weight_row(int st, int m, int I) {
  return tile_row<PHASE>(st, m & 7) + (m < 8 ? 0 : PHASE == 0 ? I : 2);
}

template <int PHASE>
__device__ __forceinline__ const uint8_t* expert_weights(const FewArgs& p, int e, int K) {
  const int64_t rows = PHASE == 0 ? 2 * (int64_t)p.I : p.H;
  return (PHASE == 0 ? p.w13 : p.w2) + e * rows * (K / 2);
}
template <int PHASE>
__device__ __forceinline__ const uint8_t* expert_scales(const FewArgs& p, int e, int K) {
  const int64_t rows = PHASE == 0 ? 2 * (int64_t)p.I : p.H;
  return (PHASE == 0 ? p.sf13 : p.sf2) + e * rows * (K / 16);
}

// ------------------------------------------------------------------ producers
template <int PHASE>
__device__ void weight_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int lane = threadIdx.x & 31, rows = 16 * g.R;
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  for (int u = u0; u < u1; ++u) {
    if (!warp_wait(L.empty + 8 * stage, phase ^ 1u, L.abort, p.status)) {
      // copies in flight land before the CTA leaves its shared memory
      for (int s = 0; s < g.stages; ++s)
        if (lane == 0 && (issued >> s & 1u)) {
          volatile int no_abort = 0;
          wait_bounded(L.full + 8 * s, issued_parity >> s & 1u, &no_abort, nullptr, kDrainNs);
        }
      __syncwarp();
      return;
    }
    const Unit t = unit_at(u, g.tiles);
    const uint8_t* W = expert_weights<PHASE>(p, r->expert[t.v], g.K);
    const uint32_t to = L.slots + stage * g.stage_bytes, bar = L.full + 8 * stage;
    if (lane == 0) mbar_arrive_expect_tx(bar, rows * (g.K / 2));
    __syncwarp();
    for (int i = lane; i < rows; i += 32)
      bulk_load(to + i * g.pitch, W + (int64_t)weight_row<PHASE>(t.tile * g.R + (i >> 4), i & 15, p.I) * (g.K / 2),
                g.K / 2, bar);
    __syncwarp();
    issued |= 1u << stage;
    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
    if (++stage == (uint32_t)g.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

template <int PHASE>
__device__ void scale_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int lane = threadIdx.x & 31, cts = g.K / 64, lines = g.R * cts * 4;
  uint32_t stage = 0, phase = 0;
  for (int u = u0; u < u1; ++u) {
    if (!warp_wait(L.empty + 8 * stage, phase ^ 1u, L.abort, p.status)) break;
    const Unit t = unit_at(u, g.tiles);
    const uint8_t* SF = expert_scales<PHASE>(p, r->expert[t.v], g.K);
    const uint32_t to = L.slots + stage * g.stage_bytes + g.scale_off;
    for (int i = lane; i < lines; i += 32) {
      const int line = i & 3, c = i >> 2, sub = c / cts, ct = c - sub * cts, st = t.tile * g.R + sub;
      const int row = PHASE == 0 ? (line >> 1) * p.I + (st >> 4) * 128 + (st & 15) * 2 + (line & 1)
                                 : (st >> 3) * 128 + (st & 7) * 4 + line;
      const uint8_t* from = SF + ((int64_t)(row >> 7) * cts + ct) * 512 + (row & 31) * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(from) : "memory");
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(L.scales + 8 * stage) : "memory");
    if (++stage == (uint32_t)g.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The first W2 tiles of this CTA's share of the second launch, into L2.
__device__ void prefetch_w2(const FewArgs& p, const Phase& g, const Route* r) {
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)r->n_list * g.tiles;
  const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  for (int u = u0; u < min(u1, u0 + kPrefetch); ++u) {
    const Unit t = unit_at(u, g.tiles);
    const uint8_t* W = expert_weights<1>(p, r->expert[t.v], g.K);
    for (int i = lane; i < 16 * g.R; i += 32)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                       W + (int64_t)weight_row<1>(t.tile * g.R + (i >> 4), i & 15, p.I) * (g.K / 2)),
                   "r"(g.K / 2)
                   : "memory");
  }
}

// ------------------------------------------------------------------ consumers
// This lane's activations of its token (assignment a, -1: none) for the warp's
// slabs, as f16 pairs scaled by one power of two; returns its inverse.
template <int PHASE, int SPW>
__device__ __forceinline__ float load_activations(const FewArgs& p, const Phase& g, int a, int kg, int q,
                                                  uint32_t (&b)[SPW][16]) {
  const int slabs = g.K / 128;
  float amax = 0.f;
  const uint16_t* x = PHASE == 0 ? p.x + (int64_t)(a < 0 ? 0 : a / p.k) * p.ld_x + q * 32 : nullptr;
  const float* h = PHASE == 1 ? p.h + (int64_t)(a < 0 ? 0 : a) * p.I + q * 32 : nullptr;
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const int slab = kg + s * g.KG;
    if (slab >= slabs || a < 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) b[s][i] = 0u;
    } else if (PHASE == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + slab * 128) + i);
        b[s][4 * i] = u.x, b[s][4 * i + 1] = u.y, b[s][4 * i + 2] = u.z, b[s][4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(b[s][i])), fabsf(bf16_hi(b[s][i]))));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(h + slab * 128) + i);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))));
      }
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  float inverse;
  const float scale = slab_scale(amax, inverse);
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const int slab = kg + s * g.KG;
    if (slab >= slabs || a < 0) continue;
    if (PHASE == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) b[s][i] = pack_f16x2(bf16_lo(b[s][i]) * scale, bf16_hi(b[s][i]) * scale);
    } else {  // read again (from L2) rather than held: 32 FP32 values a slab
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(h + slab * 128) + i);
        b[s][2 * i] = pack_f16x2(u.x * scale, u.y * scale);
        b[s][2 * i + 1] = pack_f16x2(u.z * scale, u.w * scale);
      }
    }
  }
  return inverse;
}

template <int PHASE, int SPW>
__device__ void consume_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, q = lane & 3;
  const int kg = warp % g.KG, sub = warp / g.KG, slabs = g.K / 128;
  const uint32_t w_off = (sub * 16 + gr) * g.pitch + q * 16;
  const uint32_t s_off = g.scale_off + sub * g.K + (q >> 1) * 64 + (gr >> 2) * 16 + (gr & 3) * 4 + (q & 1) * 2;
  const uint32_t part = L.part + warp * 512 + lane * 16;
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1;
  uint32_t b[SPW][16];
  float i0 = 0.f, i1 = 0.f, alpha = 0.f;
  int have = -1;
  for (int u = u0; u < u1; ++u) {
    const Unit t = unit_at(u, g.tiles);
    if (t.v != have) {
      have = t.v;
      alpha = 1.f / __ldg((PHASE == 0 ? p.gs13 : p.gs2) + r->expert[t.v]);
      const float inv = load_activations<PHASE, SPW>(p, g, r->member[t.v][gr], kg, q, b);
      i0 = __shfl_sync(0xffffffffu, inv, q * 8);
      i1 = __shfl_sync(0xffffffffu, inv, q * 8 + 4);
    }
    if (!warp_wait(L.scales + 8 * stage, phase, L.abort, p.status) ||
        !warp_wait(L.full + 8 * stage, phase, L.abort, p.status))
      return;
    const uint32_t at = L.slots + stage * g.stage_bytes;
    float c[4] = {}, d[4] = {};
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
      const int slab = kg + s * g.KG;
      if (slab < slabs) {
        const uint4 w0 = lds128(at + w_off + slab * 64), w1 = lds128(at + w_off + 8 * g.pitch + slab * 64);
        const uint32_t s0 = lds16(at + s_off + slab * 128), s1 = lds16(at + s_off + slab * 128 + 32);
        mma_slab(c, d, w0, w1, s0, s1, b[s]);
      }
    }
    __syncwarp();
    arrive_if(lane == 0, L.empty + 8 * stage);
    if (!warp_wait(L.part_empty + 8 * buf, buf_phase, L.abort, p.status)) return;
    // alpha first: neither factor leaves FP32's range
    sts128(part + buf * (kWarps * 512), (c[0] + d[0]) * alpha * i0, (c[1] + d[1]) * alpha * i1,
           (c[2] + d[2]) * alpha * i0, (c[3] + d[3]) * alpha * i1);
    __syncwarp();
    arrive_if(lane == 0, L.part_full + 8 * buf);
    if (++stage == (uint32_t)g.stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (++buf == kPartBufs) {
      buf = 0;
      buf_phase ^= 1u;
    }
  }
}

// ------------------------------------------------------------------ join
template <int PHASE>
__device__ void join_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, q = lane & 3;
  uint32_t buf = 0, phase = 0;
  for (int u = u0; u < u1; ++u) {
    const Unit t = unit_at(u, g.tiles);
    const int a0 = r->member[t.v][2 * q], a1 = r->member[t.v][2 * q + 1];
    if (!warp_wait(L.part_full + 8 * buf, phase, L.abort, p.status)) return;
    for (int sub = 0; sub < g.R; ++sub) {
      const uint32_t from = L.part + buf * (kWarps * 512) + sub * g.KG * 512 + lane * 16;
      float c[4] = {};
      for (int i = 0; i < g.KG; ++i) {
        const uint4 v = lds128(from + i * 512);
        c[0] += __uint_as_float(v.x), c[1] += __uint_as_float(v.y);
        c[2] += __uint_as_float(v.z), c[3] += __uint_as_float(v.w);
      }
      const int row = tile_row<PHASE>(t.tile * g.R + sub, gr);
      if (PHASE == 0) {
        if (a0 >= 0) p.h[(int64_t)a0 * p.I + row] = swiglu(c[0], c[2], p.gate_limit, p.up_limit);
        if (a1 >= 0) p.h[(int64_t)a1 * p.I + row] = swiglu(c[1], c[3], p.gate_limit, p.up_limit);
      } else {
        if (a0 >= 0) {
          float* y = p.y + (int64_t)a0 * p.H + row;
          y[0] = c[0] * r->weight[a0];
          y[2] = c[2] * r->weight[a0];
        }
        if (a1 >= 0) {
          float* y = p.y + (int64_t)a1 * p.H + row;
          y[0] = c[1] * r->weight[a1];
          y[2] = c[3] * r->weight[a1];
        }
      }
    }
    __syncwarp();
    arrive_if(lane == 0, L.part_empty + 8 * buf);
    if (++buf == kPartBufs) {
      buf = 0;
      phase ^= 1u;
    }
  }
}

// Second launch, after its tiles: a CTA counts each of them at its output tile
// (the n_list-th to do so sums that tile's rows over the experts, j ascending,
// so the order of arrival does not show).  Its own rows are published first.
__device__ void count_tiles(const FewArgs& p, const Phase& g, const Route* r, int u0, int u1, int* s_mine,
                            int* s_count) {
  const int lane = threadIdx.x & 31;
  __threadfence();
  __syncwarp();
  for (int u = u0 + lane; u < u1; u += 32) {
    const int tile = unit_at(u, g.tiles).tile;
    if (atomicAdd(p.done + tile, 1) == r->n_list - 1) s_mine[atomicAdd(s_count, 1)] = tile;
  }
  __threadfence();
}

__device__ void sum_tiles(const FewArgs& p, const Phase& g, const Route* r, const int* s_mine, int count) {
  const int cols = 16 * g.R, per = p.T * cols;
  for (int i = threadIdx.x; i < count * per; i += kThreads) {
    const int tile = s_mine[i / per], t = i % per / cols, c = i % cols;
    const int n = weight_row<1>(tile * g.R + (c >> 4), c & 15, 0);
    float sum = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int a = t * p.k + j;
      if (r->id[a] >= 0) sum += __ldcg(p.y + (int64_t)a * p.H + n);
    }
    p.out[(int64_t)t * p.H + n] = (uint16_t)pack_bf16x2(sum, sum);
  }
}

template <int PHASE, int SPW>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const FewArgs p, const Phase g, const Phase next) {
  extern __shared__ uint8_t smem[];
  __shared__ Route route;
  __shared__ uint64_t s_bars[3 * kMaxStages + 2 * kPartBufs];
  __shared__ int s_abort, s_count;
  __shared__ int s_mine[kFewMaxTiles];
  const int warp = threadIdx.x >> 5;
  Ring L;
  L.slots = smem_u32(smem);
  L.part = L.slots + g.stages * g.stage_bytes;
  L.full = smem_u32(s_bars);
  L.scales = L.full + 8 * kMaxStages;
  L.empty = L.scales + 8 * kMaxStages;
  L.part_full = L.empty + 8 * kMaxStages;
  L.part_empty = L.part_full + 8 * kPartBufs;
  L.abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(L.full + 8 * i, 1);
      mbar_init(L.scales + 8 * i, 32);
      mbar_init(L.empty + 8 * i, kWarps);
    }
    for (int i = 0; i < kPartBufs; ++i) {
      mbar_init(L.part_full + 8 * i, kWarps);
      mbar_init(L.part_empty + 8 * i, 1);
    }
    s_abort = 0;
    s_count = 0;
    fence_mbar_init();
  }
  if (PHASE == 0) {
    pdl_wait();  // logits and activations may come from the kernel just before, and its caller may still use h
    pdl_trigger();
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) *p.status = 0;
      for (int i = threadIdx.x; i < kFewMaxTiles; i += kThreads) p.done[i] = 0;
    }
  }
  // The second launch reads the router's output before it waits for the first:
  // that started only when whatever wrote it was complete.
  route_all(p, &route);
  __syncthreads();
  const int64_t units = (int64_t)route.n_list * g.tiles;
  const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  if (warp < kWarps) {
    if constexpr (SPW > 2) regs_inc<kRegsConsumer>();
    if (PHASE == 1) pdl_wait();
    consume_loop<PHASE, SPW>(p, g, L, &route, u0, u1);
  } else {
    if constexpr (SPW > 2) regs_dec<kRegsOther>();
    if (warp == kWarps) {
      if (PHASE == 1) pdl_wait();
      join_loop<PHASE>(p, g, L, &route, u0, u1);
      if (PHASE == 1) count_tiles(p, g, &route, u0, u1, s_mine, &s_count);
    } else if (warp == kWarps + 1) {
      weight_loop<PHASE>(p, g, L, &route, u0, u1);
      if (PHASE == 0) prefetch_w2(p, next, &route);
    } else if (warp == kWarps + 2) {
      scale_loop<PHASE>(p, g, L, &route, u0, u1);
    }
  }
  __syncthreads();
  if (PHASE == 1 && !s_abort) {
    pdl_trigger();
    if (route.n_list == 0) {  // no expert at all: zero rows
      pdl_wait();
      for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < (int64_t)p.T * p.H;
           i += (int64_t)gridDim.x * kThreads)
        p.out[i] = 0;
    } else {
      sum_tiles(p, g, &route, s_mine, s_count);
    }
  }
}

Phase phase_of(int K, int m16_tiles, size_t smem) {
  Phase g = {};
  g.K = K;
  g.R = 1;
  while (g.R < kWarps && 2 * g.R * K <= 4096) g.R *= 2;
  g.KG = kWarps / g.R;
  g.tiles = m16_tiles / g.R;  // 16 or more m16 tiles, in sixteens
  g.pitch = (K / 2) % 128 == 64 ? K / 2 : K / 2 + 64;
  g.scale_off = 16 * g.R * g.pitch;
  g.stage_bytes = g.scale_off + g.R * K;
  const int n = (int)((smem - kPartBufs * kWarps * 512) / g.stage_bytes);
  g.stages = n < kMaxStages ? n : kMaxStages;
  return g;
}

template <int PHASE, int SPW>
cudaError_t launch(const FewArgs& a, int num_sms, cudaStream_t s) {
  static int configured = -1;
  static size_t dynamic = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured != dev) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, few_kernel<PHASE, SPW>)) != cudaSuccess) return e;
    // setmaxnreg.inc waits for what the other warps give back: launch only with the allocation it is sized for
    if (SPW > 2 && fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    dynamic = 232448 - 1024 - fa.sharedSizeBytes;
    e = cudaFuncSetAttribute(few_kernel<PHASE, SPW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dynamic);
    if (e != cudaSuccess) return e;
    configured = dev;
  }
  const Phase first = phase_of(a.H, a.I / 8, dynamic), second = phase_of(a.I, a.H / 16, dynamic);
  const Phase& g = PHASE == 0 ? first : second;
  const size_t smem = (size_t)g.stages * g.stage_bytes + kPartBufs * kWarps * 512;
  return launch_kernel(few_kernel<PHASE, SPW>, dim3(num_sms), dim3(kThreads), smem, s, true, a, g, second);
}

template <int PHASE>
cudaError_t launch_phase(const FewArgs& a, int K, int num_sms, cudaStream_t s) {
  return K > 4096 ? launch<PHASE, 4>(a, num_sms, s) : launch<PHASE, 2>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_moe_few(const FewArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = launch_phase<0>(a, a.H, num_sms, s);
  return e == cudaSuccess ? launch_phase<1>(a, a.I, num_sms, s) : e;
}

}  // namespace nvfp4
