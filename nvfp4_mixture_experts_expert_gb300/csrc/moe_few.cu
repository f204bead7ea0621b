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
// the next eight.
//
// A token's activations are scaled by a power of two, one for a warp's share of
// K, that puts their largest at 2^14..2^15, and the sum is scaled back in FP32.
// bf16 values down to 2^-31 of the largest are then exact in f16; what the rounding
// of smaller ones leaves is added in passes of its own (add_rest), so x is used
// exactly.  The FP32 h is rounded to 11 bits, and to multiples of 2^-38 of the
// share's largest below 2^-28 of it: an eighth of what the output's rounding to
// bf16 does.  Measured with a second f16 term for h's other bits, the error of 8
// tokens against 64 bits is 0.001680 instead of 0.001691 (0.001680 is the
// rounding to bf16 alone) and the layer takes 81.1 us instead of 74.8 (1 token
// 32.5 / 29.7, 32 tokens 138 / 128): h stays one term.
//
// The 128 x 4 scale tiles keep rows r, r + 32, r + 64, r + 96 in one 16-byte
// line, so the rows of an m16 tile are taken as whole lines: W13, 2 lines of
// gate rows and the same 2 of up rows (8 features; gate in accumulator rows
// 0-7, up in rows 8-15, so a lane holds both of its feature); W2, 4 lines.
// A tensor map with the dimensions (64 or 128 bytes of a row, line, row of the
// line, piece of the row, 128-row block) then brings all of a tile's rows, piece
// by piece, in one or two copies; row by row, a warp's issue of the copies took
// longer than their arrival.  The copy engine takes about as long for 64 bytes
// of a row as for 128, so the pieces are 128 bytes where K % 256 == 0.  The
// swizzle of the piece's width makes the consumers' reads conflict-free (whole
// rows come in as fast, but two rows then share the banks of each read: 870
// cycles of shared memory a tile instead of 375, of the 1,570 that HBM takes).
//
// Two launches of one kernel, h between them, and a sum; one CTA per SM, which
// takes a range of the (list entry, tile) pairs.  A tile is R m16 tiles (up to 32
// KB of packed weights) over all of K.  Its warps:
//   8 consumers      KG = 8 / R of them share an m16 tile and split K by slabs;
//                    their activations stay in registers while the entry lasts
//   warp 8           the weights' copies into the ring
//   warp 9           the scales', 16 bytes a line: as 32-byte pieces they would
//                    be a third of the copy engine's work
//   warps 10, 11     tile by tile in turn: join the KG sums in a fixed order;
//                    SwiGLU, or the weighted row of W2 h
// Every CTA of the first launch routes for itself (3 to 5 us; a launch of its own
// would take as long); the second finds the tables in the workspace.  It starts
// as CTAs of the first leave (programmatic dependent launch) and fills its rings
// before it waits for h, and the first asks for the second's first weights to be
// brought into L2, so HBM idles little between the two.
//
// Bound: reading the chosen experts' weights, at 32 tokens (48 experts of H 4096,
// I 2048, top 6: 680 MB) 100 us at the rate of a copy; the layer takes 125, of
// which the first launch's stream runs at 6.5 TB/s.  The rest is what comes
// before a launch's first tile (routing, activations, the ring's first copies),
// the way from one launch to the next and the sum: ~17 us of one token's 29,
// whose weights take 12.5.  Measured beside what was kept, at the time (8 / 32
// tokens, us in a row of calls): sixteen consumer warps 85 / 161 where eight took
// 83 / 156; weights not marked for early eviction 90 / 165 instead of 83 / 156
// (they push scales, activations and the next launch's weights out of L2); warps
// that wait by polling 94 / 172 instead of 92 / 169; consumers that read the next
// tiles before they finish the last products 103 / 187 instead of 92 / 169.
//
// Size counts too: most of the code runs once a launch, behind misses of the
// instruction cache, so loops off the stream are kept rolled.  127 and 105 KB of
// code in the two launches took 0.6 to 1.1 us more than 91 and 74 (3 % at one
// token, 4 % at 5 tokens of a small layer), 147 and 125 KB another 5.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "per_device.h"
#include "ptx.cuh"
#include "route_key.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 8;  // consumers
constexpr int kThreads = 32 * (kWarps + 4);
constexpr int kRegsLaunch = 168;   // per thread; 64,512 of the SM's 65,536 registers
constexpr int kRegsConsumer = 216; // 64 of them activations
constexpr int kRegsOther = 72;
static_assert(128 * (2 * kRegsConsumer + kRegsOther) <= kThreads * kRegsLaunch, "the register split must fit");
constexpr int kMaxStages = 16;
constexpr int kJoinWarps = 2;
constexpr int kPartBufs = 4;       // tiles whose sums wait to be joined
constexpr int kFirstCopies = 2;
constexpr int kPrefetch = 3;       // W2 tiles a CTA of the first launch brings into L2
constexpr int kEntryTiles = 1;     // what another list entry costs a CTA
constexpr int kGroup = 8;  // tokens of one list entry

// Routing tables: every (token, expert) assignment a = t * k + j, and the list
// of (expert, up to 8 of its assignments).
struct alignas(16) Route {
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
// none left gets a zero row.  A largest logit of +inf or NaN makes the weights NaN.  An expert named twice is computed once, with the
// sum of the two weights.  NK: logits a lane.
template <int NK>
__device__ __forceinline__ void route_one(const FewArgs& p, int t, int lane, int32_t* s_id, float* s_w,
                                          uint32_t* s_mask) {
  int id = -1;
  float w = 0.f;
  if (p.logits) {
    uint64_t key[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < p.E ? route_key(__ldg(p.logits + (int64_t)t * p.E + e), e) : 0ull;
    }
    uint64_t mine = 0ull;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
      uint64_t best = key[0];
#pragma unroll
      for (int i = 1; i < NK; ++i) best = key[i] > best ? key[i] : best;
      const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
      const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
      const uint64_t win = ((uint64_t)hi << 32) | lo;
#pragma unroll
      for (int i = 0; i < NK; ++i)
        if (key[i] == win) key[i] = 0ull;
      if (lane == j) mine = win;
    }
    const float top = key_value(__shfl_sync(0xffffffffu, mine, 0));
    float z = 0.f;
    if (lane < p.k) {
      const float l = key_value(mine);
      id = key_expert(mine);
      z = l == -INFINITY ? 0.f : expf(l - top);
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
#pragma unroll 1
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
#pragma unroll 1
  for (int i = tid; i < kFewAssignments * kGroup / 8; i += kThreads) reinterpret_cast<uint4*>(r->member)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  __syncthreads();
#pragma unroll 1
  for (int t = warp; t < p.T; t += kThreads / 32) {
    if (p.E <= 32)
      route_one<1>(p, t, lane, r->id, r->weight, s_mask);
    else if (p.E <= 64)
      route_one<2>(p, t, lane, r->id, r->weight, s_mask);
    else
      route_one<8>(p, t, lane, r->id, r->weight, s_mask);
  }
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
#pragma unroll 1
  for (int a = tid; a < p.T * p.k; a += kThreads) {
    const int e = r->id[a], t = a / p.k;
    if (e < 0) continue;
    const int rank = __popc(s_mask[e] & ((1u << t) - 1u));
    const int v = s_first[e] + rank / kGroup;
    r->expert[v] = e;
    r->member[v][rank % kGroup] = (int16_t)a;
  }
}

// The first launch's first CTA leaves the tables for the second, whose CTAs then
// need not route again: complete once `ready` holds the call's number, until the
// sum takes it back.  The second launch starts after that CTA has triggered it; a
// CTA that finds the tables missing all the same routes for itself.  Numbers are a
// process's own, so what another call left, one whose later launches failed among
// them, is not taken for this call's.
struct alignas(16) RouteTable {
  uint64_t ready, pad;
  Route route;
};
static_assert(sizeof(RouteTable) <= kFewTableBytes, "the workspace's share");
constexpr int kRouteWords = sizeof(Route) / 16;

__device__ __forceinline__ void leave_route(const FewArgs& p, const Route& r) {
  RouteTable* t = static_cast<RouteTable*>(p.table);
  for (int i = threadIdx.x; i < kRouteWords; i += kThreads)
    reinterpret_cast<uint4*>(&t->route)[i] = reinterpret_cast<const uint4*>(&r)[i];
  __syncthreads();
  if (threadIdx.x == 0)
    asm volatile("fence.acq_rel.gpu;\nst.release.gpu.global.b64 [%0], %1;" ::"l"(&t->ready), "l"(p.call) : "memory");
}
__device__ __forceinline__ bool take_route(const FewArgs& p, Route* r) {
  const RouteTable* t = static_cast<const RouteTable*>(p.table);
  uint64_t ready;
  asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(ready) : "l"(&t->ready) : "memory");
  if (ready == p.call)
    for (int i = threadIdx.x; i < kRouteWords; i += kThreads)
      reinterpret_cast<uint4*>(r)[i] = __ldcg(reinterpret_cast<const uint4*>(&t->route) + i);
  return __syncthreads_and(ready == p.call);
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
  asm("{\n.reg .b16 t, lo, hi;\n.reg .b32 h;\ncvt.u16.u32 t, %2;\ncvt.rn.f16x2.e4m3x2 h, t;\n"
      "mov.b32 {lo, hi}, h;\nmov.b32 %0, {lo, lo};\nmov.b32 %1, {hi, hi};\n}"
      : "=r"(s0), "=r"(s1)
      : "r"(codes));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The lane's 32 weights of two rows of two tiles (words in K order, the rows' two
// scales) times its 32 activations of one token, over the quad: 128 of K.  Two
// sums a tile, so that a product does not wait for the one before it.
// Decoding is what the consumers do: a pair of weights takes a conversion (2
// cycles of the ALU pipe) and a multiplication (2 of the FP16 pipe), 3 together.
__device__ __forceinline__ void mma_slab(float (&c)[2][4], float (&d)[2][4], const uint4 (&w)[2][2],
                                         const uint32_t (&sc)[2][2], const uint32_t (&b)[16]) {
  uint32_t s[2][2][2], x[2][2][4];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      scale_pairs(sc[t][r], s[t][r][0], s[t][r][1]);
      x[t][r][0] = w[t][r].x, x[t][r][1] = w[t][r].y, x[t][r][2] = w[t][r].z, x[t][r][3] = w[t][r].w;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t f[2][2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) decode8(x[t][r][i], s[t][r][i >> 1], f[t][r]);
#pragma unroll
    for (int t = 0; t < 2; ++t) mma_f16(c[t], f[t][0][0], f[t][1][0], f[t][0][1], f[t][1][1], b[4 * i], b[4 * i + 1]);
#pragma unroll
    for (int t = 0; t < 2; ++t)
      mma_f16(d[t], f[t][0][2], f[t][1][2], f[t][0][3], f[t][1][3], b[4 * i + 2], b[4 * i + 3]);
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
__device__ __forceinline__ int exponent_of(float pow2) { return (int)(__float_as_uint(pow2) >> 23) - 127; }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float rounded_f16(float v) {
  float r;
  asm("{\n.reg .b16 h;\ncvt.rn.f16.f32 h, %1;\ncvt.f32.f16 %0, h;\n}" : "=f"(r) : "f"(v));
  return r;
}
// silu(g) = g / (1 + e^-g) = g e^g / (1 + e^g), the one whose exponential is at most
// 1: the fast quotient (2 ulp) holds for divisors of 1 to 2, not for those past
// 2^126 that a gate below -87 would give.  The IEEE quotient takes 0.6 us a call
// (one token), most of it the way to its code.
__device__ __forceinline__ float swiglu(float gate, float up, float gate_limit, float up_limit) {
  gate = clamp_up(gate, gate_limit);
  up = -clamp_up(-clamp_up(up, up_limit), up_limit);
  const float t = expf(-fabsf(gate));
  return __fdividef(gate < 0.f ? gate * t : gate, 1.f + t) * up;
}

// Where row r of m16 tile `st` lies in the order of its copy (line fastest):
// feature (phase 0, r < 8: its gate row; the up rows are a copy of their own) or
// output column (phase 1, r < 16).
template <int PHASE>
__device__ __forceinline__ int tile_row(int st, int r) {
  return PHASE == 0 ? (st >> 4) * 128 + (st & 15) * 2 + (r & 1) + 32 * (r >> 1)
                    : (st >> 3) * 128 + (st & 7) * 4 + (r & 3) + 32 * (r >> 2);
}
// The copied row that accumulator row g (0-7) takes.  With 128-byte pieces, two
// rows that eight lanes read together have to differ in bit 2 to miss each
// other's banks under the swizzle.
__device__ __forceinline__ int copied_row(int g, int wide) { return wide ? (g & 1) << 2 | g >> 1 : g; }

// What a launch needs to know of its product (0: W13 x, 1: W2 h).
struct Phase {
  int K, R, KG;       // R m16 tiles a tile, KG = kWarps / R warps along K
  int tiles;          // per list entry
  int blocks;         // 128-row blocks of an expert's matrix
  int wide;           // 128-byte pieces of a row, else 64
  int stage_bytes, stages;
};

struct Ring {
  uint32_t slots, part;  // a tile's weights (8K bytes an m16 tile), then its scales (K bytes each); the warps' sums
  uint32_t full, scales, empty;  // a slot's weights, its scales have landed; it has been read
  uint32_t part_full, part_empty;
  volatile int* abort;
};

// The list entry and tile of unit u.
struct Unit {
  int v, tile;
  __device__ __forceinline__ void advance(int n, int tiles) {  // n <= tiles
    tile += n;
    if (tile >= tiles) {
      tile -= tiles;
      ++v;
    }
  }
};
__device__ __forceinline__ Unit unit_at(int u, int tiles) {
  const int v = (int)((uint32_t)u / (uint32_t)tiles);
  return {v, u - v * tiles};
}

// This CTA's units [u0, u1).  Going over to another list entry costs time (its
// activations are loaded behind the copies under way), so the CTAs are dealt to
// the entries first where that leaves none with more than kEntryTiles over its
// even share of all units (8 tokens: 74.7 us instead of 77.7; 32: 138 instead of 141).
__device__ __forceinline__ void share_of(int n, int tiles, int& u0, int& u1) {
  const uint32_t G = gridDim.x, c = blockIdx.x;
  const uint32_t units = (uint32_t)n * tiles;  // at most 256 * 1024: times G within 32 bits
  const uint32_t even = (units + G - 1) / G;
  if (n > 0 && (uint32_t)n <= G && (tiles + G / n - 1) / (G / n) <= even + kEntryTiles) {
    const uint32_t v = ((c + 1) * n - 1) / G, c0 = v * G / n, count = (v + 1) * G / n - c0;
    u0 = (int)(v * tiles + tiles * (c - c0) / count);
    u1 = (int)(v * tiles + tiles * (c - c0 + 1) / count);
  } else {
    u0 = (int)(units * c / G);
    u1 = (int)(units * (c + 1) / G);
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
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

// ------------------------------------------------------------------ producer
// Line and 128-row block of m16 tile st of an expert.  Phase 0 has the gate rows
// and, I rows on, the up rows.
template <int PHASE>
struct TileAt {
  int line, block;
  __device__ TileAt(const Phase& g, int e, int st)
      : line(PHASE == 0 ? (st & 15) * 2 : (st & 7) * 4), block(e * g.blocks + (PHASE == 0 ? st >> 4 : st >> 3)) {}
};

__device__ __forceinline__ void load_5d(uint32_t dst, const CUtensorMap* map, int line, int block, uint32_t bar,
                                        uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3, %2, %2, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(line), "r"(block), "r"(bar), "l"(policy)
      : "memory");
}

// The first W2 tiles of this CTA's share of the second launch, into L2.
__device__ void prefetch_w2(const FewMaps& m, const Phase& g, const Route* r) {
  int u0, u1;
  share_of(r->n_list, g.tiles, u0, u1);
  if (!elect_one()) return;
#pragma unroll 1
  for (int u = u0; u < min(u1, u0 + kPrefetch); ++u) {
    const Unit t = unit_at(u, g.tiles);
#pragma unroll 1
    for (int i = 0; i < g.R; ++i) {
      const TileAt<1> at(g, r->expert[t.v], t.tile * g.R + i);
      asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %1, %1, %3}];" ::"l"(
                       reinterpret_cast<uint64_t>(&m.next_w)),
                   "r"(0), "r"(at.line), "r"(at.block)
                   : "memory");
    }
  }
}

template <int PHASE>
__device__ void copy_loop(const FewArgs& p, const FewMaps& m, const Phase& g, const Phase& next, const Ring& L,
                          const Route* r, int u0, int u1) {
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  const uint64_t policy = evict_first_policy();
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  Unit t = unit_at(u0, g.tiles);
  if (p.stall) u1 = min(u1, u0 + 1);
  for (int u = u0; u < u1; ++u, t.advance(1, g.tiles)) {
    bool ok = warp_wait_asleep(L.empty + 8 * stage, phase ^ 1u, L.abort, p.status);
    // Two tiles under way until the first lands: they keep HBM busy, and the
    // consumers' first tile does not share its rate with all of the ring's.
    if (ok && u - u0 >= kFirstCopies && u - u0 < g.stages)
      ok = warp_wait_asleep(L.full + 8 * (stage - kFirstCopies), 0, L.abort, p.status);
    if (!ok) break;
    const int e = r->expert[t.v];
    if (leader) {
      const uint32_t w = L.slots + stage * g.stage_bytes, bar = L.full + 8 * stage;
      mbar_arrive_expect_tx(bar, 8 * g.K * g.R);
#pragma unroll 1
      for (int i = 0; i < g.R; ++i) {
        const TileAt<PHASE> at(g, e, t.tile * g.R + i);
        load_5d(w + i * 8 * g.K, &m.w, at.line, at.block, bar, policy);
        if (PHASE == 0) load_5d(w + i * 8 * g.K + 4 * g.K, &m.w, at.line, at.block + g.blocks / 2, bar, policy);
      }
    }
    __syncwarp();
    issued |= 1u << stage;
    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
    if (++stage == (uint32_t)g.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (PHASE == 0) prefetch_w2(m, next, r);
  // The copies land before the warp leaves, also where another role gives up later.
  if (lane == 0) {
    volatile int no_abort = 0;
#pragma unroll 1
    for (int s = 0; s < g.stages; ++s)
      if (issued >> s & 1u) wait_bounded(L.full + 8 * s, issued_parity >> s & 1u, &no_abort, nullptr, kDrainNs);
  }
  __syncwarp();
}

// The tile's scale lines, 16 bytes (four rows by four columns) a copy: per m16
// tile and scale column / 4, the gate's two lines and the up's, or W2's four.
template <int PHASE>
__device__ void scale_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int lane = threadIdx.x & 31, line = lane & 3, cts = g.K / 64;
  const uint8_t* all = PHASE == 0 ? p.sf13 : p.sf2;
  const uint64_t policy = evict_first_policy();
  uint32_t stage = 0, phase = 0;
  Unit t = unit_at(u0, g.tiles);
  for (int u = u0; u < u1; ++u, t.advance(1, g.tiles)) {
    if (!warp_wait_asleep(L.empty + 8 * stage, phase ^ 1u, L.abort, p.status)) break;
    const int e = r->expert[t.v];
    uint32_t to = L.slots + stage * g.stage_bytes + 8 * g.K * g.R + lane * 16;
#pragma unroll 1
    for (int i = 0; i < g.R; ++i) {
      const TileAt<PHASE> at(g, e, t.tile * g.R + i);
      const int block = at.block + (PHASE == 0 ? (line >> 1) * (g.blocks / 2) : 0);
      const uint8_t* from = all + ((int64_t)block * cts + (lane >> 2)) * 512 +
                            (at.line + (PHASE == 0 ? line & 1 : line)) * 16;
#pragma unroll 4
      for (int ct = lane >> 2; ct < cts; ct += 8, from += 8 * 512, to += 512)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                     "l"(policy)
                     : "memory");
      // K = 64 * cts: the lanes past an odd end have made one copy less
      to = L.slots + stage * g.stage_bytes + 8 * g.K * g.R + (i + 1) * g.K + lane * 16;
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(L.scales + 8 * stage) : "memory");
    if (++stage == (uint32_t)g.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ consumers
// This lane's activations of its token for the warp's slabs, as f16 pairs scaled
// by one power of two, whose inverse is returned.  x (of assignment a, -1: none):
// `rest` is the number of passes that its values too small for f16 beside the
// largest need (the warp's tokens' most; 0 but for rows whose values span more
// than 2^31).  Magnitudes are compared as bf16 bits, two at a time.
template <int SPW>
__device__ __forceinline__ float load_x(const FewArgs& p, const Phase& g, int a, int kg, int q, uint32_t (&b)[SPW][16],
                                        int& rest) {
  const int slabs = g.K / 128;
  const uint16_t* x = p.x + (int64_t)(a < 0 ? 0 : a / p.k) * p.ld_x + q * 32;
  uint32_t most = 0u, least = 0x7fff7fffu;  // of two columns; least of |x| + 0x7fff, signed: 0 comes last
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const int slab = kg + s * g.KG;
    if (slab >= slabs || a < 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) b[s][i] = 0u;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + slab * 128) + i);
        b[s][4 * i] = u.x, b[s][4 * i + 1] = u.y, b[s][4 * i + 2] = u.z, b[s][4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t mag = b[s][i] & 0x7fff7fffu;
        most = __vmaxs2(most, mag);
        least = __vmins2(least, mag + 0x7fff7fffu);
      }
    }
  }
  most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 2));
  least = __vmins2(least, __shfl_xor_sync(0xffffffffu, least, 1));
  least = __vmins2(least, __shfl_xor_sync(0xffffffffu, least, 2));
  const uint32_t top = max(most & 0xffffu, most >> 16);
  const uint32_t low = min((least & 0xffffu) ^ 0x8000u, (least >> 16) ^ 0x8000u);  // the smallest above 0, less 1
  float inverse;
  const float scale = slab_scale(__uint_as_float(top << 16), inverse);
  const int exponent = exponent_of(scale), field = max((int)(low + 1) >> 7, 1), left = 78 - field - exponent;
  // 8 bits are exact in f16 from 2^-17 on; what is left down to the smallest value's last bit, 2^(field - 134), is
  // exact by add_rest's passes, of which the first adds 39 to the exponent and each other 32.  Beside an infinity
  // or a NaN nothing is missed.
  rest = top >= 0x7f80u || (int)(low + 1) >> 7 >= 110 - exponent ? 0 : left <= 0 ? 1 : 1 + (left + 31) / 32;
  rest = (int)__reduce_max_sync(0xffffffffu, (uint32_t)rest);
#pragma unroll
  for (int s = 0; s < SPW; ++s)
#pragma unroll
    for (int i = 0; i < 16; ++i) b[s][i] = pack_f16x2(bf16_lo(b[s][i]) * scale, bf16_hi(b[s][i]) * scale);
  return inverse;
}
// h with more than four slabs a warp.
template <int SPW>
__device__ __forceinline__ float load_long_h(const FewArgs& p, const Phase& g, int a, int kg, int q,
                                             uint32_t (&b)[SPW][16]) {
  const int slabs = g.K / 128;
  float amax = 0.f;
  const float* h = p.h + (int64_t)(a < 0 ? 0 : a) * p.I + q * 32;
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const int slab = kg + s * g.KG;
    if (slab >= slabs || a < 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) b[s][i] = 0u;
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // read again (from L2) rather than held: 32 FP32 values a slab
      const float4 u = __ldcg(reinterpret_cast<const float4*>(h + slab * 128) + i);
      b[s][2 * i] = pack_f16x2(u.x * scale, u.y * scale);
      b[s][2 * i + 1] = pack_f16x2(u.z * scale, u.w * scale);
    }
  }
  return inverse;
}

// 32 bytes (a whole sector), past L1.
__device__ __forceinline__ void load_sector(const float* p, float (&v)[8]) {
  asm volatile("ld.relaxed.gpu.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
}
// The same for h with four slabs a warp at most: the FP32 values stay in
// registers between their maximum and their rounding, so that all loads are in
// flight together, once (32 tokens: 142 us instead of 155; all SMs read h at the
// same time), by whole sectors (128 instead of 134: 16 bytes a lane would take
// each sector twice).
template <int SPW>
__device__ __forceinline__ float load_h(const FewArgs& p, const Phase& g, int a, int kg, int q, uint32_t (&b)[SPW][16]) {
  const float* h = p.h + (int64_t)(a < 0 ? 0 : a) * p.I + q * 32;
  float v[SPW][4][8];
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const int slab = kg + s * g.KG;
    const bool in = slab < g.K / 128 && a >= 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[s][i][j] = 0.f;
      if (in) load_sector(h + slab * 128 + 8 * i, v[s][i]);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int s = 0; s < SPW; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[s][i][j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  float inverse;
  const float scale = slab_scale(amax, inverse);
#pragma unroll
  for (int s = 0; s < SPW; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[s][4 * i + j] = pack_f16x2(v[s][i][2 * j] * scale, v[s][i][2 * j + 1] * scale);
  return inverse;
}

// v += the products of what load_x's rounding to f16 left of the smallest values.
// Those remainders have 8 bits at most and lie below 2^-25 as scaled there; pass by
// pass the ones of 32 powers of two are taken, from memory again, and go the way
// of the others.  Slow, so its code is kept small, and off the way of any row
// whose values lie within 2^31 of its largest.  `at`, `second`, `s_off`, `s_second`:
// the tile, and in it the lane's second row and the scales of its two; `weight_at`:
// its first row's weights of a slab.
template <typename WeightAt>
__device__ __forceinline__ void add_rest(const FewArgs& p, const Phase& g, int a, int kg, int q, float inverse, int rest,
                                         float alpha, uint32_t at, uint32_t second, uint32_t s_off, uint32_t s_second,
                                         const WeightAt& weight_at, float (&v)[4]) {
  const uint16_t* x = p.x + (int64_t)(a < 0 ? 0 : a / p.k) * p.ld_x + q * 32;
  const int first = -exponent_of(inverse);
#pragma unroll 1
  for (int pass = 0; pass < rest; ++pass) {
    const int exponent = min(first + 39 + 32 * pass, 157);  // past 148 nothing is left
    float c[4] = {};
#pragma unroll 1
    for (int i = kg * 4; i < g.K / 32; i = i % 4 == 3 ? i + 4 * g.KG - 3 : i + 1) {  // a quarter of a slab's 32 columns
      const int slab = i / 4, part = i % 4;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (a >= 0) u = __ldg(reinterpret_cast<const uint4*>(x + slab * 128) + part);
      const uint32_t in[4] = {u.x, u.y, u.z, u.w};
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float r[2] = {bf16_lo(in[j]), bf16_hi(in[j])};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          r[n] = fmaf(-rounded_f16(r[n] * pow2f(first)), inverse, r[n]) * pow2f(exponent / 2) *
                 pow2f(exponent - exponent / 2);
          if (!(fabsf(r[n]) >= 0x1p-17f && fabsf(r[n]) < 0x1p15f)) r[n] = 0.f;
        }
        b[j] = pack_f16x2(r[0], r[1]);
      }
      uint32_t f[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t s[2];
        scale_pairs(lds16(at + s_off + (slab - kg) * 128 + n * s_second), s[0], s[1]);
        decode8(lds32(at + weight_at(slab) + n * second + part * 4), part < 2 ? s[0] : s[1], f[n]);
      }
      mma_f16(c, f[0][0], f[1][0], f[0][1], f[1][1], b[0], b[1]);
      mma_f16(c, f[0][2], f[1][2], f[0][3], f[1][3], b[2], b[3]);
    }
    const float down0 = pow2f(-(exponent / 2)), down1 = pow2f(exponent / 2 - exponent);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] += c[j] * alpha * __shfl_sync(0xffffffffu, down0, q * 8 + (j & 1) * 4) *
              __shfl_sync(0xffffffffu, down1, q * 8 + (j & 1) * 4);
  }
}

template <int PHASE, int SPW>
__device__ void consume_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int u0, int u1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, q = lane & 3;
  const int kg = warp % g.KG, sub = warp / g.KG, slabs = g.K / 128;
  // this lane's two rows, slab by slab, and their scales
  const int row = copied_row(gr, g.wide);
  const auto weight_at = [&](int slab) -> uint32_t {
    return sub * 8 * g.K + (g.wide ? (slab >> 1) * (PHASE == 0 ? 1024 : 2048) + row * 128 +
                                         ((((slab & 1) * 4 + q) ^ row) << 4)
                                   : slab * (PHASE == 0 ? 512 : 1024) + row * 64 + ((q ^ (row >> 1 & 3)) << 4));
  };
  uint32_t w_off[SPW];
#pragma unroll
  for (int s = 0; s < SPW; ++s) w_off[s] = weight_at(kg + s * g.KG);
  const uint32_t second = PHASE == 0 ? 4 * g.K : g.wide ? 1024 : 512;
  const uint32_t s_off = 8 * g.K * g.R + sub * g.K + kg * 128 + (q >> 1) * 64 + (q & 1) * 2 +
                         (PHASE == 0 ? (row & 1) * 16 + (row >> 1) * 4 : (row & 3) * 16 + (row >> 2) * 4);
  constexpr uint32_t s_second = PHASE == 0 ? 32 : 8;
  const uint32_t part = L.part + warp * 512 + lane * 16;
  uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1;
  uint32_t b[SPW][16];
  float inv = 0.f, i0 = 0.f, i1 = 0.f, alpha = 0.f;
  int rest = 0;
  Unit t = unit_at(u0, g.tiles);
  bool fresh = true;
  for (int u = u0; u < u1;) {
    if (fresh) {
      alpha = 1.f / __ldg((PHASE == 0 ? p.gs13 : p.gs2) + r->expert[t.v]);
      if constexpr (PHASE == 0)
        inv = load_x<SPW>(p, g, r->member[t.v][gr], kg, q, b, rest);
      else if constexpr (SPW <= 4)
        inv = load_h<SPW>(p, g, r->member[t.v][gr], kg, q, b);
      else
        inv = load_long_h<SPW>(p, g, r->member[t.v][gr], kg, q, b);
      i0 = __shfl_sync(0xffffffffu, inv, q * 8);
      i1 = __shfl_sync(0xffffffffu, inv, q * 8 + 4);
    }
    // Two tiles at a time while the list entry lasts: waiting, handing over the
    // sums and coming back cost about half of what one tile's products take.
    // Both have landed and buffers for their sums are free (of one tile, each is asked twice).
    const int n = min(2, min(u1 - u, g.tiles - t.tile));
    const uint32_t stage2 = stage + 1 == (uint32_t)g.stages ? 0u : stage + 1, phase2 = stage2 ? phase : phase ^ 1u;
    const uint32_t buf2 = buf + 1 == kPartBufs ? 0u : buf + 1, buf_phase2 = buf2 ? buf_phase : buf_phase ^ 1u;
    {
      const uint32_t s2 = n == 2 ? stage2 : stage, ph2 = n == 2 ? phase2 : phase;
      const uint32_t b2 = n == 2 ? buf2 : buf, bp2 = n == 2 ? buf_phase2 : buf_phase;
      const uint32_t bars[6] = {L.full + 8 * stage, L.scales + 8 * stage,   L.full + 8 * s2,
                                L.scales + 8 * s2,  L.part_empty + 8 * buf, L.part_empty + 8 * b2};
      const uint32_t parities[6] = {phase, phase, ph2, ph2, buf_phase, bp2};
      if (!warp_wait_every(bars, parities, L.abort, p.status)) return;
    }
    // both tiles' products side by side: each alone is a chain of waits
    float c[2][4] = {}, d[2][4] = {};
    const uint32_t at0 = L.slots + stage * g.stage_bytes, at1 = n == 2 ? L.slots + stage2 * g.stage_bytes : at0;
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
      if (kg + s * g.KG < slabs) {
        const uint32_t ss = s_off + s * g.KG * 128;
        const uint4 w[2][2] = {{lds128(at0 + w_off[s]), lds128(at0 + w_off[s] + second)},
                               {lds128(at1 + w_off[s]), lds128(at1 + w_off[s] + second)}};
        const uint32_t sc[2][2] = {{lds16(at0 + ss), lds16(at0 + ss + s_second)},
                                   {lds16(at1 + ss), lds16(at1 + ss + s_second)}};
        mma_slab(c, d, w, sc, b[s]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < n)  // alpha first: neither factor leaves FP32's range
        sts128(part + (i ? buf2 : buf) * (kWarps * 512), (c[i][0] + d[i][0]) * alpha * i0,
               (c[i][1] + d[i][1]) * alpha * i1, (c[i][2] + d[i][2]) * alpha * i0, (c[i][3] + d[i][3]) * alpha * i1);
    if constexpr (PHASE == 0)
      if (rest)
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t to = part + (i ? buf2 : buf) * (kWarps * 512);
          const uint4 sum = lds128(to);
          float v[4] = {__uint_as_float(sum.x), __uint_as_float(sum.y), __uint_as_float(sum.z), __uint_as_float(sum.w)};
          add_rest(p, g, r->member[t.v][gr], kg, q, inv, rest, alpha, i ? at1 : at0, second, s_off, s_second, weight_at, v);
          sts128(to, v[0], v[1], v[2], v[3]);
        }
    __syncwarp();
    arrive_if(lane == 0, L.empty + 8 * stage);
    arrive_if(lane == 0, L.part_full + 8 * buf);
    arrive_if(lane == 0 && n == 2, L.empty + 8 * stage2);
    arrive_if(lane == 0 && n == 2, L.part_full + 8 * buf2);
    u += n;
    fresh = t.tile + n == g.tiles;
    t.advance(n, g.tiles);
    stage += n;
    if (stage >= (uint32_t)g.stages) {
      stage -= g.stages;
      phase ^= 1u;
    }
    buf += n;
    if (buf >= kPartBufs) {
      buf -= kPartBufs;
      buf_phase ^= 1u;
    }
  }
}

// ------------------------------------------------------------------ join
template <int PHASE, int R>
__device__ __forceinline__ void join_loop(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int which,
                                          int u0, int u1) {
  constexpr int KG = kWarps / R;
  const int n = PHASE == 0 ? p.I : p.H;
  const int lane = threadIdx.x & 31, gr = lane >> 2, q = lane & 3;
  uint32_t buf = which, phase = 0;
  Unit t = unit_at(u0 + which, g.tiles);
  for (int u = u0 + which; u < u1; u += kJoinWarps, t.advance(kJoinWarps, g.tiles)) {
    const int a0 = r->member[t.v][2 * q], a1 = r->member[t.v][2 * q + 1];
    const float p0 = PHASE == 1 && a0 >= 0 ? r->weight[a0] : 0.f, p1 = PHASE == 1 && a1 >= 0 ? r->weight[a1] : 0.f;
    if (!warp_wait_asleep(L.part_full + 8 * buf, phase, L.abort, p.status)) return;
    const uint32_t from = L.part + buf * (kWarps * 512) + lane * 16;
    float* to0 = (PHASE == 0 ? p.h : p.y) + (int64_t)a0 * n;
    float* to1 = (PHASE == 0 ? p.h : p.y) + (int64_t)a1 * n;
#pragma unroll 1
    for (int sub = 0; sub < R; ++sub) {
      float c[4];
#pragma unroll
      for (int i = 0; i < KG; ++i) {
        const uint4 v = lds128(from + (sub * KG + i) * 512);
        const float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = i ? c[k] + f[k] : f[k];
      }
      const int row = tile_row<PHASE>(t.tile * R + sub, copied_row(gr, g.wide));
      if (PHASE == 0) {
        const float h0 = swiglu(c[0], c[2], p.gate_limit, p.up_limit);
        const float h1 = swiglu(c[1], c[3], p.gate_limit, p.up_limit);
        if (a0 >= 0) to0[row] = h0;
        if (a1 >= 0) to1[row] = h1;
      } else {  // accumulator row gr + 8 is output column row + 64
        if (a0 >= 0) to0[row] = c[0] * p0, to0[row + 64] = c[2] * p0;
        if (a1 >= 0) to1[row] = c[1] * p1, to1[row + 64] = c[3] * p1;
      }
    }
    __syncwarp();
    arrive_if(lane == 0, L.part_empty + 8 * buf);
    if ((buf += kJoinWarps) >= kPartBufs) {
      buf -= kPartBufs;
      phase ^= 1u;
    }
  }
}

template <int PHASE>
__device__ void join_tiles(const FewArgs& p, const Phase& g, const Ring& L, const Route* r, int which, int u0, int u1) {
  switch (g.R) {
    case 1: return join_loop<PHASE, 1>(p, g, L, r, which, u0, u1);
    case 2: return join_loop<PHASE, 2>(p, g, L, r, which, u0, u1);
    case 4: return join_loop<PHASE, 4>(p, g, L, r, which, u0, u1);
    default: return join_loop<PHASE, 8>(p, g, L, r, which, u0, u1);
  }
}

// out[t] = bf16(the sum of the token's weighted rows, j ascending).
__global__ void __launch_bounds__(256) few_sum_kernel(const FewArgs p) {
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) static_cast<RouteTable*>(p.table)->ready = 0;
  const int i = blockIdx.x * 256 + threadIdx.x, per = p.H / 4;  // four columns a thread
  if (i >= p.T * per) return;
  const int t = i / per, n = i - t * per;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < p.k; ++j) {
    const int a = t * p.k + j;
    if (p.ids[a] >= 0) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p.y + (int64_t)a * p.H) + n);
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
  }
  reinterpret_cast<uint2*>(p.out + (int64_t)t * p.H)[n] = make_uint2(pack_bf16x2(sum.x, sum.y),
                                                                     pack_bf16x2(sum.z, sum.w));
}

template <int PHASE, int SPW>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewMaps m, const FewArgs p, const Phase g,
                                                           const Phase next) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Route route;
  __shared__ uint64_t s_bars[3 * kMaxStages + 2 * kPartBufs];
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5;
  Ring L;
  L.slots = (smem_u32(smem) + 1023u) & ~1023u;
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
    fence_mbar_init();
    prefetch_tmap(&m.w);
  }
  if (PHASE == 0) {
    pdl_wait();  // logits and activations may come from the kernel just before, and its caller may still use h
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    // on their way to L2 while the tokens are routed
    for (int i = threadIdx.x * 32; p.logits && i < p.T * p.E; i += kThreads * 32) prefetch_l2(p.logits + i);
    const int lines = (p.H + 63) / 64;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.T * lines; i += gridDim.x * kThreads)
      prefetch_l2(p.x + (int64_t)(i / lines) * p.ld_x + i % lines * 64);
    if (threadIdx.x < p.E) {
      prefetch_l2(p.gs13 + threadIdx.x);
      prefetch_l2(p.gs2 + threadIdx.x);
    }
  }
  if (PHASE == 0 || !take_route(p, &route)) {
    // also the second launch may read the router's output before it waits for the
    // first: that started only when whatever wrote it was complete
    route_all(p, &route);
    __syncthreads();
  }
  if (PHASE == 0) {
    if (blockIdx.x == 0) {
      if (threadIdx.x < p.T * p.k) p.ids[threadIdx.x] = route.id[threadIdx.x];
      leave_route(p, route);
    }
    pdl_trigger();
  }
  int u0, u1;
  share_of(route.n_list, g.tiles, u0, u1);
  if (warp < kWarps) {
    regs_inc<kRegsConsumer>();
    if (PHASE == 1) pdl_wait();
    consume_loop<PHASE, SPW>(p, g, L, &route, u0, u1);
  } else {
    regs_dec<kRegsOther>();
    if (warp == kWarps) {
      copy_loop<PHASE>(p, m, g, next, L, &route, u0, u1);
    } else if (warp == kWarps + 1) {
      scale_loop<PHASE>(p, g, L, &route, u0, u1);
    } else {
      if (PHASE == 1) pdl_wait();
      join_tiles<PHASE>(p, g, L, &route, warp - (kWarps + 2), u0, u1);
    }
  }
  __syncthreads();  // no warp's copies outlive the CTA
}

// `entries`: the most entries the list can have.  R doubles up to 32 KB of
// weights a tile as long as a CTA keeps eight tiles: with fewer, one more or less
// is a large part of its time (5 tokens, H 1792, I 640: 21.6 us instead of 26.1).
Phase phase_of(int K, int m16_tiles, int blocks, size_t smem, int64_t entries, int num_sms) {
  Phase g = {};
  g.K = K;
  g.R = 1;
  while (g.R < kWarps && 2 * g.R * K <= 4096 && entries * m16_tiles >= 2 * g.R * 8 * (int64_t)num_sms) g.R *= 2;
  g.KG = kWarps / g.R;
  g.tiles = m16_tiles / g.R;  // 16 or more m16 tiles, in sixteens
  g.blocks = blocks;
  g.wide = K % 256 == 0;
  g.stage_bytes = (9 * K * g.R + 1023) / 1024 * 1024;
  const int n = (int)((smem - 1024 - kPartBufs * kWarps * 512) / g.stage_bytes);
  g.stages = n < kMaxStages ? n : kMaxStages;
  return g;
}

template <int PHASE, int SPW>
cudaError_t launch(const FewArgs& a, const FewMaps& m, int num_sms, cudaStream_t s) {
  static PerDevice<size_t, cudaError_t> memory;  // dynamic shared memory of a CTA
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const size_t* dynamic = nullptr;
  e = memory.get(dev, &dynamic, [](size_t& bytes) {
    cudaFuncAttributes fa;
    if (const cudaError_t e = cudaFuncGetAttributes(&fa, few_kernel<PHASE, SPW>)) return e;
    // setmaxnreg.inc waits for what the other warps give back: launch only with the allocation it is sized for
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    bytes = 232448 - 1024 - fa.sharedSizeBytes;
    return cudaFuncSetAttribute(few_kernel<PHASE, SPW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
  if (e != cudaSuccess) return e;
  const Phase first = phase_of(a.H, a.I / 8, 2 * a.I / 128, *dynamic, a.T * a.k, num_sms);
  const Phase second = phase_of(a.I, a.H / 16, a.H / 128, *dynamic, a.T * a.k, num_sms);
  const Phase& g = PHASE == 0 ? first : second;
  const size_t smem = 1024 + (size_t)g.stages * g.stage_bytes + kPartBufs * kWarps * 512;
  return launch_kernel(few_kernel<PHASE, SPW>, dim3(num_sms), dim3(kThreads), smem, s, true, m, a, g, second);
}

// Above K = 4096 a warp holds up to eight slabs (W2's kernel then spills 436 bytes)
// and the ring two or three tiles, which do not keep HBM busy: H 7168, I 2048, top
// 8 of 16 takes 58.8 us for one token and 101 for eight, of 29.2 and 58.1 at the
// rate of a copy.
template <int PHASE>
cudaError_t launch_phase(const FewArgs& a, const FewMaps& m, int K, int num_sms, cudaStream_t s) {
  return K > 4096 ? launch<PHASE, 8>(a, m, num_sms, s) : launch<PHASE, 4>(a, m, num_sms, s);
}

}  // namespace

cudaError_t launch_moe_few(const FewArgs& args, const FewMaps& w13, const FewMaps& w2, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> calls{0x6f75746564214d4bull};  // nothing that memory is likely to hold
  FewArgs a = args;
  a.call = calls.fetch_add(1, std::memory_order_relaxed);
  FewMaps m = w13;
  m.next_w = w2.w;
  cudaError_t e = launch_phase<0>(a, m, a.H, num_sms, s);
  if (e == cudaSuccess) e = launch_phase<1>(a, w2, a.I, num_sms, s);
  if (e != cudaSuccess) return e;
  return launch_kernel(few_sum_kernel, dim3((a.T * (a.H / 4) + 255) / 256), dim3(256), 0, s, true, a);
}

}  // namespace nvfp4
