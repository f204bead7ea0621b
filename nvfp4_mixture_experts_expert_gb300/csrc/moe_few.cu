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
// The 128 x 4 scale tiles keep rows r, r + 32, r + 64, r + 96 in one 16-byte
// line, so the rows of an m16 tile are taken as whole lines: W13, 2 lines of
// gate rows and the same 2 of up rows (8 features; gate in accumulator rows
// 0-7, up in rows 8-15, so a lane holds both of its feature); W2, 4 lines.
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"
#include "route_key.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
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
  for (int t = warp; t < p.T; t += kWarps) route_one(p, t, lane, r->id, r->weight, s_mask);
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

__global__ void __launch_bounds__(kThreads) few_route_kernel(const FewArgs p) {
  if (threadIdx.x == 0) *p.status = 0;
  route_all(p, reinterpret_cast<Route*>(p.route));
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
// times its 32 activations of one token, over the quad: 128 of K.
__device__ __forceinline__ void mma_slab(float (&c)[4], const uint4& w0, const uint4& w1, uint32_t sc0, uint32_t sc1,
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
    mma_f16(c, r0[2], r1[2], r0[3], r1[3], b[4 * i + 2], b[4 * i + 3]);
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
// 32 values -> f16 pairs scaled by the quad's (one token's) power of two.
__device__ __forceinline__ void to_f16(const float (&f)[32], uint32_t (&b)[16], float& inverse) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const float s = slab_scale(amax, inverse);
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = pack_f16x2(f[2 * i] * s, f[2 * i + 1] * s);
}

// Where row g (and, in W2, row g + 8) of m16 tile `st` lies: feature (phase 0)
// or output column (phase 1).
template <int PHASE>
__device__ __forceinline__ int tile_row(int st, int g) {
  const int i = g >> 2, j = g & 3;
  return PHASE == 0 ? (st >> 4) * 128 + (st & 15) * 2 + i + 32 * j : (st >> 3) * 128 + (st & 7) * 4 + i + 32 * j;
}

// PHASE 0: h of one list entry's assignments for R * 8 features; PHASE 1: their
// weighted W2 rows for R * 16 columns.  KG warps split K by slabs of 128 (sums
// joined in shared memory, fixed order), R = 16 / KG m16 tiles a block.
template <int PHASE>
__global__ void __launch_bounds__(kThreads) few_product_kernel(const FewArgs p, int KG) {
  const Route* r = reinterpret_cast<const Route*>(p.route);
  const int v = blockIdx.y;
  if (v >= r->n_list) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int R = kWarps / KG, kg = warp % KG, st = blockIdx.x * R + warp / KG;
  const int e = r->expert[v];
  const int K = PHASE == 0 ? p.H : p.I, rows = PHASE == 0 ? 2 * p.I : p.H;
  const int row0 = tile_row<PHASE>(st, g), row1 = PHASE == 0 ? p.I + row0 : row0 + 2;
  const uint8_t* W = (PHASE == 0 ? p.w13 : p.w2) + (int64_t)e * rows * (K / 2);
  const uint8_t* SF = (PHASE == 0 ? p.sf13 : p.sf2) + (int64_t)e * rows * (K / 16);
  const int a = r->member[v][g];  // this lane's token
  __shared__ float4 part[kWarps][32];
  const float alpha = 1.f / (PHASE == 0 ? p.gs13 : p.gs2)[e];
  float acc[4] = {};
  for (int slab = kg; slab < K / 128; slab += KG) {
    const int k0 = slab * 128 + q * 32;
    const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(W + (int64_t)row0 * (K / 2) + k0 / 2));
    const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(W + (int64_t)row1 * (K / 2) + k0 / 2));
    const uint32_t s0 = __ldg(reinterpret_cast<const uint16_t*>(SF + sf_offset(row0, k0 / 16, K / 16)));
    const uint32_t s1 = __ldg(reinterpret_cast<const uint16_t*>(SF + sf_offset(row1, k0 / 16, K / 16)));
    float f[32];
    if (a < 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = 0.f;
    } else if (PHASE == 0) {
      const uint4* x = reinterpret_cast<const uint4*>(p.x + (int64_t)(a / p.k) * p.ld_x + k0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldg(x + i);
        f[8 * i] = bf16_lo(u.x), f[8 * i + 1] = bf16_hi(u.x), f[8 * i + 2] = bf16_lo(u.y), f[8 * i + 3] = bf16_hi(u.y);
        f[8 * i + 4] = bf16_lo(u.z), f[8 * i + 5] = bf16_hi(u.z);
        f[8 * i + 6] = bf16_lo(u.w), f[8 * i + 7] = bf16_hi(u.w);
      }
    } else {
      const float4* h = reinterpret_cast<const float4*>(p.h + (int64_t)a * p.I + k0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 u = h[i];
        f[4 * i] = u.x, f[4 * i + 1] = u.y, f[4 * i + 2] = u.z, f[4 * i + 3] = u.w;
      }
    }
    uint32_t b[16];
    float inv;
    to_f16(f, b, inv);
    float c[4] = {};
    mma_slab(c, w0, w1, s0, s1, b);
    const float i0 = __shfl_sync(0xffffffffu, inv, q * 8), i1 = __shfl_sync(0xffffffffu, inv, q * 8 + 4);
    acc[0] = fmaf(c[0] * alpha, i0, acc[0]);  // alpha first: neither factor leaves FP32's range
    acc[1] = fmaf(c[1] * alpha, i1, acc[1]);
    acc[2] = fmaf(c[2] * alpha, i0, acc[2]);
    acc[3] = fmaf(c[3] * alpha, i1, acc[3]);
  }
  part[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (kg != 0) return;
  float4 c = part[warp][lane];
  for (int i = 1; i < KG; ++i) {
    const float4 o = part[warp + i][lane];
    c.x += o.x, c.y += o.y, c.z += o.z, c.w += o.w;
  }
  const float lo[2] = {c.x, c.y}, hi[2] = {c.z, c.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int to = r->member[v][2 * q + i];
    if (to < 0) continue;
    if (PHASE == 0) {
      const float gate = clamp_up(lo[i], p.gate_limit);
      const float up = -clamp_up(-clamp_up(hi[i], p.up_limit), p.up_limit);
      p.h[(int64_t)to * p.I + row0] = gate / (1.f + expf(-gate)) * up;
    } else {
      const float w = r->weight[to];
      p.y[(int64_t)to * p.H + row0] = lo[i] * w;
      p.y[(int64_t)to * p.H + row1] = hi[i] * w;
    }
  }
}

__global__ void __launch_bounds__(256) few_combine_kernel(const FewArgs p) {
  const Route* r = reinterpret_cast<const Route*>(p.route);
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;  // H % 256 == 0
  float sum = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int a = t * p.k + j;
    if (r->id[a] >= 0) sum += p.y[(int64_t)a * p.H + n];
  }
  p.out[(int64_t)t * p.H + n] = (uint16_t)pack_bf16x2(sum, sum);
}

int k_groups(int K) {
  int kg = 1;
  while (kg < kWarps && 2 * kg <= K / 128) kg *= 2;
  return kg;
}

}  // namespace

size_t moe_few_route_words() { return sizeof(Route) / 4; }

cudaError_t launch_moe_few(const FewArgs& a, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const int A = a.T * a.k;
  const int most = A < a.E + A / kGroup ? A : a.E + A / kGroup;
  cudaError_t e = launch_kernel(few_route_kernel, dim3(1), dim3(kThreads), 0, s, false, a);
  if (e != cudaSuccess) return e;
  const int kg1 = k_groups(a.H), kg2 = k_groups(a.I);
  e = launch_kernel(few_product_kernel<0>, dim3(a.I / 8 / (kWarps / kg1), most), dim3(kThreads), 0, s, false, a, kg1);
  if (e != cudaSuccess) return e;
  e = launch_kernel(few_product_kernel<1>, dim3(a.H / 16 / (kWarps / kg2), most), dim3(kThreads), 0, s, false, a, kg2);
  if (e != cudaSuccess) return e;
  return launch_kernel(few_combine_kernel, dim3(a.H / 256, a.T), dim3(256), 0, s, false, a);
}

}  // namespace nvfp4
