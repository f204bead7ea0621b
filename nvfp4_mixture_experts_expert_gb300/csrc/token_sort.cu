// Tokens sorted by expert and back (see nvfp4_sort_tokens, nvfp4_combine_tokens
// and their gradients).
//
//   sort      rows[inverse[t][j]] = x[t]
//   its grad  dx[t] = sum_j drows[inverse[t][j]]                 (combine without weights)
//   combine   out[t] = residual[t] + sum_j w[t][j] * rows[inverse[t][j]]
//   its grad  drows[inverse[t][j]] = w[t][j] * dout[t],  dw[t][j] = dout[t] . rows[inverse[t][j]]
//
// The order is by expert, then by the assignment's flat index f = t * top_k + j
// (no atomic decides a row): a stable counting sort by one cluster of eight CTAs,
// whose 256 warps each own a contiguous range of f.  Up to kFusedAssignments the
// kernel that copies the rows works the order out itself, every block for its own
// token, and there is one launch.  Sums over j are FP32 in the order of j.
//
// Bound: HBM, each row read and written once.  8192 x 4096, 6 of 48 experts, bf16: sort
// into slots of 128 rows 81 us on the GPU (495 MB, 73 us at the 6.8 TB/s of a copy; the
// order 9.6 of them), combine and its gradient together 206 us (1.34 GB, 198 us).  One
// token: sort 3.3 us, combine 2.6, launch and two trips to memory.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "nvfp4_format.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 32;
constexpr int kOrderWarps = 32;
constexpr int kOrderCtas = 8;
// 512 assignments of 4096 columns 4.0 us in one launch against 6.3 in two, 1024 5.4
// against 6.5 (512 columns 4.6 against 5.5); 2048 8.6 against 7.6 (11.7 against 5.6),
// every block looking through all of them.
constexpr int kFusedAssignments = 1024;
constexpr int kHeld = 8;  // ids a lane

// 0 .. E - 1, or E: held elsewhere.
__device__ __forceinline__ int local_expert(int32_t id, int32_t start, int E) {
  const int64_t e = (int64_t)id - start;
  return e >= 0 && e < E ? (int)e : E;
}

// The lanes with the same expert (0 .. 2^bits - 1), by a vote on each bit: a
// match.any takes a warp longer than six votes (49152 assignments of 48 experts 14.3 us
// instead of 12.2).
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
  uint32_t peers = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xffffffffu, (e >> b) & 1);
    peers &= (e >> b) & 1 ? set : ~set;
  }
  return peers;
}

// Warp 0: s_off[e] = sum of the aligned counts before e, s_off[E] the total.
__device__ __forceinline__ void scan_offsets(const int32_t* count, int32_t* s_off, int E, int align, int lane) {
  int off = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    const int c = e < E ? (count[e] + align - 1) & -align : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (e < E) s_off[e] = off + incl - c;
    off += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) s_off[E] = off;
}

// Phase 1: each warp counts its range's assignments per expert.  Phase 2: prefix
// sums over the warps, over the CTAs (distributed shared memory) and, aligned,
// over the experts.  Phase 3: each warp goes over its range again and hands out rows.
// Eight CTAs because they can meet without a second launch.  Bound by the instructions
// of eight warps a scheduler: ids, experts and peers of the first pass kept in registers
// take the order of 49152 assignments from 12.2 to 9.6 us (4004: 3.8; 524288 of 128
// experts: 95, where the rows take 1.3 ms).
__global__ void __cluster_dims__(kOrderCtas, 1, 1) __launch_bounds__(kOrderWarps * 32) token_order_kernel(
    const SortArgs p) {
  __shared__ int32_t hist[kOrderWarps][kMaxExperts];
  __shared__ int32_t cta_total[kMaxExperts], total[kMaxExperts], below[kMaxExperts], s_off[kMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
  const uint32_t rank = cluster_ctarank();
  for (int i = threadIdx.x; i < kOrderWarps * kMaxExperts; i += blockDim.x) (&hist[0][0])[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();  // only now: copy_rows_kernel reads x before it waits for this one
  const int64_t n = p.T * p.k, g = (int64_t)rank * kOrderWarps + warp, warps = kOrderCtas * kOrderWarps;
  const int64_t f0 = n * g / warps, f1 = n * (g + 1) / warps;
  const int bits = 32 - __clz(E);  // of 0 .. E; E: no expert held here
  // 32 kHeld ids at a time, and those of a range that has no more stay in registers
  const bool one = f1 - f0 <= 32 * kHeld;
  int e[kHeld];
  uint32_t peers[kHeld];
  auto take = [&](int64_t base) {
    int id[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) id[i] = base + i * 32 + lane < f1 ? p.ids[base + i * 32 + lane] : 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (base + i * 32 >= f1) break;
      e[i] = base + i * 32 + lane < f1 ? local_expert(id[i], p.start, E) : E;
      peers[i] = same_expert(e[i], bits);
    }
  };
  for (int64_t base = f0; base < f1; base += 32 * kHeld) {
    take(base);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (base + i * 32 >= f1) break;
      if (e[i] < E && lane == __ffs(peers[i]) - 1) hist[warp][e[i]] += __popc(peers[i]);
      __syncwarp();
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int c[kOrderWarps], sum = 0;
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) c[w] = hist[w][e];
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) {
      hist[w][e] = sum;
      sum += c[w];
    }
    cta_total[e] = sum;
  }
  cluster_sync_all();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const uint32_t a = smem_u32(&cta_total[e]);
    int sum = 0, lower = 0;
#pragma unroll
    for (int q = 0; q < kOrderCtas; ++q) {
      const int c = (int)ld_shared_cluster_u32(mapa_shared(a, (uint32_t)q));
      sum += c;
      lower += q < (int)rank ? c : 0;
    }
    total[e] = sum;
    below[e] = lower;
  }
  __syncthreads();
  cluster_arrive_relaxed();  // this CTA's reads of the others' shared memory are done
  if (warp == 0) scan_offsets(total, s_off, E, p.align, lane);
  __syncthreads();
  for (int i = threadIdx.x; i < kOrderWarps * E; i += blockDim.x) {
    const int w = i / E, e = i - w * E;
    hist[w][e] += s_off[e] + below[e];
  }
  if (rank == 0) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
      p.offsets[e] = s_off[e];
      if (e < E) p.counts[e] = total[e];
    }
  }
  __syncthreads();
  for (int64_t base = f0; base < f1; base += 32 * kHeld) {
    if (!one) take(base);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (base + i * 32 >= f1) break;
      const int64_t f = base + i * 32 + lane;
      int row = -1;
      if (e[i] < E) row = hist[warp][e[i]] + __popc(peers[i] & ((1u << lane) - 1u));
      __syncwarp();
      if (e[i] < E && lane == __ffs(peers[i]) - 1) hist[warp][e[i]] += __popc(peers[i]);
      __syncwarp();
      if (f < f1) p.inverse[f] = row;
      if (row >= 0) p.source[row] = (int32_t)f;
    }
  }
  // rows without an assignment: between the experts, and behind the last
  const int64_t t0 = (int64_t)rank * blockDim.x + threadIdx.x, step = (int64_t)kOrderCtas * blockDim.x;
  if (p.align > 1) {
    const int pad = p.align - 1;
    for (int i = (int)t0; i < E * pad; i += (int)step) {
      const int e = i / pad, r = s_off[e] + total[e] + (i - e * pad);
      if (r < s_off[e + 1]) p.source[r] = -1;
    }
  }
  for (int64_t r = s_off[E] + t0; r < p.capacity; r += step) p.source[r] = -1;
  cluster_wait();
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void store16(uint8_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// A warp writes pad row i of the E * (align - 1) possible ones as zeros.
__device__ __forceinline__ void zero_pad_row(uint8_t* rows, int64_t ld, int nvec, const int32_t* offsets,
                                             const int32_t* counts, int E, int align, int64_t i, int lane) {
  const int pad = align - 1;
  if (i >= (int64_t)E * pad) return;
  const int e = (int)(i / pad), r = offsets[e] + counts[e] + (int)(i - (int64_t)e * pad);
  if (r >= offsets[e + 1]) return;
  for (int c = lane; c < nvec; c += 32) store16(rows + r * ld + c * 16, make_uint4(0, 0, 0, 0));
}

// Two of a token's vectors: c and c + blockDim.x.
struct TokenPiece {
  uint4 a, b;
  bool two;
};
__device__ __forceinline__ TokenPiece load_piece(const SortArgs& p, int64_t t, int c) {
  const uint8_t* x = p.x + t * p.ld_x;
  TokenPiece v = {};
  v.two = c + (int)blockDim.x < p.nvec;
  if (c < p.nvec) v.a = load16(x + c * 16);
  if (v.two) v.b = load16(x + (c + blockDim.x) * 16);
  return v;
}
// A token's vectors, of which `v` is the thread's first piece, to its rows.
__device__ __forceinline__ void copy_token(const SortArgs& p, int64_t t, const int32_t* row, TokenPiece v) {
  const int nt = blockDim.x;
  for (int c = threadIdx.x; c < p.nvec; c += 2 * nt) {
    if (c != threadIdx.x) v = load_piece(p, t, c);
    for (int j = 0; j < p.k; ++j) {
      const int64_t r = row[j];
      if (r < 0) continue;
      store16(p.rows + r * p.ld_rows + c * 16, v.a);
      if (v.two) store16(p.rows + r * p.ld_rows + (c + nt) * 16, v.b);
    }
  }
}

// A token per block, then blocks that write pad rows, a row per warp.  x is there as
// soon as the ordering kernel has begun (it waits for what came before it).
__global__ void __launch_bounds__(512) copy_rows_kernel(const SortArgs p) {
  pdl_trigger();
  const int64_t t = blockIdx.x;
  TokenPiece first = {};
  if (t < p.T) first = load_piece(p, t, threadIdx.x);
  pdl_wait();
  if (t >= p.T) {
    const int warps = blockDim.x >> 5;
    zero_pad_row(p.rows, p.ld_rows, p.nvec, p.offsets, p.counts, p.E, p.align,
                 (t - p.T) * warps + (threadIdx.x >> 5), threadIdx.x & 31);
    return;
  }
  __shared__ int32_t row[kMaxTopK];
  if (threadIdx.x < p.k) row[threadIdx.x] = p.inverse[t * p.k + threadIdx.x];
  __syncthreads();
  copy_token(p, t, row, first);
}

// The same with the order worked out by every block: counts and aligned offsets
// of all experts, and the rank of its own token's assignments.
__global__ void __launch_bounds__(512) sort_few_kernel(const SortArgs p) {
  pdl_trigger();
  __shared__ int32_t ids[kFusedAssignments];
  __shared__ int32_t count[kMaxExperts], off[kMaxExperts + 1], rank[kMaxTopK], row[kMaxTopK];
  const int n = (int)p.T * p.k, E = p.E, k = p.k, tid = threadIdx.x, nt = blockDim.x;
  for (int e = tid; e < E; e += nt) count[e] = 0;
  if (tid < kMaxTopK) rank[tid] = 0;
  __syncthreads();
  pdl_wait();
  for (int f = tid; f < n; f += nt) {
    const int e = local_expert(p.ids[f], p.start, E);
    ids[f] = e;
    if (e < E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (tid < 32) scan_offsets(count, off, E, p.align, tid);
  const int64_t t = blockIdx.x;
  TokenPiece first = {};
  if (t < p.T && p.rows) first = load_piece(p, t, tid);
  if (t < p.T) {
    const int mine = (int)t * k;
    for (int f = tid; f < mine + k; f += nt) {  // the ones before an assignment with its expert
      const int e = ids[f];
      for (int j = 0; j < k; ++j)
        if (f < mine + j && e == ids[mine + j]) atomicAdd(&rank[j], 1);
    }
  }
  __syncthreads();
  if (t >= p.T) {  // pad rows
    const int warps = nt >> 5;
    const int64_t i = (t - p.T) * warps + (tid >> 5);
    if (p.rows) zero_pad_row(p.rows, p.ld_rows, p.nvec, off, count, E, p.align, i, tid & 31);
    const int pad = p.align - 1;
    if (i < (int64_t)E * pad && (tid & 31) == 0) {
      const int e = (int)(i / pad), r = off[e] + count[e] + (int)(i - (int64_t)e * pad);
      if (r < off[e + 1]) p.source[r] = -1;
    }
    return;
  }
  if (tid < k) {
    const int f = (int)t * k + tid, e = ids[f], r = e < E ? off[e] + rank[tid] : -1;
    row[tid] = r;
    p.inverse[f] = r;
    if (r >= 0) p.source[r] = f;
  }
  if (t == 0) {
    for (int e = tid; e <= E; e += nt) {
      p.offsets[e] = off[e];
      if (e < E) p.counts[e] = count[e];
    }
    for (int64_t r = off[E] + tid; r < p.capacity; r += nt) p.source[r] = -1;
  }
  __syncthreads();
  if (p.rows) copy_token(p, t, row, first);
}

// ------------------------------------------------------------------ sums over a token's rows

// 16 bytes of a row as FP32 values.
template <int DT>
struct Vec;
template <>
struct Vec<kTypeBf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<kTypeF16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = d.x, f[2 * i + 1] = d.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<kTypeF32> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

constexpr int kInFlight = 8;  // rows of a token loaded at once

// A token's columns [c0, c1) (vectors) per block, gridDim.y blocks a token: out =
// residual + sum over j of w * row.  Without weights every row counts once.
template <int DT>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs p) {
  using V = Vec<DT>;
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x;
  __shared__ int32_t row[kMaxTopK];
  __shared__ float wt[kMaxTopK];
  if (threadIdx.x < p.k) {
    row[threadIdx.x] = p.inverse[t * p.k + threadIdx.x];
    wt[threadIdx.x] = p.weights ? p.weights[t * p.k + threadIdx.x] : 1.f;
  }
  __syncthreads();
  const int c0 = (int)((int64_t)p.nvec * blockIdx.y / gridDim.y), c1 = (int)((int64_t)p.nvec * (blockIdx.y + 1) / gridDim.y);
  for (int c = c0 + threadIdx.x; c < c1; c += blockDim.x) {
    float acc[V::N] = {};
    if (p.residual) V::get(load16(p.residual + t * p.ld_residual + c * 16), acc);
    for (int j0 = 0; j0 < p.k; j0 += kInFlight) {
      uint4 v[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (j0 + j < p.k && row[j0 + j] >= 0) v[j] = load16(p.rows + row[j0 + j] * p.ld_rows + c * 16);
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        if (j0 + j >= p.k || row[j0 + j] < 0) continue;
        float f[V::N];
        V::get(v[j], f);
#pragma unroll
        for (int i = 0; i < V::N; ++i) acc[i] = fmaf(wt[j0 + j], f[i], acc[i]);
      }
    }
    store16(p.out + t * p.ld_out + c * 16, V::put(acc));
  }
}

// A token per block (dout read once for its rows), then blocks that write pad rows.
template <int DT>
__global__ void __launch_bounds__(256) combine_grad_kernel(const CombineGradArgs p) {
  using V = Vec<DT>;
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (t >= p.T) {
    zero_pad_row(p.drows, p.ld_drows, p.nvec, p.offsets, p.counts, p.E, p.align, (t - p.T) * warps + warp, lane);
    return;
  }
  __shared__ int32_t row[kMaxTopK];
  __shared__ float wt[kMaxTopK];
  __shared__ float part[8][kInFlight];
  if (threadIdx.x < p.k) {
    row[threadIdx.x] = p.inverse[t * p.k + threadIdx.x];
    wt[threadIdx.x] = p.weights[t * p.k + threadIdx.x];
  }
  __syncthreads();
  for (int j0 = 0; j0 < p.k; j0 += kInFlight) {
    float dot[kInFlight] = {};
    for (int c = threadIdx.x; c < p.nvec; c += blockDim.x) {
      uint4 v[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (j0 + j < p.k && row[j0 + j] >= 0) v[j] = load16(p.rows + row[j0 + j] * p.ld_rows + c * 16);
      float d[V::N];
      V::get(load16(p.dout + t * p.ld_dout + c * 16), d);
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        if (j0 + j >= p.k || row[j0 + j] < 0) continue;
        float f[V::N], o[V::N];
        V::get(v[j], f);
#pragma unroll
        for (int i = 0; i < V::N; ++i) {
          dot[j] = fmaf(d[i], f[i], dot[j]);
          o[i] = wt[j0 + j] * d[i];
        }
        store16(p.drows + row[j0 + j] * p.ld_drows + c * 16, V::put(o));
      }
    }
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      if (j0 + j >= p.k) break;
#pragma unroll
      for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kInFlight && j0 + threadIdx.x < p.k) {
      float s = 0.f;
      for (int w = 0; w < warps; ++w) s += part[w][threadIdx.x];
      p.dweights[t * p.k + j0 + threadIdx.x] = row[j0 + threadIdx.x] >= 0 ? s : 0.f;
    }
    __syncthreads();
  }
}

// Threads of a block for rows of nvec vectors: whole warps, about two vectors each.
int threads_for(int nvec, int most) {
  const int t = ((nvec + 1) / 2 + 31) / 32 * 32;
  return t < 64 ? 64 : t > most ? most : t;
}

int64_t pad_blocks(int E, int align, int threads) {
  const int warps = threads / 32;
  return ((int64_t)E * (align - 1) + warps - 1) / warps;
}

}  // namespace

cudaError_t launch_sort_tokens(const SortArgs& a, cudaStream_t s) {
  const int64_t n = a.T * a.k;
  const int threads = threads_for(a.nvec, 512);
  if (n > 0 && n <= kFusedAssignments) {
    // a vector a thread, and threads enough to look through all assignments
    const int nt = a.nvec >= 512 ? 512 : a.nvec > 256 ? (a.nvec + 31) / 32 * 32 : 256;
    return launch_kernel(sort_few_kernel, dim3((unsigned)(a.T + pad_blocks(a.E, a.align, nt))), dim3(nt), 0, s, true,
                         a);
  }
  cudaError_t e = launch_kernel(token_order_kernel, dim3(kOrderCtas), dim3(kOrderWarps * 32), 0, s, true, a);
  if (e != cudaSuccess || !a.rows || n == 0) return e;
  return launch_kernel(copy_rows_kernel, dim3((unsigned)(a.T + pad_blocks(a.E, a.align, threads))), dim3(threads), 0, s,
                       true, a);
}

cudaError_t launch_combine_tokens(const CombineArgs& a, int type, int num_sms, cudaStream_t s) {
  // a few tokens: several blocks share a token's columns
  int parts = 1;
  while (a.T * parts < num_sms && a.nvec / (parts * 2) >= 32) parts *= 2;
  const int threads = threads_for(a.nvec / parts * (parts > 1 ? 2 : 1), 256);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3((unsigned)a.T, parts), dim3(threads), 0, s, true, a);
  };
  return type == kTypeBf16  ? go(combine_kernel<kTypeBf16>)
         : type == kTypeF16 ? go(combine_kernel<kTypeF16>)
                            : go(combine_kernel<kTypeF32>);
}

cudaError_t launch_combine_tokens_grad(const CombineGradArgs& a, int type, cudaStream_t s) {
  const int threads = threads_for(a.nvec, 256);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3((unsigned)(a.T + pad_blocks(a.E, a.align, threads))), dim3(threads), 0, s, true,
                         a);
  };
  return type == kTypeBf16  ? go(combine_grad_kernel<kTypeBf16>)
         : type == kTypeF16 ? go(combine_grad_kernel<kTypeF16>)
                            : go(combine_grad_kernel<kTypeF32>);
}

}  // namespace nvfp4
