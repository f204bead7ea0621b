// The linear's products on the tensor cores (linear_gemm.cuh): plan, launch, and the
// kernels without an activation.
#include "linear_gemm.cuh"

#include "per_device.h"

namespace nvfp4 {

namespace {

using namespace linear_gemm;

// Clusters of the split and of the pair form that the GPU holds at a time.
struct Fit {
  Clusters split, pair;
};
cudaError_t clusters_that_fit(const Fit** out) {
  static PerDevice<Fit, cudaError_t> fit;  // one CTA a SM in all forms
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  return fit.get(dev, out, [](Fit& f) {
    if (const cudaError_t e = configure<128, true, false, kEpiPlain>()) return e;
    if (const cudaError_t e = configure<256, false, true, kEpiPlain>()) return e;
    if (const cudaError_t e = max_clusters(linear_gemm_kernel<128, true, false, kEpiPlain>, kThreads,
                                           Cfg<128, false>::SMEM, f.split))
      return e;
    return max_clusters(linear_gemm_kernel<256, false, true, kEpiPlain>, kThreads, Cfg<256, true>::SMEM, f.pair);
  });
}

}  // namespace

cudaError_t launch_linear_plain(LinearArgs& p, int slots, cudaStream_t s) {
  return launch_form<kEpiPlain>(p, slots, s);
}

// The plan that takes least time by the times of a K-block and of a tile's epilogue
// (beside the next tile's products) in each form, and of the join where the CTAs of a
// cluster share a tile's K (one round of tiles with SMs to spare).  Measured: pairs 25.7
// us for 1024 x 4096 x 4096 (256 columns 28.7, 128 35), 128 columns 20 for 512 x 4096 x
// 4096 (pairs 25, 64 columns 28), 128 columns with four CTAs a tile 11.7 for 16 x 4096 x
// 4096 (one 19.3), 64 columns with eight 8.9 for 64 x 256 x 8192 (one 24.8).  Pairs on
// groups of rows run turned, a K-block in less time where a tile has fewer tokens, and
// with an epilogue that SwiGLU's arithmetic makes longer: 32 groups of 300 rows, 4096 x
// 4096, 260 us (256 columns 319, 128 361; not turned 315), of 1024 rows of 512 inputs,
// SwiGLU, 138 (256 columns 109).  Weight
// gradients of groups run as single CTAs: the rows behind a group's last would have to
// be set to zero in both CTAs' operands (by remote stores and a fence of the cluster 521
// us instead of 427 for 32 groups of 384 rows, 4096 x 4096; with nothing set to zero 385
// instead of 387).
cudaError_t linear_gemm_plan(LinearArgs& p, int num_sms) {
  const Fit* fit = nullptr;
  const cudaError_t e = clusters_that_fit(&fit);
  if (e != cudaSuccess) return e;
  struct Form {
    int bn, pair, block_ns, tile_ns, join_ns;
  };
  constexpr Form kForms[4] = {
      {256, 1, 310, 3100, 0}, {256, 0, 385, 2700, 0}, {128, 0, 250, 1600, 4500}, {64, 0, 190, 1000, 3000}};
  const bool pairs = p.ep.act == kActSwiglu;
  const int64_t k = p.counts && p.by_k ? (p.K + p.G - 1) / p.G : p.K;  // of a group, on average
  const int64_t kbs = (k + kBK - 1) / kBK;
  int64_t least = INT64_MAX;
  for (Form f : kForms) {
    const int rows = f.pair ? 2 * kBM : kBM, out_cols = pairs ? f.bn / 2 : f.bn;
    const int64_t slots = f.pair ? fit->pair.most[2] : num_sms;
    if (slots == 0 || (f.pair && p.by_k && p.counts)) continue;
    // rows of groups: half a tile more for each that can have any, at least one
    const int64_t some = p.M < p.G ? p.M : p.G, whole = (p.M + rows - 1) / rows;
    const int64_t mt = p.by_k               ? (int64_t)p.G * whole
                       : !p.counts          ? whole
                       : whole > some / 2   ? whole + some / 2
                                            : some;
    const bool turned = f.pair && p.counts && !p.by_k;
    if (turned) {
      const int64_t tokens = (p.M + mt - 1) / mt + 16;  // of a tile, in steps of 32
      f.block_ns = 135 + 7 * (int)(tokens < 256 ? tokens : 256) / 10;
      if (pairs) f.tile_ns = 4100;
    }
    const int64_t tiles = mt * ((p.N + out_cols - 1) / out_cols);
    for (int c = 1; c <= (f.bn < 256 && !p.counts ? kMaxSplit : 1) && c <= kbs; ++c) {
      if (c > 1 && (tiles * c > num_sms || tiles > fit->split.most[c])) continue;
      const int64_t loop_ns = (kbs + c - 1) / c * f.block_ns, rounds = (tiles * c + slots - 1) / slots;
      const int64_t ns = rounds * (loop_ns > f.tile_ns ? loop_ns : f.tile_ns) + f.tile_ns + (c > 1 ? f.join_ns : 0);
      if (ns < least) least = ns, p.bn = f.bn, p.pair = f.pair, p.turned = turned, p.split = c;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_linear_gemm(LinearArgs& p, int num_sms, cudaStream_t s) {
  int slots = num_sms;
  if (p.pair) {
    const Fit* fit = nullptr;
    const cudaError_t e = clusters_that_fit(&fit);
    if (e != cudaSuccess) return e;
    slots = fit->pair.most[2];
  }
  return p.ep.act == kActSwiglu ? launch_linear_swiglu(p, slots, s)
         : p.ep.act != kActNone ? launch_linear_activation(p, slots, s)
                                : launch_linear_plain(p, slots, s);
}

}  // namespace nvfp4
