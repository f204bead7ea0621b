// The linear's products on the tensor cores (linear_gemm.cuh), the kernels with SwiGLU.
#include "linear_gemm.cuh"

namespace nvfp4 {

cudaError_t launch_linear_swiglu(LinearArgs& p, int slots, cudaStream_t s) {
  return linear_gemm::launch_form<kEpiSwiglu>(p, slots, s);
}

}  // namespace nvfp4
