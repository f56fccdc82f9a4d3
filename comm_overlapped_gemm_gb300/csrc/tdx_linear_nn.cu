// bf16 instances of the product kernel, form NN.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_nn(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<false, NN, kFlat, false>(p, pair, want, stream)
                    : launch_linear_g<false, NN, kRows, false>(p, pair, want, stream);
}

}  // namespace tdx
