// bf16 instances of the product kernel, form NN, sums in segments.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_nn_long(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  if (p.out_type == TDX_FP32)
    return g == kFlat ? launch_linear_g<false, NN, kFlat, kSegments>(p, pair, want, stream)
                      : launch_linear_g<false, NN, kRows, kSegments>(p, pair, want, stream);
  return g == kFlat ? launch_linear_g<false, NN, kFlat, kLongSegments>(p, pair, want, stream)
                    : launch_linear_g<false, NN, kRows, kLongSegments>(p, pair, want, stream);
}

}  // namespace tdx
