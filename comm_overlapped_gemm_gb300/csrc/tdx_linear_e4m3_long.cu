// e4m3 instances of the product kernel (forward product only), sums in segments.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_e4m3_long(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  if (p.out_type == TDX_FP32)
    return g == kFlat ? launch_linear_g<true, NN, kFlat, kSegments>(p, pair, want, stream)
                      : launch_linear_g<true, NN, kRows, kSegments>(p, pair, want, stream);
  return g == kFlat ? launch_linear_g<true, NN, kFlat, kLongSegments>(p, pair, want, stream)
                    : launch_linear_g<true, NN, kRows, kLongSegments>(p, pair, want, stream);
}

}  // namespace tdx
