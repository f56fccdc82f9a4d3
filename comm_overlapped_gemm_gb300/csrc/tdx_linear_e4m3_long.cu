// e4m3 instances of the product kernel (forward product only), sums of segments in fp32.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_e4m3_long(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<true, NN, kFlat, true>(p, pair, want, stream)
                    : launch_linear_g<true, NN, kRows, true>(p, pair, want, stream);
}

}  // namespace tdx
