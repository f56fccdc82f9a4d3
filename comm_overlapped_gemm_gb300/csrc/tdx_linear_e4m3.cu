// e4m3 instances of the product kernel (forward product only).
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_e4m3(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<true, NN, kFlat, kOnce>(p, pair, want, stream)
                    : launch_linear_g<true, NN, kRows, kOnce>(p, pair, want, stream);
}

}  // namespace tdx
