// bf16 instances of the product kernel, form TN.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_tn(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<false, TN, kFlat, kOnce>(p, pair, want, stream)
                    : launch_linear_g<false, TN, kSums, kOnce>(p, pair, want, stream);
}

}  // namespace tdx
