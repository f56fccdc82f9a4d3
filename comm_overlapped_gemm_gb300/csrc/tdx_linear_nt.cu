// bf16 instances of the product kernel, form NT.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_nt(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<false, NT, kFlat, kOnce>(p, pair, want, stream)
                    : launch_linear_g<false, NT, kRows, kOnce>(p, pair, want, stream);
}

}  // namespace tdx
