// bf16 instances of the product kernel, form TN, sums in segments.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_tn_long(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  if (p.out_type == TDX_FP32)
    return g == kFlat ? launch_linear_g<false, TN, kFlat, kSegments>(p, pair, want, stream)
                      : launch_linear_g<false, TN, kSums, kSegments>(p, pair, want, stream);
  return g == kFlat ? launch_linear_g<false, TN, kFlat, kLongSegments>(p, pair, want, stream)
                    : launch_linear_g<false, TN, kSums, kLongSegments>(p, pair, want, stream);
}

}  // namespace tdx
