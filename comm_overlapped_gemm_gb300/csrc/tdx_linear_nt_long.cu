// bf16 instances of the product kernel, form NT, sums in segments.
#include "tdx_linear.cuh"

namespace tdx {

tdx_status launch_linear_nt_long(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  if (p.out_type == TDX_FP32)
    return g == kFlat ? launch_linear_g<false, NT, kFlat, kSegments>(p, pair, want, stream)
                      : launch_linear_g<false, NT, kRows, kSegments>(p, pair, want, stream);
  return g == kFlat ? launch_linear_g<false, NT, kFlat, kLongSegments>(p, pair, want, stream)
                    : launch_linear_g<false, NT, kRows, kLongSegments>(p, pair, want, stream);
}

}  // namespace tdx
