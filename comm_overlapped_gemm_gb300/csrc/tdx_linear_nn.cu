// bf16 instances of the product kernel, form NN.
#include "tdx_linear.cuh"

namespace tdx {

int lin_clusters(int split) {
  static std::atomic<int> cache[64][kMostSplit + 1];
  const int guess = 16 / split * 8;   // where it cannot be asked: 8 groups of 16 SMs
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return guess;
  const int known = cache[dev][split].load(std::memory_order_relaxed);
  if (known > 0) return known;
  using C = LinCfg<false, NN, kFlat, false>;
  auto* kernel = tdx_linear_kernel<false, NN, kFlat, false, kOnce>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess) return guess;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(split * 64, 1, 1);
  cfg.blockDim = dim3(kNumThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return guess;
  cache[dev][split].store(n, std::memory_order_relaxed);
  return n;
}

tdx_status launch_linear_nn(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream) {
  return g == kFlat ? launch_linear_g<false, NN, kFlat, kOnce>(p, pair, want, stream)
                    : launch_linear_g<false, NN, kRows, kOnce>(p, pair, want, stream);
}

}  // namespace tdx
