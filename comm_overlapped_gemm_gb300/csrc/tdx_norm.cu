// Root-mean-square norm of x + residual and its gradient (tdx_rmsnorm, tdx_rmsnorm_bwd).
#include "tdx_rows.cuh"

namespace tdx {

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    const int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

constexpr int kThreads = 256;
constexpr int kBwdParts = 304;   // most row groups whose partial weight gradients are added at the end

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* h;
  void* y;
  float* row_scale;
  float* rstd;
  int T, H;
  int64_t ld_x, ld_r, ld_h, ld_y;
  float eps, inv_scale;
};

// Sum (or maximum) over the block; every thread gets it.
template <bool MAX>
__device__ float block_reduce(float v, float* sm) {
  v = MAX ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = sm[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) r = MAX ? fmaxf(r, sm[i]) : r + sm[i];
  return r;
}

// One block per row: a pass for the sum of squares, a pass for the largest |y| where the row's scale
// is wanted, a pass that stores.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) tdx_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = kVec<T>;
  __shared__ float sm[kThreads / 32];
  griddep_wait();
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + t * p.ld_x;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + t * p.ld_r : nullptr;
  const T* w = static_cast<const T*>(p.weight);
  T* h = p.h ? static_cast<T*>(p.h) + t * p.ld_h : nullptr;
  O* y = static_cast<O*>(p.y) + t * p.ld_y;

  auto load_h = [&](int c, float (&v)[N]) {
    load_vec(x + c, v);
    if (r != nullptr) {
      float a[N];
      load_vec(r + c, a);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += a[i];
    }
  };
  float ss = 0.0f;
  for (int c = threadIdx.x * N; c < p.H; c += kThreads * N) {
    float v[N];
    load_h(c, v);
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = block_reduce<false>(ss, sm);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.H) + p.eps);
  float inv = p.inv_scale;
  if (p.row_scale != nullptr) {
    float m = 0.0f;
    for (int c = threadIdx.x * N; c < p.H; c += kThreads * N) {
      float v[N], g[N];
      load_h(c, v);
      load_vec(w + c, g);
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i] * rstd * g[i]));
    }
    m = block_reduce<true>(m, sm);
    const float s = m > 0.0f ? m / 448.0f : 1.0f;
    inv = 1.0f / s;
    if (threadIdx.x == 0) p.row_scale[t] = s;
  }
  if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[t] = rstd;
  for (int c = threadIdx.x * N; c < p.H; c += kThreads * N) {
    float v[N], g[N];
    load_h(c, v);
    load_vec(w + c, g);
    if (h != nullptr) store_vec(h + c, v);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] * rstd * g[i] * inv;
    store_vec(y + c, v);
  }
}

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dres;
  void* dx;
  float* part;   // [grid][H] partial weight gradients
  int T, H;
  int64_t ld_dy, ld_h, ld_dres, ld_dx;
};

// A block takes rows b, b + grid, ... and adds up dy * n of its columns in shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_rmsnorm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int N = kVec<T>;
  extern __shared__ float dw[];
  __shared__ float sm[kThreads / 32];
  griddep_wait();
  for (int c = threadIdx.x * N; c < p.H; c += kThreads * N)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[c + i] = 0.0f;
  const T* w = static_cast<const T*>(p.weight);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + t * p.ld_dy;
    const T* h = static_cast<const T*>(p.h) + t * p.ld_h;
    const float rstd = p.rstd[t];
    float dot = 0.0f;
    for (int c = threadIdx.x * N; c < p.H; c += kThreads * N) {
      float d[N], v[N], g[N];
      load_vec(dy + c, d);
      load_vec(h + c, v);
      load_vec(w + c, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = v[i] * rstd;
        dot = fmaf(d[i] * g[i], n, dot);
        dw[c + i] = fmaf(d[i], n, dw[c + i]);
      }
    }
    const float mean = block_reduce<false>(dot, sm) / static_cast<float>(p.H);
    const T* dr = p.dres ? static_cast<const T*>(p.dres) + t * p.ld_dres : nullptr;
    T* dx = static_cast<T*>(p.dx) + t * p.ld_dx;
    for (int c = threadIdx.x * N; c < p.H; c += kThreads * N) {
      float d[N], v[N], g[N];
      load_vec(dy + c, d);
      load_vec(h + c, v);
      load_vec(w + c, g);
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = rstd * (d[i] * g[i] - v[i] * rstd * mean);
      if (dr != nullptr) {
        load_vec(dr + c, v);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] += v[i];
      }
      store_vec(dx + c, d);
    }
  }
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
  for (int c = threadIdx.x * N; c < p.H; c += kThreads * N)
#pragma unroll
    for (int i = 0; i < N; ++i) out[c + i] = dw[c + i];
}

// dweight[c] = the partial sums of column c in the order of the row groups
__global__ void __launch_bounds__(kThreads) tdx_rmsnorm_dweight_kernel(const float* part, float* dweight, int parts, int H) {
  griddep_wait();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= H) return;
  float s = 0.0f;
  for (int b = 0; b < parts; ++b) s += part[static_cast<int64_t>(b) * H + c];
  dweight[c] = s;
}

template <typename T>
tdx_status launch_norm(tdx_dtype out, const NormParams& p, cudaStream_t st) {
  switch (out) {
    case TDX_BF16: return launch_rows(tdx_rmsnorm_kernel<T, bf16>, p.T, kThreads, 0, st, p);
    case TDX_FP32: return launch_rows(tdx_rmsnorm_kernel<T, float>, p.T, kThreads, 0, st, p);
    default: return launch_rows(tdx_rmsnorm_kernel<T, e4m3>, p.T, kThreads, 0, st, p);
  }
}

template <typename T>
tdx_status launch_norm_bwd(const NormBwdParams& p, int grid, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(p.H) * sizeof(float);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(tdx_rmsnorm_bwd_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           32768 * static_cast<int>(sizeof(float))) != cudaSuccess)
    return TDX_ERR_CUDA;
  return launch_rows(tdx_rmsnorm_bwd_kernel<T>, grid, kThreads, smem, st, p);
}

tdx_norm_opts norm_defaults() {
  tdx_norm_opts o;
  std::memset(&o, 0, sizeof(o));
  o.out_dtype = TDX_BF16;
  o.eps = 1e-6f;
  o.out_scale = 1.0f;
  return o;
}

tdx_status check_sizes(int T, int H, tdx_dtype dtype) {
  if (T < 0 || H <= 0 || !known(dtype)) return TDX_ERR_INVALID_ARG;
  return dtype == TDX_FP8_E4M3 ? TDX_ERR_UNSUPPORTED : TDX_OK;
}

int bwd_parts(int T) { return T < kBwdParts ? T : kBwdParts; }

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_norm_opts_default(tdx_norm_opts* opts) {
  if (opts == nullptr) return TDX_ERR_INVALID_ARG;
  *opts = norm_defaults();
  return TDX_OK;
}

tdx_status tdx_rmsnorm(const void* x, const void* residual, const void* weight, void* h_out, void* y, float* row_scale,
                       float* rstd, int T, int H, tdx_dtype dtype, const tdx_norm_opts* opts, void* stream) {
  const tdx_norm_opts o = opts ? *opts : norm_defaults();
  tdx_status s = check_sizes(T, H, dtype);
  if (s != TDX_OK) return s;
  if (x == nullptr || weight == nullptr || y == nullptr || (h_out != nullptr && residual == nullptr))
    return TDX_ERR_INVALID_ARG;
  if (!known(o.out_dtype) || !(o.eps >= 0.0f) || !std::isfinite(o.eps) || !positive_finite(o.out_scale))
    return TDX_ERR_INVALID_ARG;
  if (row_scale != nullptr && o.out_dtype != TDX_FP8_E4M3) return TDX_ERR_INVALID_ARG;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  const size_t elt = bytes_of(dtype);
  if ((s = row_stride(o.ld_x, H, elt, &p.ld_x)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_residual, H, elt, &p.ld_r)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_h, H, elt, &p.ld_h)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_y, H, bytes_of(o.out_dtype), &p.ld_y)) != TDX_OK) return s;
  if ((H * elt) % 16 != 0 || (H * bytes_of(o.out_dtype)) % 16 != 0) return TDX_ERR_ALIGNMENT;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h_out, 16) || !aligned(y, 16) ||
      !aligned(row_scale, 4) || !aligned(rstd, 4))
    return TDX_ERR_ALIGNMENT;
  if (T == 0) return TDX_OK;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.h = h_out;
  p.y = y;
  p.row_scale = row_scale;
  p.rstd = rstd;
  p.T = T;
  p.H = H;
  p.eps = o.eps;
  p.inv_scale = o.out_dtype == TDX_FP8_E4M3 ? 1.0f / o.out_scale : 1.0f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_norm<bf16>(o.out_dtype, p, st) : launch_norm<float>(o.out_dtype, p, st);
}

tdx_status tdx_rmsnorm_bwd_workspace_size(int T, int H, tdx_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return TDX_ERR_INVALID_ARG;
  const tdx_status s = check_sizes(T, H, dtype);
  if (s != TDX_OK) return s;
  if (H > 32768) return TDX_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(T > 0 ? bwd_parts(T) : 1) * H * sizeof(float);
  return TDX_OK;
}

tdx_status tdx_rmsnorm_bwd(const void* dy, const void* h, const void* weight, const float* rstd, const void* dres,
                           void* dx, float* dweight, void* workspace, size_t workspace_bytes, int T, int H,
                           tdx_dtype dtype, const tdx_norm_opts* opts, void* stream) {
  const tdx_norm_opts o = opts ? *opts : norm_defaults();
  size_t need = 0;
  tdx_status s = tdx_rmsnorm_bwd_workspace_size(T, H, dtype, &need);
  if (s != TDX_OK) return s;
  if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr || dweight == nullptr)
    return TDX_ERR_INVALID_ARG;
  NormBwdParams p;
  std::memset(&p, 0, sizeof(p));
  const size_t elt = bytes_of(dtype);
  if ((s = row_stride(o.ld_x, H, elt, &p.ld_dy)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_residual, H, elt, &p.ld_dres)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_h, H, elt, &p.ld_h)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_y, H, elt, &p.ld_dx)) != TDX_OK) return s;
  if ((H * elt) % 16 != 0) return TDX_ERR_ALIGNMENT;
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dres, 16) || !aligned(dx, 16) ||
      !aligned(dweight, 16) || !aligned(rstd, 4))
    return TDX_ERR_ALIGNMENT;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return TDX_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int parts = bwd_parts(T);
  float* part = static_cast<float*>(workspace);
  if (T > 0) {
    p.dy = dy;
    p.h = h;
    p.weight = weight;
    p.rstd = rstd;
    p.dres = dres;
    p.dx = dx;
    p.part = part;
    p.T = T;
    p.H = H;
    s = dtype == TDX_BF16 ? launch_norm_bwd<bf16>(p, parts, st) : launch_norm_bwd<float>(p, parts, st);
    if (s != TDX_OK) return s;
  }
  return launch_rows(tdx_rmsnorm_dweight_kernel, (H + kThreads - 1) / kThreads, kThreads, 0, st,
                     static_cast<const float*>(part), dweight, parts, H);
}

}  // extern "C"
