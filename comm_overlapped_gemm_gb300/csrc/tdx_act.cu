// Gated SiLU between two products and its gradient (tdx_swiglu, tdx_swiglu_bwd).
#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kThreads = 256;

struct ActParams {
  const void* y;
  void* out;
  const void* dout;
  const float* row_scale;
  const int32_t* dest;
  int R, I, topk;
  int64_t ld_y, ld_out;
  float inv_scale;
};

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_wait();
  const int per = p.I / N;
  const int64_t all = static_cast<int64_t>(p.R) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i - r * per) * N;
    int64_t row = r;
    float s = 1.0f;
    if (p.dest != nullptr) {
      row = p.dest[r];
      if (row < 0 || row >= p.R) continue;
    }
    if (p.row_scale != nullptr) s = p.row_scale[p.topk > 0 ? r / p.topk : r];
    const T* y = static_cast<const T*>(p.y) + row * p.ld_y + c;
    float g[N], u[N];
    load_vec(y, g);
    load_vec(y + p.I, u);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float a = g[k] * s;
      g[k] = a / (1.0f + expf(-a)) * (u[k] * s) * p.inv_scale;
    }
    store_vec(static_cast<O*>(p.out) + row * p.ld_out + c, g);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_bwd_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_wait();
  const int per = p.I / N;
  const int64_t all = static_cast<int64_t>(p.R) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i - r * per) * N;
    const T* y = static_cast<const T*>(p.y) + r * p.ld_y + c;
    float g[N], u[N], d[N];
    load_vec(y, g);
    load_vec(y + p.I, u);
    load_vec(static_cast<const T*>(p.dout) + r * p.ld_out + c, d);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float s = 1.0f / (1.0f + expf(-g[k]));
      const float du = d[k] * g[k] * s;
      g[k] = d[k] * u[k] * s * fmaf(g[k], 1.0f - s, 1.0f);
      u[k] = du;
    }
    T* o = static_cast<T*>(p.out) + r * p.ld_y + c;
    store_vec(o, g);
    store_vec(o + p.I, u);
  }
}

unsigned act_grid(const ActParams& p, int n) {
  const int64_t blocks = (static_cast<int64_t>(p.R) * (p.I / n) + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(sm_count() > 0 ? sm_count() : kRefSMs) * 8;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
tdx_status launch_act(tdx_dtype out, const ActParams& p, cudaStream_t st) {
  const unsigned grid = act_grid(p, kVec<T>);
  switch (out) {
    case TDX_BF16: return launch_rows(tdx_swiglu_kernel<T, bf16>, grid, kThreads, 0, st, p);
    case TDX_FP32: return launch_rows(tdx_swiglu_kernel<T, float>, grid, kThreads, 0, st, p);
    default: return launch_rows(tdx_swiglu_kernel<T, e4m3>, grid, kThreads, 0, st, p);
  }
}

tdx_act_opts act_defaults() {
  tdx_act_opts o;
  std::memset(&o, 0, sizeof(o));
  o.out_dtype = TDX_BF16;
  o.out_scale = 1.0f;
  return o;
}

// The checks both directions share; fills sizes and strides
tdx_status act_params(int R, int I, tdx_dtype dtype, tdx_dtype out, const tdx_act_opts& o, ActParams* p) {
  if (R < 0 || I <= 0 || I > (1 << 29) || !known(dtype) || !known(out)) return TDX_ERR_INVALID_ARG;
  if (dtype == TDX_FP8_E4M3) return TDX_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  tdx_status s = row_stride(o.ld_y, 2 * static_cast<int64_t>(I), bytes_of(dtype), &p->ld_y);
  if (s != TDX_OK) return s;
  if ((s = row_stride(o.ld_out, I, bytes_of(out), &p->ld_out)) != TDX_OK) return s;
  if ((I * bytes_of(dtype)) % 16 != 0 || (I * bytes_of(out)) % 16 != 0) return TDX_ERR_ALIGNMENT;
  p->R = R;
  p->I = I;
  p->inv_scale = 1.0f;
  return TDX_OK;
}

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_act_opts_default(tdx_act_opts* opts) {
  if (opts == nullptr) return TDX_ERR_INVALID_ARG;
  *opts = act_defaults();
  return TDX_OK;
}

tdx_status tdx_swiglu(const void* y, void* out, const float* row_scale, const int32_t* dest, int R, int I,
                      tdx_dtype dtype, const tdx_act_opts* opts, void* stream) {
  const tdx_act_opts o = opts ? *opts : act_defaults();
  ActParams p;
  const tdx_status s = act_params(R, I, dtype, o.out_dtype, o, &p);
  if (s != TDX_OK) return s;
  if (y == nullptr || out == nullptr || !positive_finite(o.out_scale) || o.topk < 0) return TDX_ERR_INVALID_ARG;
  if ((o.topk > 0) != (dest != nullptr) || (o.topk > 0 && (R % o.topk != 0 || row_scale == nullptr)))
    return TDX_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(row_scale, 4) || !aligned(dest, 4)) return TDX_ERR_ALIGNMENT;
  if (R == 0) return TDX_OK;
  p.y = y;
  p.out = out;
  p.row_scale = row_scale;
  p.dest = dest;
  p.topk = o.topk;
  if (o.out_dtype == TDX_FP8_E4M3) p.inv_scale = 1.0f / o.out_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_act<bf16>(o.out_dtype, p, st) : launch_act<float>(o.out_dtype, p, st);
}

tdx_status tdx_swiglu_bwd(const void* y, const void* dout, void* dy, int R, int I, tdx_dtype dtype,
                          const tdx_act_opts* opts, void* stream) {
  const tdx_act_opts o = opts ? *opts : act_defaults();
  ActParams p;
  const tdx_status s = act_params(R, I, dtype, dtype, o, &p);
  if (s != TDX_OK) return s;
  if (y == nullptr || dout == nullptr || dy == nullptr) return TDX_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(dout, 16) || !aligned(dy, 16)) return TDX_ERR_ALIGNMENT;
  if (R == 0) return TDX_OK;
  p.y = y;
  p.dout = dout;
  p.out = dy;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_rows(tdx_swiglu_bwd_kernel<bf16>, act_grid(p, 8), kThreads, 0, st, p)
                           : launch_rows(tdx_swiglu_bwd_kernel<float>, act_grid(p, 4), kThreads, 0, st, p);
}

}  // extern "C"
