// Gated SiLU between two products and its gradient (tdx_swiglu, tdx_swiglu_bwd).
#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kThreads = 256;
// Vectors per thread of a large call. 1 / 2 / 4 / 8: forwards 262144 x 2048 472 / 454 / 468 / 482 us and
// 8192 x 2048 (scaled by token) 19.6 / 19.5 / 22.0 / 31.9 us, backwards 65533 x 3584 333 / 329 / 330 /
// 393 us (bf16).
constexpr int kWide = 2;

struct ActParams {
  const void* y;
  void* out;
  const void* dout;
  const float* row_scale;
  const int32_t* dest;
  int R, I, topk;
  int cols;        // 16-byte vectors of a row that a block takes
  int rows;        // rows that a block takes
  int col_blocks;  // blocks along a row
  int magic;       // ceil(2^20 / cols): l / cols = l * magic >> 20 for l and cols up to 1024
  int64_t ld_y, ld_out;
  float inv_scale;
};

// a * sigmoid(a) with the approximate exponential and quotient: together within 2^-22 * (2 + |a|) of
// it, far inside the output's rounding (bf16, e4m3) or of the order of fp32's own (8 roundings at
// |a| = 1). exp(-a) = inf gives -0, as the exact quotient does. The exact expf and quotient took the
// kernel from memory-bound to issue-bound (262144 x 2048 bf16: 669 us).
__device__ __forceinline__ float silu(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

// The block's l-th vector: its row of the call (dest not applied) and its first column
template <int N>
__device__ __forceinline__ bool place(const ActParams& p, int l, int rb, int cb, int64_t* r, int* c) {
  const int lr = (l * p.magic) >> 20;
  *r = static_cast<int64_t>(rb) * p.rows + lr;
  *c = (cb * p.cols + l - lr * p.cols) * N;
  return lr < p.rows && *r < p.R && *c < p.I;
}

// Bound by HBM: 6 bytes an element in bf16, 7.1 TB/s at 262144 x 2048 (454 us, a plain copy's rate 482);
// 8192 x 2048 takes 19.5 us of 15.1, the launch's ramp and tail the rest. Each thread issues all loads of its
// V vectors before it computes, so that a block has 2 V x 4 KiB in flight; a block takes whole rows where
// they are short and a stretch of one row where they are long, which leaves a multiplication and a shift to
// find a vector's row.
template <typename T, typename O, int V>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_launch_dependents();
  const int rb = blockIdx.x / p.col_blocks, cb = blockIdx.x - rb * p.col_blocks;
  uint4 qg[V], qu[V];
  int64_t row[V];
  int col[V];
  bool on[V];
  float s[V];
  griddep_wait();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    int64_t r;
    on[v] = place<N>(p, v * kThreads + threadIdx.x, rb, cb, &r, &col[v]);
    row[v] = r;
    s[v] = 1.0f;
    if (on[v] && p.row_scale != nullptr) {
      if (p.dest != nullptr) {
        row[v] = p.dest[r];
        on[v] = row[v] >= 0 && row[v] < p.R;
        r /= p.topk;
      }
      s[v] = p.row_scale[r];
    }
    if (on[v]) {
      const T* y = static_cast<const T*>(p.y) + row[v] * p.ld_y + col[v];
      qg[v] = __ldcs(reinterpret_cast<const uint4*>(y));
      qu[v] = __ldcs(reinterpret_cast<const uint4*>(y + p.I));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!on[v]) continue;
    float g[N], u[N];
    unpack(qg[v], g, T{});
    unpack(qu[v], u, T{});
    const float su = s[v] * p.inv_scale;
#pragma unroll
    for (int k = 0; k < N; ++k) g[k] = silu(g[k] * s[v]) * (u[k] * su);
    store_vec(static_cast<O*>(p.out) + row[v] * p.ld_out + col[v], g);
  }
}

// As above: 10 bytes an element in bf16, 7.1 TB/s at 65533 x 3584 (329 us). dy may be y: a thread writes only what it has read.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_bwd_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_launch_dependents();
  const int rb = blockIdx.x / p.col_blocks, cb = blockIdx.x - rb * p.col_blocks;
  uint4 qg[V], qu[V], qd[V];
  int64_t row[V];
  int col[V];
  bool on[V];
  griddep_wait();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    on[v] = place<N>(p, v * kThreads + threadIdx.x, rb, cb, &row[v], &col[v]);
    if (on[v]) {
      const T* y = static_cast<const T*>(p.y) + row[v] * p.ld_y + col[v];
      qg[v] = __ldcs(reinterpret_cast<const uint4*>(y));
      qu[v] = __ldcs(reinterpret_cast<const uint4*>(y + p.I));
      qd[v] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.dout) + row[v] * p.ld_out + col[v]));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!on[v]) continue;
    float g[N], u[N], d[N];
    unpack(qg[v], g, T{});
    unpack(qu[v], u, T{});
    unpack(qd[v], d, T{});
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-g[k]));
      const float ds = d[k] * s;
      d[k] = ds * u[k] * fmaf(g[k], 1.0f - s, 1.0f);
      u[k] = ds * g[k];
    }
    T* o = static_cast<T*>(p.out) + row[v] * p.ld_y + col[v];
    store_vec(o, d);
    store_vec(o + p.I, u);
  }
}

// Split the call into blocks of about V * kThreads vectors; returns the grid.
unsigned act_split(ActParams* p, int n, int V) {
  const int per = p->I / n, most = V * kThreads;
  p->cols = per < most ? per : most;
  p->rows = most / p->cols;
  p->col_blocks = (per + p->cols - 1) / p->cols;
  p->magic = ((1 << 20) + p->cols - 1) / p->cols;
  return static_cast<unsigned>((static_cast<int64_t>(p->R) + p->rows - 1) / p->rows * p->col_blocks);
}

// kWide vectors per thread once that fills the device four times over, else one, so that small calls spread
// over more SMs
bool act_large(const ActParams& p, int n) {
  const int sms = sm_count() > 0 ? sm_count() : kRefSMs;
  return static_cast<int64_t>(p.R) * (p.I / n) >= static_cast<int64_t>(sms) * 8 * kThreads;
}

template <typename T, typename O>
tdx_status launch_act_t(ActParams& p, cudaStream_t st) {
  if (act_large(p, kVec<T>)) {
    const unsigned grid = act_split(&p, kVec<T>, kWide);
    return launch_rows(tdx_swiglu_kernel<T, O, kWide>, grid, kThreads, 0, st, p);
  }
  const unsigned grid = act_split(&p, kVec<T>, 1);
  return launch_rows(tdx_swiglu_kernel<T, O, 1>, grid, kThreads, 0, st, p);
}

template <typename T>
tdx_status launch_act(tdx_dtype out, ActParams& p, cudaStream_t st) {
  switch (out) {
    case TDX_BF16: return launch_act_t<T, bf16>(p, st);
    case TDX_FP32: return launch_act_t<T, float>(p, st);
    default: return launch_act_t<T, e4m3>(p, st);
  }
}

template <typename T>
tdx_status launch_act_bwd(ActParams& p, cudaStream_t st) {
  if (act_large(p, kVec<T>)) {
    const unsigned grid = act_split(&p, kVec<T>, kWide);
    return launch_rows(tdx_swiglu_bwd_kernel<T, kWide>, grid, kThreads, 0, st, p);
  }
  const unsigned grid = act_split(&p, kVec<T>, 1);
  return launch_rows(tdx_swiglu_bwd_kernel<T, 1>, grid, kThreads, 0, st, p);
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
  if (y == nullptr || out == nullptr || !usable_scale(o.out_scale) || o.topk < 0) return TDX_ERR_INVALID_ARG;
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
  return dtype == TDX_BF16 ? launch_act_bwd<bf16>(p, st) : launch_act_bwd<float>(p, st);
}

}  // extern "C"
