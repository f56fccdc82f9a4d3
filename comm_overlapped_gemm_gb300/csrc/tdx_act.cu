// Gated SiLU between two products and its gradient (tdx_swiglu, tdx_swiglu_bwd).
#include <algorithm>

#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kThreads = 128;
constexpr int kWide = 2;          // vectors per thread of a large call
constexpr int kDestBlocks = 24;   // blocks per SM that go round where rows are found through dest

struct ActParams {
  const void* y;
  void* out;
  const void* dout;
  const float* row_scale;
  const int32_t* dest;
  int R, I;
  int per;          // 16-byte vectors of a row of I
  int64_t all;      // vectors of the call, R * per
  uint64_t magic;   // ceil(2^64 / per), 0 for per = 1
  uint64_t magic_k; // the same for topk
  int64_t ld_y, ld_out;
  float inv_scale;
};

// 2^x and 1/x by the special-function unit (2 and 1 ulp), subnormal results 0
__device__ __forceinline__ float power_of_2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a * sigmoid(a) of two values; sigmoid(a) and 1 - sigmoid(a). For fp32 results (kExact) with expf and the IEEE
// quotient, which costs nothing there (65536 x 2048 fp32 224 us either way). For the others exp(-a) = 2^(-a log2 e)
// and the reciprocal are approximate: within 2^-22 * (4 + |a|) relative, |a| < 89, which a rounding to 8 bits hides;
// with the exact forms that kernel is bound by issue slots (262144 x 2048 bf16, one vector per thread: 669 us). The
// divisor is taken times 1/16, so that its reciprocal is no subnormal where exp(-a) is below fp32's largest.
// exp(-a) = inf gives -0 and 0, as the exact quotient does.
constexpr float kLog2e = 1.44269504f, kPart = 0.0625f;
template <bool kExact>
__device__ __forceinline__ f32x2 silu(f32x2 a) {
  if (kExact) return pair(first(a) / (1.0f + expf(-first(a))), second(a) / (1.0f + expf(-second(a))));
  const f32x2 z = mul2(a, pair(-kLog2e, -kLog2e)), part = pair(kPart, kPart);
  const f32x2 d = fma2(pair(power_of_2(first(z)), power_of_2(second(z))), part, part);
  return mul2(mul2(a, part), pair(reciprocal(first(d)), reciprocal(second(d))));
}
template <bool kExact>
__device__ __forceinline__ float sigmoid(float a, float* rest) {
  if (kExact) {
    const float e = expf(-a), s = 1.0f / (1.0f + e);
    *rest = e < INFINITY ? e * s : 1.0f;   // 1 - s without the difference's cancellation
    return s;
  }
  const float s = kPart * reciprocal(fmaf(power_of_2(-kLog2e * a), kPart, kPart));
  *rest = 1.0f - s;
  return s;
}

// i / d as the high half of i * ceil(2^64 / d): exact as long as i * (the product of d and that - 2^64) < 2^64,
// that is i < 2^37 for d up to 2^27
uint64_t magic_of(int d) { return d == 1 ? 0 : ~UINT64_C(0) / d + 1; }
__device__ __forceinline__ int64_t divide(int64_t i, uint64_t magic) {
  return magic != 0 ? static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(i), magic)) : i;
}
// The call's i-th vector: its row (dest not applied) and first column
template <int N>
__device__ __forceinline__ int64_t place(const ActParams& p, int64_t i, int* c) {
  const int64_t r = divide(i, p.magic);
  *c = static_cast<int>(i - r * p.per) * N;
  return r;
}

// Bound by HBM: 6 bytes an element in bf16, 7.2 TB/s at 262144 x 2048 (446 us, a plain copy's rate 482); 8192 x
// 2048 takes 16.1 us of 15.1. The call's vectors are dealt out in the order of their addresses, V x kThreads to
// a block, whatever the row's length; a thread issues all loads of its V vectors before it computes.
// With scalar products: V = 1 / 2 / 4 / 8 with 256 threads 472 / 454 / 468 / 482 us; 128 / 256 / 512 threads with
// V = 2 448 / 454 / 459. In pairs of values, with 128 and 2: 446; 131072 x 2048 to e4m3 199 -> 188.
// kDest: rows are found through dest, which puts a second memory latency in front of a block's loads. So
// blocks go round and look up their next rows and scales while the loads of the present ones are under way:
// 8192 x 2048 18.1 us, 262144 x 2048 502 us; at 18.4 and 506 us a block per piece took 19.6 and 545, 8 (all
// resident) / 10 / 16 blocks per SM that go round 522 / 622 / 509.
template <typename T, typename O, int V, bool kDest>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_launch_dependents();
  int64_t row[V], next_row[V];   // -1: nothing to do
  int col[V], next_col[V];
  float s[V], next_s[V];
  int64_t i = static_cast<int64_t>(blockIdx.x) * (V * kThreads) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (V * kThreads);
  auto find = [&](int64_t from) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t at = from + v * kThreads;
      next_row[v] = -1;
      next_s[v] = 1.0f;
      if (at < p.all) {
        const int64_t r = place<N>(p, at, &next_col[v]);
        next_row[v] = r;
        if (kDest) {
          next_row[v] = p.dest[r];
          if (next_row[v] >= p.R) next_row[v] = -1;
          next_s[v] = p.row_scale[divide(r, p.magic_k)];
        } else if (p.row_scale != nullptr) {
          next_s[v] = p.row_scale[r];
        }
      }
    }
  };
  griddep_wait();
  find(i);
  do {
    uint4 qg[V], qu[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      row[v] = next_row[v];
      col[v] = next_col[v];
      s[v] = next_s[v];
      if (row[v] >= 0) {
        const T* y = static_cast<const T*>(p.y) + row[v] * p.ld_y + col[v];
        qg[v] = __ldcs(reinterpret_cast<const uint4*>(y));
        qu[v] = __ldcs(reinterpret_cast<const uint4*>(y + p.I));
      }
    }
    i += step;
    if (kDest) find(i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (row[v] < 0) continue;
      f32x2 g[N / 2], u[N / 2];
      unpack(qg[v], g, T{});
      unpack(qu[v], u, T{});
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        g[k] = mul2(g[k], pair(s[v], s[v]));
        g[k] = mul2(silu<sizeof(O) == 4>(g[k]), mul2(u[k], pair(s[v], s[v])));
        // the scale last: u / out_scale may be infinite where silu(g) is 0
        if (sizeof(O) == 1) g[k] = mul2(g[k], pair(p.inv_scale, p.inv_scale));
      }
      store_vec(static_cast<O*>(p.out) + row[v] * p.ld_out + col[v], g);
    }
  } while (kDest && i - threadIdx.x < p.all);
}

// As above: 10 bytes an element in bf16, 7.1 TB/s at 65533 x 3584 (330 us, a plain copy's rate 352). dy may be
// y: a thread writes only what it has read.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) tdx_swiglu_bwd_kernel(const __grid_constant__ ActParams p) {
  constexpr int N = kVec<T>;
  griddep_launch_dependents();
  uint4 qg[V], qu[V], qd[V];
  int64_t row[V];
  int col[V];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (V * kThreads) + threadIdx.x;
  griddep_wait();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    row[v] = -1;
    if (i + v * kThreads < p.all) {
      row[v] = place<N>(p, i + v * kThreads, &col[v]);
      const T* y = static_cast<const T*>(p.y) + row[v] * p.ld_y + col[v];
      qg[v] = __ldcs(reinterpret_cast<const uint4*>(y));
      qu[v] = __ldcs(reinterpret_cast<const uint4*>(y + p.I));
      qd[v] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.dout) + row[v] * p.ld_out + col[v]));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (row[v] < 0) continue;
    float g[N], u[N], d[N];
    unpack(qg[v], g, T{});
    unpack(qu[v], u, T{});
    unpack(qd[v], d, T{});
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float rest;
      const float s = sigmoid<sizeof(T) == 4>(g[k], &rest);
      const float ds = d[k] * s;
      d[k] = ds * u[k] * fmaf(g[k], rest, 1.0f);
      u[k] = ds * g[k];
    }
    T* o = static_cast<T*>(p.out) + row[v] * p.ld_y + col[v];
    store_vec(o, d);
    store_vec(o + p.I, u);
  }
}

int act_sms() { return sm_count() > 0 ? sm_count() : kRefSMs; }

// Splits the call into vectors of n elements; whether it is large: enough of them to fill the device four
// times over with kWide per thread (a small call spreads over more SMs with one).
bool act_split(ActParams* p, int n) {
  p->per = p->I / n;
  p->all = static_cast<int64_t>(p->R) * p->per;
  p->magic = magic_of(p->per);
  return p->all >= static_cast<int64_t>(act_sms()) * 2048;
}

unsigned act_grid(const ActParams& p, int V) { return static_cast<unsigned>((p.all + V * kThreads - 1) / (V * kThreads)); }

template <typename T, typename O, int V>
tdx_status launch_act_v(const ActParams& p, cudaStream_t st) {
  const unsigned grid = act_grid(p, V);
  if (p.dest == nullptr) return launch_rows(tdx_swiglu_kernel<T, O, V, false>, grid, kThreads, 0, st, p);
  const unsigned most = static_cast<unsigned>(act_sms() * kDestBlocks);
  return launch_rows(tdx_swiglu_kernel<T, O, V, true>, std::min(grid, most), kThreads, 0, st, p);
}

template <typename T, typename O>
tdx_status launch_act_t(ActParams& p, cudaStream_t st) {
  return act_split(&p, kVec<T>) ? launch_act_v<T, O, kWide>(p, st) : launch_act_v<T, O, 1>(p, st);
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
  if (act_split(&p, kVec<T>)) return launch_rows(tdx_swiglu_bwd_kernel<T, kWide>, act_grid(p, kWide), kThreads, 0, st, p);
  return launch_rows(tdx_swiglu_bwd_kernel<T, 1>, act_grid(p, 1), kThreads, 0, st, p);
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
  if (o.topk > 0) p.magic_k = magic_of(o.topk);
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
