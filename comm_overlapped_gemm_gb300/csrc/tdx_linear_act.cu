// Gradient of the linear layer's activation and bias (tdx_linear_act_bwd).
#include <algorithm>

#include "tdx_actmath.cuh"
#include "tdx_linear.h"
#include "tdx_rows.cuh"

namespace tdx {

tdx_linear_opts linear_defaults();

namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;       // rows whose loads a thread has in flight
constexpr int kMostBlocks = 912;    // 6 blocks for each of 152 SMs

struct ActBwdParams {
  const bf16* dy;
  const bf16* z;
  bf16* dz;
  float* part;      // [row groups][N], or dbias itself for one group; NULL: no sums
  int M, cols;
  int lanes;        // lanes of a row, a power of two; threads / lanes rows at a time
  int64_t ld_dy, ld_z;
};

// sigmoid of two values whose exponents times -log2(e) are z, and what is left to 1
__device__ __forceinline__ f32x2 sigmoid2(f32x2 z, f32x2* rest) {
  const f32x2 part = pair(kPart, kPart);
  const f32x2 d = fma2(pair(power_of_2(first(z)), power_of_2(second(z))), part, part);
  const f32x2 s = mul2(part, pair(reciprocal(first(d)), reciprocal(second(d))));
  *rest = fma2(s, pair(-1.0f, -1.0f), pair(1.0f, 1.0f));
  return s;
}

// dz of two values z (gates), given dy; SWIGLU alone uses u, and leaves its gradient there. In pairs: one value at a
// time, 73% of the issue slots held the loads up (16381 x 8192 GELU_TANH 133 us).
template <int ACT>
__device__ __forceinline__ void act_backward(f32x2& dy, f32x2 x, f32x2& u) {
  auto both = [](float v) { return pair(v, v); };
  f32x2 rest;
  if (ACT == TDX_ACT_RELU) {
    dy = pair(first(x) > 0.0f ? first(dy) : 0.0f, second(x) > 0.0f ? second(dy) : 0.0f);
  } else if (ACT == TDX_ACT_GELU) {
    auto one = [](float v) {
      return fmaf(v * kInvRoot2Pi, power_of_2(-0.5f * kLog2e * v * v), 0.5f * erfcf(-kHalfRoot * v));
    };
    dy = mul2(dy, pair(one(first(x)), one(second(x))));
  } else if (ACT == TDX_ACT_GELU_TANH) {
    // past 16 the derivative is 0 or 1, and x^2 would overflow for values of a mask; a NaN stays
    auto near = [](float v) { return fabsf(v) > 16.0f ? copysignf(16.0f, v) : v; };
    x = pair(near(first(x)), near(second(x)));
    const f32x2 square = mul2(x, x);
    const f32x2 z = mul2(x, fma2(both(-kLog2e * kGelu2 * kGeluCube), square, both(-kLog2e * kGelu2)));
    const f32x2 s = sigmoid2(z, &rest);
    const f32x2 slope = fma2(both(3.0f * kGelu2 * kGeluCube), square, both(kGelu2));
    dy = mul2(mul2(dy, s), fma2(mul2(x, rest), slope, both(1.0f)));
  } else if (ACT == TDX_ACT_SILU || ACT == TDX_ACT_SWIGLU) {
    const f32x2 ds = mul2(dy, sigmoid2(mul2(x, both(-kLog2e)), &rest));
    dy = mul2(ds, fma2(x, rest, both(1.0f)));
    if (ACT == TDX_ACT_SWIGLU) {
      dy = mul2(dy, u);
      u = mul2(ds, x);
    }
  }
}

// Bound by HBM. A warp reads whole lines of a row (several rows where a row is short), a thread keeps the
// sums of its 8 columns (16 for SWIGLU) in registers over its rows; they are joined in shared memory
// in a fixed order. 16381 x 8192 GELU_TANH with dbias 128 us (6.3 TB/s), SWIGLU 111. Blocks with chunks of
// neighbouring rows, each reading a front of its own, took 136; the next rows' loads in front of the present ones' work
// 139 to 158 (more rows in flight, fewer hits of open DRAM pages); 4 blocks of 64 registers per SM 140.
template <int ACT>
__global__ void __launch_bounds__(kThreads) tdx_linear_act_bwd_kernel(const __grid_constant__ ActBwdParams p) {
  constexpr bool kGated = ACT == TDX_ACT_SWIGLU;
  constexpr int kSums = kGated ? 16 : 8;
  __shared__ float sm[kThreads][kSums + 1];
  griddep_launch_dependents();
  const int at = threadIdx.x % p.lanes, sub = threadIdx.x / p.lanes, step = kThreads / p.lanes;
  const int col = (blockIdx.x * p.lanes + at) * 8;
  const bool mine = col < p.cols;
  f32x2 sum[kSums / 2] = {};
  griddep_wait();
  if (mine) {
    // the row groups take turns, so that the blocks at work together read one front of the rows
    const int64_t turn = static_cast<int64_t>(gridDim.y) * kRowsAhead * step;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * kRowsAhead * step + sub; r0 < p.M; r0 += turn) {
      uint4 qd[kRowsAhead], qz[kRowsAhead], qu[kRowsAhead];
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        const int64_t r = r0 + k * step;
        if (r < p.M) {
          qd[k] = __ldcs(reinterpret_cast<const uint4*>(p.dy + r * p.ld_dy + col));
          if (ACT != TDX_ACT_NONE) qz[k] = __ldcs(reinterpret_cast<const uint4*>(p.z + r * p.ld_z + col));
          if (kGated) qu[k] = __ldcs(reinterpret_cast<const uint4*>(p.z + r * p.ld_z + p.cols + col));
        }
      }
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        const int64_t r = r0 + k * step;
        if (r < p.M) {
          f32x2 d[4], z[4], u[4];
          unpack(qd[k], d, bf16{});
          if (ACT != TDX_ACT_NONE) unpack(qz[k], z, bf16{});
          if (kGated) unpack(qu[k], u, bf16{});
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            act_backward<ACT>(d[i], z[i], u[i]);
            sum[i] = add2(sum[i], d[i]);
            if (kGated) sum[kSums / 2 - 4 + i] = add2(sum[kSums / 2 - 4 + i], u[i]);
          }
          if (p.dz != nullptr) {
            store_vec(p.dz + r * p.ld_z + col, d);
            if (kGated) store_vec(p.dz + r * p.ld_z + p.cols + col, u);
          }
        }
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int i = 0; i < kSums / 2; ++i) {
    sm[threadIdx.x][2 * i] = first(sum[i]);
    sm[threadIdx.x][2 * i + 1] = second(sum[i]);
  }
  __syncthreads();
  const int64_t row = static_cast<int64_t>(blockIdx.y) * (kGated ? 2 : 1) * p.cols;
  for (int i = threadIdx.x; i < p.lanes * kSums; i += kThreads) {
    const int lane = i / kSums, k = i % kSums;
    const int c = (blockIdx.x * p.lanes + lane) * 8 + (k & 7);
    if (c >= p.cols) continue;
    float a = 0.0f;
    for (int s = 0; s < step; ++s) a += sm[s * p.lanes + lane][k];
    p.part[row + c + (k >= 8 ? p.cols : 0)] = a;
  }
}

int lanes_of(int cols) {
  int n = 1;
  while (n < 32 && n * 8 < cols) n *= 2;
  return n;
}
int col_blocks(int cols) { return (cols + lanes_of(cols) * 8 - 1) / (lanes_of(cols) * 8); }

// Row groups: as many as kMostBlocks allows, but none without rows for every thread's loads
int groups_of(int M, int cols) {
  const int64_t turn = kThreads / lanes_of(cols) * kRowsAhead;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMostBlocks / col_blocks(cols), (M + turn - 1) / turn)));
}

tdx_status launch_act(tdx_activation act, const ActBwdParams& p, dim3 grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  switch (act) {
    case TDX_ACT_RELU: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_RELU>, p); break;
    case TDX_ACT_GELU: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_GELU>, p); break;
    case TDX_ACT_GELU_TANH: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_GELU_TANH>, p); break;
    case TDX_ACT_SILU: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_SILU>, p); break;
    case TDX_ACT_SWIGLU: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_SWIGLU>, p); break;
    default: e = cudaLaunchKernelEx(&cfg, tdx_linear_act_bwd_kernel<TDX_ACT_NONE>, p); break;
  }
  return e == cudaSuccess ? TDX_OK : TDX_ERR_CUDA;
}

tdx_status check_sizes(int M, int N, tdx_dtype dtype, const tdx_linear_opts& o) {
  if (M < 0 || N <= 0 || !known(dtype) || o.act < TDX_ACT_NONE || o.act > TDX_ACT_SWIGLU) return TDX_ERR_INVALID_ARG;
  if (o.act == TDX_ACT_SWIGLU && N % 2 != 0) return TDX_ERR_INVALID_ARG;
  return dtype != TDX_BF16 || M > (1 << 30) || N > (1 << 28) ? TDX_ERR_UNSUPPORTED : TDX_OK;
}

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_linear_act_bwd_workspace_size(int M, int N, tdx_dtype dtype, const tdx_linear_opts* opts, size_t* bytes) {
  if (bytes == nullptr) return TDX_ERR_INVALID_ARG;
  const tdx_linear_opts o = opts ? *opts : linear_defaults();
  const tdx_status s = check_sizes(M, N, dtype, o);
  if (s != TDX_OK) return s;
  *bytes = static_cast<size_t>(groups_of(M, o.act == TDX_ACT_SWIGLU ? N / 2 : N)) * N * sizeof(float);
  return TDX_OK;
}

tdx_status tdx_linear_act_bwd(const void* dy, const void* z, void* dz, float* dbias, void* workspace,
                              size_t workspace_bytes, int M, int N, tdx_dtype dtype, const tdx_linear_opts* opts,
                              void* stream) {
  const tdx_linear_opts o = opts ? *opts : linear_defaults();
  size_t need = 0;
  tdx_status s = tdx_linear_act_bwd_workspace_size(M, N, dtype, &o, &need);
  if (s != TDX_OK) return s;
  const bool gated = o.act == TDX_ACT_SWIGLU;
  // tensors of M = 0 rows have no address
  if (M > 0 && (dy == nullptr || (dz == nullptr && dbias == nullptr) || (o.act != TDX_ACT_NONE && z == nullptr)))
    return TDX_ERR_INVALID_ARG;
  ActBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.cols = gated ? N / 2 : N;
  if ((s = row_stride(o.ld_c, p.cols, 2, &p.ld_dy)) != TDX_OK || (s = row_stride(o.ld_z, N, 2, &p.ld_z)) != TDX_OK)
    return s;
  if (p.cols % 8 != 0) return TDX_ERR_ALIGNMENT;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16) || !aligned(dbias, 16)) return TDX_ERR_ALIGNMENT;
  if (dbias != nullptr && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need))
    return TDX_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int groups = groups_of(M, p.cols);
  if (M == 0 && dbias == nullptr) return TDX_OK;
  p.dy = static_cast<const bf16*>(dy);
  p.z = static_cast<const bf16*>(z);
  p.dz = static_cast<bf16*>(dz);
  p.M = M;
  p.lanes = lanes_of(p.cols);
  if (dbias != nullptr) p.part = groups > 1 ? static_cast<float*>(workspace) : dbias;
  s = launch_act(o.act, p, dim3(static_cast<unsigned>(col_blocks(p.cols)), static_cast<unsigned>(groups), 1), st);
  if (s != TDX_OK || dbias == nullptr || groups == 1) return s;
  return launch_sum_parts(static_cast<const float*>(workspace), dbias, groups, N, st);
}

}  // extern "C"
