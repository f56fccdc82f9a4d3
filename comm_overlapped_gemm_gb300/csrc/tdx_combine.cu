// Sum of a token's expert rows and its gradient (tdx_moe_combine, tdx_moe_combine_bwd).
#include <algorithm>

#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kThreads = 128;      // forwards
constexpr int kBwdThreads = 256;
constexpr int kFew = 4, kFewSlots = 4;   // forwards, few slots: vectors per thread, most slots

struct CombineParams {
  const void* z;
  const int32_t* dest;
  const float* gates;
  const void* dout;
  void* out;        // forwards out, backwards dZ
  float* dgates;
  int R, T, per, topk;   // per: 16-byte vectors of a row
  int64_t all;           // forwards: vectors of the call
  uint64_t magic;        // of per
  int64_t ld_z, ld_out;
};

// Bound by HBM: topk rows read for one written. The call's vectors are dealt out in the order of their addresses, one
// to a thread: the rows' indexes first, then all its loads (8 at a time) before it adds them in slot order.
// 8192 x 7168, top 8, bf16 165 us (6.4 TB/s); 256 threads 181, 10 blocks per SM 224 for lack of registers.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) tdx_moe_combine_kernel(const __grid_constant__ CombineParams p) {
  constexpr int N = kVec<T>;
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  griddep_wait();
  if (i >= p.all) return;
  const int64_t t = divide(i, p.magic);
  const int c = static_cast<int>(i - t * p.per) * N;
  const int32_t* dest = p.dest + t * p.topk;
  const float* gates = p.gates != nullptr ? p.gates + t * p.topk : nullptr;
  float sum[N] = {};
  for (int j0 = 0; j0 < p.topk; j0 += 8) {
    uint4 q[8];
    int row[8];
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      row[j] = j0 + j < p.topk ? dest[j0 + j] : -1;
      g[j] = gates != nullptr && j0 + j < p.topk ? gates[j0 + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (row[j] >= p.R) row[j] = -1;
      if (row[j] >= 0) q[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.z) + row[j] * p.ld_z + c));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (row[j] < 0) continue;
      float v[N];
      unpack(q[j], v, T{});
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] = fmaf(g[j], v[k], sum[k]);
    }
  }
  store_vec(static_cast<O*>(p.out) + t * p.ld_out + c, sum);
}

// The same for few slots a token: kFew vectors a thread, so that as many loads are in flight. 8192 x 7168, top 2, bf16
// 72 us (with one vector a thread 112), top 4 108 (124), 16384 x 7168, top 1, 115 (203). For top 8 it holds more
// registers and takes 202.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) tdx_moe_combine_few_kernel(const __grid_constant__ CombineParams p) {
  constexpr int N = kVec<T>;
  constexpr int V = kFew, K = 8 / V;   // K: slots whose loads are in flight together
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (V * kThreads) + threadIdx.x;
  int64_t t[V];   // token, -1: none
  int c[V];
  float sum[V][N] = {};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t at = i + v * kThreads;
    t[v] = at < p.all ? divide(at, p.magic) : -1;
    c[v] = static_cast<int>(at - t[v] * p.per) * N;
  }
  griddep_wait();
  for (int j0 = 0; j0 < p.topk; j0 += K) {
    uint4 q[V][K];
    int row[V][K];
    float g[V][K];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const bool is = t[v] >= 0 && j0 + j < p.topk;
        row[v][j] = is ? p.dest[t[v] * p.topk + j0 + j] : -1;
        g[v][j] = is && p.gates != nullptr ? p.gates[t[v] * p.topk + j0 + j] : 1.0f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (row[v][j] >= p.R) row[v][j] = -1;
        if (row[v][j] >= 0)
          q[v][j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.z) + row[v][j] * p.ld_z + c[v]));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (row[v][j] < 0) continue;
        float f[N];
        unpack(q[v][j], f, T{});
#pragma unroll
        for (int k = 0; k < N; ++k) sum[v][k] = fmaf(g[v][j], f[k], sum[v][k]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (t[v] >= 0) store_vec(static_cast<O*>(p.out) + t[v] * p.ld_out + c[v], sum[v]);
}

// A block per token: dout's row once, each of its expert rows once (for the gates' gradient) and
// written once; bound by HBM (8191 x 7168, top 8, bf16 300 us, 6.65 TB/s). The sums over a row go through the lanes and then the warps, in a fixed order.
template <typename T, int K>
__global__ void __launch_bounds__(kBwdThreads) tdx_moe_combine_bwd_kernel(const __grid_constant__ CombineParams p) {
  constexpr int N = kVec<T>;
  constexpr int kWarps = kBwdThreads / 32;
  __shared__ float sm[kWarps][K];
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  griddep_wait();
  int row[K];
  float g[K], dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    row[j] = j < p.topk ? p.dest[t * p.topk + j] : -1;
    if (row[j] >= p.R) row[j] = -1;
    g[j] = p.gates != nullptr && j < p.topk ? p.gates[t * p.topk + j] : 1.0f;
    dot[j] = 0.0f;
  }
  const T* dout = static_cast<const T*>(p.dout) + t * p.ld_out;
  for (int i = threadIdx.x; i < p.per; i += blockDim.x) {
    const int c = i * N;
    float d[N];
    const uint4 qd = __ldcs(reinterpret_cast<const uint4*>(dout + c));
    uint4 q[K];
    if (p.dgates != nullptr) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (row[j] >= 0) q[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.z) + row[j] * p.ld_z + c));
    }
    unpack(qd, d, T{});
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (row[j] < 0) continue;
      if (p.dgates != nullptr) {
        float v[N];
        unpack(q[j], v, T{});
#pragma unroll
        for (int k = 0; k < N; ++k) dot[j] = fmaf(d[k], v[k], dot[j]);
      }
      if (p.out != nullptr) {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = g[j] * d[k];
        store_vec(static_cast<T*>(p.out) + row[j] * p.ld_z + c, v);
      }
    }
  }
  if (p.dgates == nullptr) return;
  const int warps = blockDim.x / 32;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    dot[j] = warp_sum(dot[j]);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5][j] = dot[j];
  }
  __syncthreads();
  if (threadIdx.x < p.topk) {
    float a = 0.0f;
    for (int w = 0; w < warps; ++w) a += sm[w][threadIdx.x];
    p.dgates[t * p.topk + threadIdx.x] = a;
  }
}

// Several vectors a thread where a token has few slots, unless SMs would then be left without blocks
template <typename T, typename O>
tdx_status launch_fwd(const CombineParams& p, cudaStream_t st) {
  const int sms = sm_count() > 0 ? sm_count() : kRefSMs;
  const bool few = p.topk <= kFewSlots && p.all >= static_cast<int64_t>(sms) * kThreads * 4 * kFew;
  const int64_t each = few ? kFew * kThreads : kThreads, blocks = (p.all + each - 1) / each;
  if (blocks > 0x7FFFFFFF) return TDX_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  return few ? launch_rows(tdx_moe_combine_few_kernel<T, O>, grid, kThreads, 0, st, p)
             : launch_rows(tdx_moe_combine_kernel<T, O>, grid, kThreads, 0, st, p);
}

template <typename T>
tdx_status launch_bwd(const CombineParams& p, cudaStream_t st) {
  const unsigned threads = static_cast<unsigned>(std::min(kBwdThreads, (p.per + 31) / 32 * 32));
  const unsigned grid = static_cast<unsigned>(p.T);
  if (p.topk <= 4) return launch_rows(tdx_moe_combine_bwd_kernel<T, 4>, grid, threads, 0, st, p);
  if (p.topk <= 8) return launch_rows(tdx_moe_combine_bwd_kernel<T, 8>, grid, threads, 0, st, p);
  return launch_rows(tdx_moe_combine_bwd_kernel<T, 16>, grid, threads, 0, st, p);
}

tdx_combine_opts combine_defaults() {
  tdx_combine_opts o;
  std::memset(&o, 0, sizeof(o));
  o.out_dtype = TDX_BF16;
  return o;
}

// The checks both directions share; fills sizes and strides. out: the type of the rows of T
tdx_status combine_params(int R, int T, int H, int topk, tdx_dtype dtype, tdx_dtype out, const tdx_combine_opts& o,
                          CombineParams* p) {
  if (R < 0 || T < 0 || H <= 0 || topk < 1 || topk > kMoeMaxTopk || !known(dtype) || !known(out))
    return TDX_ERR_INVALID_ARG;
  if (dtype == TDX_FP8_E4M3 || out == TDX_FP8_E4M3) return TDX_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  tdx_status s = row_stride(o.ld_z, H, bytes_of(dtype), &p->ld_z);
  if (s != TDX_OK) return s;
  if ((s = row_stride(o.ld_out, H, bytes_of(out), &p->ld_out)) != TDX_OK) return s;
  if (H * bytes_of(dtype) % 16 != 0 || H * bytes_of(out) % 16 != 0) return TDX_ERR_ALIGNMENT;
  p->R = R;
  p->T = T;
  p->topk = topk;
  p->per = static_cast<int>(H * bytes_of(dtype) / 16);
  p->all = static_cast<int64_t>(T) * p->per;
  p->magic = magic_of(p->per);
  return TDX_OK;
}

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_combine_opts_default(tdx_combine_opts* opts) {
  if (opts == nullptr) return TDX_ERR_INVALID_ARG;
  *opts = combine_defaults();
  return TDX_OK;
}

tdx_status tdx_moe_combine(const void* Z, const int32_t* dest, const float* gates, void* out, int R, int T, int H,
                           int topk, tdx_dtype dtype, const tdx_combine_opts* opts, void* stream) {
  const tdx_combine_opts o = opts ? *opts : combine_defaults();
  CombineParams p;
  const tdx_status s = combine_params(R, T, H, topk, dtype, o.out_dtype, o, &p);
  if (s != TDX_OK) return s;
  // tensors of no rows (Z: R = 0, the others: T = 0) have no address
  if ((R > 0 && Z == nullptr) || (T > 0 && (dest == nullptr || out == nullptr))) return TDX_ERR_INVALID_ARG;
  if (!aligned(Z, 16) || !aligned(out, 16) || !aligned(dest, 4) || !aligned(gates, 4)) return TDX_ERR_ALIGNMENT;
  if (T == 0) return TDX_OK;
  p.z = Z;
  p.dest = dest;
  p.gates = gates;
  p.out = out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == TDX_BF16) return o.out_dtype == TDX_BF16 ? launch_fwd<bf16, bf16>(p, st) : launch_fwd<bf16, float>(p, st);
  return o.out_dtype == TDX_BF16 ? launch_fwd<float, bf16>(p, st) : launch_fwd<float, float>(p, st);
}

tdx_status tdx_moe_combine_bwd(const void* dout, const void* Z, const int32_t* dest, const float* gates, void* dZ,
                               float* dgates, int R, int T, int H, int topk, tdx_dtype dtype,
                               const tdx_combine_opts* opts, void* stream) {
  const tdx_combine_opts o = opts ? *opts : combine_defaults();
  CombineParams p;
  const tdx_status s = combine_params(R, T, H, topk, dtype, dtype, o, &p);
  if (s != TDX_OK) return s;
  // tensors of no rows (Z and dZ: R = 0, the others: T = 0) have no address
  if (T > 0 && (dout == nullptr || dest == nullptr || (R > 0 && dZ == nullptr && dgates == nullptr) ||
                (R > 0 && dgates != nullptr && Z == nullptr)))
    return TDX_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(Z, 16) || !aligned(dZ, 16) || !aligned(dest, 4) || !aligned(gates, 4) ||
      !aligned(dgates, 4))
    return TDX_ERR_ALIGNMENT;
  if (T == 0) return TDX_OK;
  p.z = Z;
  p.dest = dest;
  p.gates = gates;
  p.dout = dout;
  p.out = dZ;
  p.dgates = dgates;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_bwd<bf16>(p, st) : launch_bwd<float>(p, st);
}

}  // extern "C"
