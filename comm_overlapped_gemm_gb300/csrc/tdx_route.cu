// Routing of tokens to experts and its gradient (tdx_moe_route, tdx_moe_route_bwd).
#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* gates;
  int32_t* counts;
  const float* dgates;
  void* dlogits;
  int T, E, k;
  int n_group, topk_group, group_top;
  int sigmoid, renorm;
  float scale;
  int64_t ld;
};

// 1 / (1 + exp(-x)), each step rounded to fp32 (no contraction of exp's last product into the sum)
__device__ __forceinline__ float sigmoid_rn(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

// Order-preserving image of a float: larger key, larger integer; NaN comes last (1), 0 is left for
// "taken or not in a chosen group". -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (f != f) return 1u;
  const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One warp per token; the row's scores and keys in shared memory, E floats each.
template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ float sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  float* score = sm + warp * 2 * E;
  uint32_t* key = reinterpret_cast<uint32_t*>(score + E);
  griddep_wait();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const T* x = static_cast<const T*>(p.logits) + t * p.ld;
    float m = -INFINITY, sum = 1.0f;
    bool nan = false;
    if (!p.sigmoid) {
      for (int e = lane; e < E; e += 32) {
        const float v = to_float(x[e]);
        m = fmaxf(m, v);
        nan |= v != v;
      }
      m = warp_max(m);
      nan = __any_sync(kAll, nan);
      sum = 0.0f;
      for (int e = lane; e < E; e += 32) sum += expf(to_float(x[e]) - m);
      sum = warp_sum(sum);
    }
    for (int e = lane; e < E; e += 32) {
      const float v = to_float(x[e]);
      float s, k;
      if (p.sigmoid) {
        s = sigmoid_rn(v);
        k = p.bias ? __fadd_rn(s, p.bias[e]) : s;
      } else {
        s = v;
        k = p.bias ? __fadd_rn(__fdiv_rn(expf(__fadd_rn(v, -m)), sum), p.bias[e]) : v;
      }
      score[e] = s;
      key[e] = ordered(k);
    }
    __syncwarp();
    if (p.n_group > 1) {
      // lane g scores group g; a group is chosen if fewer than topk_group groups come before it
      const int per = E / p.n_group;
      float gs = -INFINITY;
      uint32_t gk = 0;
      if (lane < p.n_group) {
        uint32_t k1 = 0, k2 = 0;
        for (int i = 0; i < per; ++i) {
          const uint32_t k = key[lane * per + i];
          if (k > k1) {
            k2 = k1;
            k1 = k;
          } else if (k > k2) {
            k2 = k;
          }
        }
        gk = k1;
        if (p.group_top == 2) {
          auto back = [](uint32_t k) { return k == 1u ? NAN : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); };
          float a = back(k1), b = per > 1 ? back(k2) : 0.0f;
          if (!p.sigmoid && p.bias == nullptr) {
            a = expf(__fadd_rn(a, -m));
            b = per > 1 ? expf(__fadd_rn(b, -m)) : 0.0f;
          }
          gs = __fadd_rn(a, b);
          gk = ordered(gs);
        }
      }
      int before = 0;
      for (int g = 0; g < p.n_group; ++g) {
        const uint32_t o = __shfl_sync(kAll, gk, g);
        before += (o > gk || (o == gk && g < lane)) ? 1 : 0;
      }
      const unsigned keep = __ballot_sync(kAll, lane < p.n_group && before < p.topk_group);
      for (int e = lane; e < E; e += 32)
        if (!((keep >> (e / per)) & 1u)) key[e] = 0;
      __syncwarp();
    }
    int mine = 0;   // lane j: the j-th chosen expert
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0;
      int at = E;
      for (int e = lane; e < E; e += 32)
        if (key[e] > best) {
          best = key[e];
          at = e;
        }
      const uint32_t top = __reduce_max_sync(kAll, best);
      const int e = static_cast<int>(__reduce_min_sync(kAll, best == top ? static_cast<uint32_t>(at) : kAll));
      if (lane == j) mine = e;
      if (lane == 0) key[e] = 0;
      __syncwarp();
    }
    const bool on = lane < p.k;
    float s = 0.0f, den = 1.0f;
    if (p.sigmoid) {
      s = on ? score[mine] : 0.0f;
      if (p.renorm) den = warp_sum(s);
    } else {
      // renormalised softmax is the softmax over the chosen logits, taken from their own maximum
      const float v = on ? score[mine] : -INFINITY;
      const float top = p.renorm ? warp_max(v) : m;
      s = top == -INFINITY ? 0.0f : expf(v - top);
      den = p.renorm ? warp_sum(s) : sum;
    }
    float g = s == 0.0f ? 0.0f : s / den * p.scale;
    if (nan) g = NAN;
    if (on) {
      p.idx[t * p.k + lane] = mine;
      p.gates[t * p.k + lane] = g;
      if (p.counts != nullptr) atomicAdd(p.counts + mine, 1);
    }
    __syncwarp();
  }
}

// One warp per token; lane j holds the j-th id and its coefficient.
template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_moe_route_bwd_kernel(const __grid_constant__ RouteParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const T* x = static_cast<const T*>(p.logits) + t * p.ld;
    T* dx = static_cast<T*>(p.dlogits) + t * p.ld;
    int id = lane < p.k ? p.idx[t * p.k + lane] : -1;
    if (id >= p.E) id = -1;
    const bool on = id >= 0;
    const float v = on ? to_float(x[id]) : -INFINITY;
    const float dg = on ? p.dgates[t * p.k + lane] * p.scale : 0.0f;
    float m = -INFINITY, inv = 0.0f;   // dense softmax: p_e = exp(x_e - m) * inv
    float d = 0.0f;                    // what the chosen expert receives
    float dot = 0.0f;
    const bool dense = !p.sigmoid && !p.renorm;
    if (p.sigmoid) {
      const float s = on ? 1.0f / (1.0f + expf(-v)) : 0.0f;
      const float q = on ? 1.0f / (1.0f + expf(v)) : 0.0f;
      float c = dg;
      if (p.renorm) {
        const float S = warp_sum(s);
        c = S > 0.0f ? (dg - warp_sum(dg * s) / S) / S : 0.0f;
      }
      d = c * s * q;
    } else if (p.renorm) {
      m = warp_max(v);
      const float e = on && m > -INFINITY ? expf(v - m) : 0.0f;
      const float S = warp_sum(e);
      const float g = S > 0.0f ? e / S : 0.0f;
      d = g * (dg - warp_sum(dg * g));
    } else {
      for (int e = lane; e < p.E; e += 32) m = fmaxf(m, to_float(x[e]));
      m = warp_max(m);
      float S = 0.0f;
      for (int e = lane; e < p.E; e += 32) S += expf(to_float(x[e]) - m);
      S = warp_sum(S);
      inv = m > -INFINITY ? 1.0f / S : 0.0f;
      d = dg;
      dot = warp_sum(on && inv > 0.0f ? dg * expf(v - m) * inv : 0.0f);
    }
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      float a = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int ij = __shfl_sync(kAll, id, j);
        const float dj = __shfl_sync(kAll, d, j);
        if (ij == e) a += dj;
      }
      if (e < p.E) {
        if (dense) a = inv > 0.0f ? expf(to_float(x[e]) - m) * inv * (a - dot) : 0.0f;
        dx[e] = static_cast<T>(a);
      }
    }
  }
}

tdx_route_opts route_defaults() {
  tdx_route_opts o;
  std::memset(&o, 0, sizeof(o));
  o.score = TDX_SCORE_SOFTMAX;
  o.n_group = 1;
  o.topk_group = 1;
  o.group_top = 1;
  o.renorm = 1;
  o.scale = 1.0f;
  return o;
}

// The checks both directions share; fills sizes, options and the stride
tdx_status route_params(int T, int E, int topk, tdx_dtype dtype, const tdx_route_opts& o, RouteParams* p) {
  if (T < 0 || E <= 0 || topk < 1 || topk > E || !known(dtype)) return TDX_ERR_INVALID_ARG;
  if (o.score != TDX_SCORE_SOFTMAX && o.score != TDX_SCORE_SIGMOID) return TDX_ERR_INVALID_ARG;
  if (o.n_group < 1 || E % o.n_group != 0 || o.topk_group < 1 || o.topk_group > o.n_group) return TDX_ERR_INVALID_ARG;
  if (o.group_top != 1 && o.group_top != 2) return TDX_ERR_INVALID_ARG;
  if ((o.renorm != 0 && o.renorm != 1) || !std::isfinite(o.scale)) return TDX_ERR_INVALID_ARG;
  if (dtype == TDX_FP8_E4M3 || E > kMoeMaxExperts || topk > kMoeMaxTopk || o.n_group > 32) return TDX_ERR_UNSUPPORTED;
  const int64_t ld = o.ld_logits == 0 ? E : o.ld_logits;
  if (ld < E || ld > (INT64_C(1) << 40)) return TDX_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  p->T = T;
  p->E = E;
  p->k = topk;
  p->n_group = o.n_group;
  p->topk_group = o.topk_group;
  p->group_top = o.group_top;
  p->sigmoid = o.score == TDX_SCORE_SIGMOID;
  p->renorm = o.renorm;
  p->scale = o.scale;
  p->ld = ld;
  return TDX_OK;
}

unsigned route_grid(int T) {
  const int blocks = (T + kWarps - 1) / kWarps;
  const int most = (sm_count() > 0 ? sm_count() : kRefSMs) * 8;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_route_opts_default(tdx_route_opts* opts) {
  if (opts == nullptr) return TDX_ERR_INVALID_ARG;
  *opts = route_defaults();
  return TDX_OK;
}

tdx_status tdx_moe_route(const void* logits, const float* bias, int32_t* topk_idx, float* gates, int32_t* counts, int T,
                         int E, int topk, tdx_dtype dtype, const tdx_route_opts* opts, void* stream) {
  const tdx_route_opts o = opts ? *opts : route_defaults();
  RouteParams p;
  const tdx_status s = route_params(T, E, topk, dtype, o, &p);
  if (s != TDX_OK) return s;
  if (logits == nullptr || topk_idx == nullptr || gates == nullptr) return TDX_ERR_INVALID_ARG;
  if (static_cast<int64_t>(topk) > static_cast<int64_t>(o.topk_group) * (E / o.n_group)) return TDX_ERR_INVALID_ARG;
  if (!aligned(logits, static_cast<unsigned>(bytes_of(dtype))) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(gates, 4) || !aligned(counts, 4))
    return TDX_ERR_ALIGNMENT;
  if (T == 0) return TDX_OK;
  p.logits = logits;
  p.bias = bias;
  p.idx = topk_idx;
  p.gates = gates;
  p.counts = counts;
  const size_t smem = static_cast<size_t>(kWarps) * 2 * E * sizeof(float);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_rows(tdx_moe_route_kernel<bf16>, route_grid(T), kThreads, smem, st, p)
                           : launch_rows(tdx_moe_route_kernel<float>, route_grid(T), kThreads, smem, st, p);
}

tdx_status tdx_moe_route_bwd(const void* logits, const int32_t* topk_idx, const float* dgates, void* dlogits, int T,
                             int E, int topk, tdx_dtype dtype, const tdx_route_opts* opts, void* stream) {
  const tdx_route_opts o = opts ? *opts : route_defaults();
  RouteParams p;
  const tdx_status s = route_params(T, E, topk, dtype, o, &p);
  if (s != TDX_OK) return s;
  if (logits == nullptr || topk_idx == nullptr || dgates == nullptr || dlogits == nullptr) return TDX_ERR_INVALID_ARG;
  const unsigned elt = static_cast<unsigned>(bytes_of(dtype));
  if (!aligned(logits, elt) || !aligned(dlogits, elt) || !aligned(topk_idx, 4) || !aligned(dgates, 4))
    return TDX_ERR_ALIGNMENT;
  if (T == 0) return TDX_OK;
  p.logits = logits;
  p.idx = const_cast<int32_t*>(topk_idx);
  p.dgates = dgates;
  p.dlogits = dlogits;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_rows(tdx_moe_route_bwd_kernel<bf16>, route_grid(T), kThreads, 0, st, p)
                           : launch_rows(tdx_moe_route_bwd_kernel<float>, route_grid(T), kThreads, 0, st, p);
}

}  // extern "C"
