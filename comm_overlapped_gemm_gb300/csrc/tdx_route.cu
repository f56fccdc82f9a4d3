// Routing of tokens to experts and its gradient (tdx_moe_route, tdx_moe_route_bwd).
#include <algorithm>

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
  int vector;        // rows may be read in the lanes' 8 or 16 bytes
  int group_lanes;   // lanes per group
};

// 1 / (1 + exp(-x)), each step rounded to fp32 (no contraction of exp's last product into the sum); the
// correctly rounded reciprocal is the correctly rounded quotient
__device__ __forceinline__ float sigmoid_rn(float x) { return __frcp_rn(__fadd_rn(1.0f, expf(-x))); }

// Order-preserving image of a float: larger key, larger integer; NaN comes last (1), 0 is left for
// "taken or not in a chosen group". -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
  const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return f != f ? 1u : o;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return o <= 1u ? NAN : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// The score of a group from its two largest keys
__device__ __forceinline__ uint32_t group_key(const RouteParams& p, uint32_t k1, uint32_t k2, bool two, float m) {
  if (p.group_top == 1) return k1;
  float a = from_ordered(k1), b = two ? from_ordered(k2) : 0.0f;
  if (!p.sigmoid && p.bias == nullptr) {
    a = expf(__fadd_rn(a, -m));
    if (two) b = expf(__fadd_rn(b, -m));
  }
  return ordered(__fadd_rn(a, b));
}

// Gate of the lane's chosen expert (lane j < k: the j-th) and the row's outputs. `v`: its score s where the
// scores are sigmoids, else its logit; m, sum: the row's softmax, used where gates are not renormalised.
__device__ __forceinline__ void finish_row(const RouteParams& p, int64_t t, int lane, int id, float v, float m, float sum,
                                           bool nan, int* hist) {
  const bool on = lane < p.k;
  float s, den = 1.0f;
  if (p.sigmoid) {
    s = on ? v : 0.0f;
    if (p.renorm) den = lanes_sum<16>(s);
  } else {
    // renormalised softmax is the softmax over the chosen logits, taken from their own maximum
    if (!on) v = -INFINITY;
    const float top = p.renorm ? lanes_max<16>(v) : m;
    s = top == -INFINITY ? 0.0f : expf(v - top);
    den = p.renorm ? lanes_sum<16>(s) : sum;
  }
  float g = s == 0.0f ? 0.0f : s / den * p.scale;
  if (nan) g = NAN;
  if (on) {
    p.idx[t * p.k + lane] = id;
    p.gates[t * p.k + lane] = g;
    if (p.counts != nullptr) atomicAdd(hist + id, 1);
  }
}

// Load the lane's V consecutive logits (columns lane * V on), -inf past the end; `vector`: in words of the
// lane's bytes, 16 at most.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* x, int lane, int E, bool vector, float (&v)[V]) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  const int c = lane * V;
  if (vector && c < E) {
    if constexpr (kBytes >= 16) {
      constexpr int N = kVec<T>;
#pragma unroll
      for (int i = 0; i < V; i += N) {
        float w[N];
        load_vec(x + c + i, w);
#pragma unroll
        for (int k = 0; k < N; ++k) v[i + k] = w[k];
      }
      return;
    } else if constexpr (V > 1) {
      constexpr int kWords = kBytes / 4;   // 1 or 2
      uint32_t w[kWords];
      if constexpr (kWords == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(x + c);
        w[0] = q.x;
        w[1] = q.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(x + c);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
        else v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = c + i < E ? to_float(x[c + i]) : -INFINITY;
}

// One warp per token, V consecutive experts per lane, everything in registers. A lane knows the two best
// of its keys (and finds further ones by another look at its V keys, which it seldom has to), so that
// each of the k rounds is a warp maximum, the lowest lane that holds it (the lowest index: lanes hold
// ascending experts), and that lane's step to its next key. Groups are aligned runs of lanes.
// Bound by issue slots: the ids have to be those of the definition, so that every sigmoid is an
// expf and a correctly rounded reciprocal.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, V <= 8 ? 4 : 2) tdx_moe_route_rows_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int hist[];   // [E], only where counts are wanted
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, c0 = lane * V;
  griddep_wait();
  if (p.counts != nullptr) {
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
  }
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = p.bias != nullptr && c0 + i < E ? p.bias[c0 + i] : 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  float x[V], next[V];
  if (t < p.T) load_logits<T, V>(static_cast<const T*>(p.logits) + t * p.ld, lane, E, p.vector, next);
  for (; t < p.T; t += step) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = next[i];
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    if (t + step < p.T) load_logits<T, V>(row + step * p.ld, lane, E, p.vector, next);
    bool nan = false;
    float m = -INFINITY, sum = 1.0f;
    uint32_t key[V];
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s = sigmoid_rn(x[i]);
        if (p.bias != nullptr) s = __fadd_rn(s, bias[i]);
        key[i] = ordered(s);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        m = fmaxf(m, x[i]);
        nan |= x[i] != x[i];
        key[i] = ordered(x[i]);
      }
      nan = __any_sync(kAll, nan);
      m = warp_max(m);
      if (!p.renorm || p.bias != nullptr) {
        float e[V];
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[i] = expf(__fadd_rn(x[i], -m));
          if (c0 + i < E) sum += e[i];
        }
        sum = warp_sum(sum);
        if (p.bias != nullptr) {
#pragma unroll
          for (int i = 0; i < V; ++i) key[i] = ordered(__fadd_rn(__fdiv_rn(e[i], sum), bias[i]));
        }
      }
    }
    // the lane's two best keys a >= b and their experts
    uint32_t a = 0, b = 0;
    int ai = 0, bi = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t k = c0 + i < E ? key[i] : 0u;
      const bool first = k > a, second = k > b;
      bi = first ? ai : second ? c0 + i : bi;
      b = max(b, min(a, k));
      ai = first ? c0 + i : ai;
      a = max(a, k);
    }
    if (p.n_group > 1) {
      // a group's run of lanes shares its two best keys; a group is chosen if fewer than topk_group come
      // before it, each lane of the run comparing a part of the groups
      const int run = p.group_lanes;
      uint32_t k1 = a, k2 = b;
      for (int o = 1; o < run; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, k1, o), o2 = __shfl_xor_sync(kAll, k2, o);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
      }
      const uint32_t mine = group_key(p, k1, k2, E > p.n_group, m);
      const int g = lane / run;
      int before = 0;
      for (int o = 0; o < p.n_group; o += run) {
        const int other = o + lane - g * run;
        const uint32_t k = __shfl_sync(kAll, mine, other * run);
        if (other < p.n_group && (k > mine || (k == mine && other < g))) ++before;
      }
      for (int o = 1; o < run; o <<= 1) before += __shfl_xor_sync(kAll, before, o);
      if (g >= p.n_group || before >= p.topk_group) a = b = 0;
    }
    int id = 0;
    uint32_t got = 0;   // lane j: the j-th expert and its key
    for (int j = 0; j < p.k; ++j) {
      const uint32_t top = __reduce_max_sync(kAll, a);
      const int src = __ffs(__ballot_sync(kAll, a == top)) - 1;
      const int e = __shfl_sync(kAll, ai, src);
      if (lane == j) {
        id = e;
        got = top;
      }
      if (lane == src) {
        a = b;
        ai = bi;
        b = 0;
        if (V > 2 && a == 0) {
          // both are taken: the best of those that come after the one just taken
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const uint32_t k = c0 + i < E ? key[i] : 0u;
            if ((k < top || (k == top && c0 + i > e)) && k > a) {
              a = k;
              ai = c0 + i;
            }
          }
        }
      }
    }
    float v = from_ordered(got);
    if (p.bias != nullptr && lane < p.k) {
      v = to_float(row[id]);
      if (p.sigmoid) v = sigmoid_rn(v);
    }
    finish_row(p, t, lane, id, v, m, sum, nan, hist);
  }
  if (p.counts != nullptr) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads)
      if (hist[e] > 0) atomicAdd(p.counts + e, hist[e]);
  }
}

// Groups that are no aligned runs of lanes: one warp per token with the row's scores and keys in shared
// memory, E floats each.
template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ float sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  float* score = sm + warp * 2 * E;
  uint32_t* key = reinterpret_cast<uint32_t*>(score + E);
  int* hist = reinterpret_cast<int*>(sm + kWarps * 2 * E);   // [E], only where counts are wanted
  griddep_launch_dependents();
  griddep_wait();
  if (p.counts != nullptr) {
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
  }
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
      uint32_t gk = 0;
      if (lane < p.n_group) {
        uint32_t k1 = 0, k2 = 0;
        for (int i = 0; i < per; ++i) {
          const uint32_t k = key[lane * per + i];
          k2 = max(k2, min(k1, k));
          k1 = max(k1, k);
        }
        gk = group_key(p, k1, k2, per > 1, m);
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
    finish_row(p, t, lane, mine, lane < p.k ? score[mine] : 0.0f, m, sum, nan, hist);
    __syncwarp();
  }
  if (p.counts != nullptr) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads)
      if (hist[e] > 0) atomicAdd(p.counts + e, hist[e]);
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

unsigned route_grid(int T, int blocks_per_sm) {
  const int blocks = (T + kWarps - 1) / kWarps;
  const int most = (sm_count() > 0 ? sm_count() : kRefSMs) * blocks_per_sm;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T, int V>
tdx_status launch_route_rows(RouteParams& p, cudaStream_t st) {
  constexpr int kBytes = std::min(16, V * static_cast<int>(sizeof(T)));
  p.vector = p.E % V == 0 && aligned(p.logits, kBytes) && (p.ld * static_cast<int64_t>(sizeof(T))) % kBytes == 0;
  p.group_lanes = p.E / p.n_group / V;
  return launch_rows(tdx_moe_route_rows_kernel<T, V>, route_grid(p.T, V <= 8 ? 4 : 2), kThreads,
                     p.counts != nullptr ? p.E * sizeof(int) : 0, st, p);
}

template <typename T>
tdx_status launch_route(RouteParams& p, cudaStream_t st) {
  const int V = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : 16;
  const int per = p.E / p.n_group;
  if (p.n_group > 1 && (per % V != 0 || ((per / V) & (per / V - 1)) != 0)) {
    const size_t smem = static_cast<size_t>(kWarps) * 2 * p.E * sizeof(float) + (p.counts != nullptr ? p.E * sizeof(int) : 0);
    return launch_rows(tdx_moe_route_kernel<T>, route_grid(p.T, 8), kThreads, smem, st, p);
  }
  switch (V) {
    case 1: return launch_route_rows<T, 1>(p, st);
    case 2: return launch_route_rows<T, 2>(p, st);
    case 4: return launch_route_rows<T, 4>(p, st);
    case 8: return launch_route_rows<T, 8>(p, st);
    default: return launch_route_rows<T, 16>(p, st);
  }
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_route<bf16>(p, st) : launch_route<float>(p, st);
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
  return dtype == TDX_BF16 ? launch_rows(tdx_moe_route_bwd_kernel<bf16>, route_grid(T, 8), kThreads, 0, st, p)
                           : launch_rows(tdx_moe_route_bwd_kernel<float>, route_grid(T, 8), kThreads, 0, st, p);
}

}  // extern "C"
