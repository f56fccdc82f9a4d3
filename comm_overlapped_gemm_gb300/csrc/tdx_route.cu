// Routing of tokens to experts and its gradient (tdx_moe_route, tdx_moe_route_bwd).
#include <algorithm>

#include "tdx_rows.cuh"

namespace tdx {
namespace {

constexpr int kWarps = 8;                // most warps of a block
constexpr int kThreads = kWarps * 32;
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
  int vector;        // the lanes' experts may be read in words of 8 or 16 bytes
  int group_shift;   // log2 of the lanes per group
  int per;           // experts per group
  int warp_floats;   // shared memory of a warp
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

// The score of a group from its two largest keys (`two`: it has two; softmax without a bias adds exp(x - m))
__device__ __forceinline__ uint32_t group_key(const RouteParams& p, float k1, float k2, bool two, float m) {
  if (p.group_top == 1) return ordered(k1);
  if (!p.sigmoid && p.bias == nullptr) {
    k1 = expf(__fadd_rn(k1, -m));
    k2 = expf(__fadd_rn(k2, -m));
  }
  return ordered(__fadd_rn(k1, two ? k2 : 0.0f));
}

// The outputs of a row held by L lanes, R chosen experts a lane: place sub + r * L of the choice in slot r.
// v: the score s where scores are sigmoids, else the logit; m, sum: the row's softmax, used where gates are
// not renormalised. The approximate exponential and quotient leave a gate within 2^-22 * (4 + |v - m|) of its
// value.
template <int L, int R>
__device__ __forceinline__ void finish_row(const RouteParams& p, int64_t t, int sub, bool write, const int (&id)[R],
                                           float (&v)[R], float m, float sum, bool nan, int* hist) {
  constexpr int kReach = L < 16 ? L : 16;   // lanes that can hold one of 16 places
  float den = sum;
  if (!p.sigmoid) {
    // renormalised softmax is the softmax over the chosen logits, taken from their own maximum
    float top = m;
    if (p.renorm) {
      top = -INFINITY;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (sub + r * L < p.k) top = fmaxf(top, v[r]);
      top = lanes_max<kReach>(top);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = top == -INFINITY ? 0.0f : __expf(v[r] - top);
    if (top == -INFINITY) den = 0.0f;
  }
  if (p.renorm) {
    den = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (sub + r * L < p.k) den += v[r];
    den = lanes_sum<kReach>(den);
  } else if (p.sigmoid) {
    den = 1.0f;
  }
  if (m == INFINITY) den = NAN;   // exp(inf - inf) stands in every score of the row
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = sub + r * L;
    if (write && j < p.k) {
      p.idx[t * p.k + j] = id[r];
      // the approximate quotient, where the sum is no subnormal
      const float q = den < 1e-37f ? v[r] / den : __fdividef(v[r], den);
      p.gates[t * p.k + j] = nan ? NAN : den == 0.0f ? 0.0f : q * p.scale;
      if (p.counts != nullptr) atomicAdd(hist + id[r], 1);
    }
  }
}

// Load V logits of a row held by L lanes, `pad` past the end. `vector`: the lane's V consecutive ones (columns c
// on, if it holds any) in words of 16 bytes at most; else columns lane, lane + L, ..., so that odd row
// lengths and addresses are read in whole lines too.
template <typename T, int L, int V>
__device__ __forceinline__ void load_logits(const T* x, int lane, int c, bool holds, int E, bool vector, float pad,
                                            float (&v)[V]) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  if (vector && holds) {
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
  for (int i = 0; i < V; ++i) v[i] = !vector && lane + i * L < E ? to_float(x[lane + i * L]) : pad;
}

// One row by one warp, from the definition's own steps: the row's scores and keys in shared memory, 2 E
// floats. The rows that tdx_moe_route_rows_kernel cannot settle, and groups that its lanes cannot hold (five of
// 100 experts), come here.
template <typename T>
__device__ __noinline__ void route_row(const RouteParams& p, int64_t t, float* score, int* hist) {
  const int lane = threadIdx.x & 31;
  const int E = p.E;
  uint32_t* key = reinterpret_cast<uint32_t*>(score + E);
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
    for (int e = lane; e < E; e += 32) sum += expf(__fadd_rn(to_float(x[e]), -m));
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
      // NaN keys (1) come last: the two largest are NaN only where nothing else is there
      uint32_t k1 = 0, k2 = 0;
      for (int i = 0; i < per; ++i) {
        const uint32_t k = key[lane * per + i];
        k2 = max(k2, min(k1, k));
        k1 = max(k1, k);
      }
      gk = group_key(p, from_ordered(k1), from_ordered(k2), per > 1, m);
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
  const int id[1] = {mine};
  float v[1] = {lane < p.k ? score[mine] : 0.0f};
  finish_row<32, 1>(p, t, lane, true, id, v, m, sum, nan, hist);
  __syncwarp();
}

// Shared memory of both kernels: p.warp_floats per warp (2 E for route_row, 32 V for the other's rows where
// they are not read in vectors), then E counters where counts are wanted
__device__ __forceinline__ int* clear_hist(const RouteParams& p, float* sm) {
  int* hist = reinterpret_cast<int*>(sm + (blockDim.x >> 5) * p.warp_floats);
  if (p.counts != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  return hist;
}
__device__ __forceinline__ void add_hist(const RouteParams& p, const int* hist) {
  if (p.counts == nullptr) return;
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x)
    if (hist[e] > 0) atomicAdd(p.counts + e, hist[e]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) tdx_moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ float sm[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  int* hist = clear_hist(p, sm);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * warps)
    route_row<T>(p, t, sm + warp * p.warp_floats, hist);
  add_hist(p, hist);
}

// V consecutive values of a 16-byte aligned place in shared memory
template <int V>
__device__ __forceinline__ void read_lane(const float* from, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(from + i);
    v[i] = q.x;
    v[i + 1] = q.y;
    v[i + 2] = q.z;
    v[i + 3] = q.w;
  }
}

// Exchange so that a >= b
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t lo = min(a, b);
  a = max(a, b);
  b = lo;
}
// Sorting networks, descending: 5 exchanges for four words, 19 for eight; of sixteen the best eight, from two
// sorted halves
__device__ __forceinline__ void sort_words(uint32_t (&w)[4]) {
  order(w[0], w[1]), order(w[2], w[3]), order(w[0], w[2]), order(w[1], w[3]), order(w[1], w[2]);
}
__device__ __forceinline__ void sort_words(uint32_t (&w)[8]) {
  order(w[0], w[1]), order(w[2], w[3]), order(w[4], w[5]), order(w[6], w[7]);
  order(w[0], w[2]), order(w[1], w[3]), order(w[4], w[6]), order(w[5], w[7]);
  order(w[1], w[2]), order(w[5], w[6]), order(w[0], w[4]), order(w[3], w[7]);
  order(w[1], w[5]), order(w[2], w[6]), order(w[1], w[4]), order(w[3], w[6]);
  order(w[2], w[4]), order(w[3], w[5]), order(w[3], w[4]);
}
__device__ __forceinline__ void best_words(const uint32_t (&w)[4], uint32_t (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = w[i];
  sort_words(s);
}
__device__ __forceinline__ void best_words(const uint32_t (&w)[8], uint32_t (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = w[i];
  sort_words(s);
}
__device__ __forceinline__ void best_words(const uint32_t (&w)[16], uint32_t (&s)[8]) {
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = w[i];
    h[i] = w[8 + i];
  }
  sort_words(s);
  sort_words(h);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = max(s[i], h[7 - i]);
  order(s[0], s[4]), order(s[1], s[5]), order(s[2], s[6]), order(s[3], s[7]);
  order(s[0], s[2]), order(s[1], s[3]), order(s[4], s[6]), order(s[5], s[7]);
  order(s[0], s[1]), order(s[2], s[3]), order(s[4], s[5]), order(s[6], s[7]);
}

// Largest of L lanes' words
template <int L>
__device__ __forceinline__ uint32_t lanes_top(uint32_t w) {
  if constexpr (L == 32) {
    w = __reduce_max_sync(kAll, w);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(kAll, w, o));
  }
  return w;
}

// L lanes per token, 32 / L tokens per warp, V consecutive experts per lane in registers; K >= topk.
//
// The choice is K + 1 maxima over the token's lanes of 32-bit words that hold a key's leading 32 - B bits
// and below them the expert, B bits, counted backwards: all words differ, equal keys come in the order of
// their experts, and a maximum names its expert, so that a round is a maximum and one lane's step to
// the next word of its sorted list (the best eight of sixteen: a lane that runs out of them sends the row to
// route_row). What the words leave open are keys that agree in their leading bits: where neighbours do, the
// exact keys of the choice and of the first word left out put them in order. Rows where the first two
// left out agree with the last one taken go to route_row, as do rows with a NaN. bf16 logits that are
// compared as such fit into the leading bits.
// A group is a run of 2^n lanes (all of them where there are no groups); entries past its end hold -inf and
// the word 0, which says that there is nothing.
//
// Bound by issue slots, not by HBM: 32768 tokens, softmax, 8 of 64 experts 7.5 us (139 warp instructions a
// token; HBM 1.6 us), sigmoid with bias, 8 of 256 in 4 of 8 groups 27.4 us (701, some 177 of them for scores: ids
// have to be those of the definition, so that every sigmoid is an expf and a correctly rounded
// reciprocal; 150 for the groups, 150 for the maxima, 42 for the sorted lists; HBM 5.3 us), 2.85 of 4
// instructions a cycle. Registers decide how much of that is reached (the bounds below cost the bf16 instances and those
// of 16 places spills of up to 36 bytes; none in fp32 for up to 8 places): 64-bit token numbers 29.6 us, biases in
// registers 27.8; with 16 lanes of 16 experts for 256 32.3, at half the blocks; three / five blocks per SM 30.2 /
// 32.2; the maxima in a loop 33.0. 512 experts, sigmoid with bias, topk 16: 50.9 us at three blocks, 54.5 at two.
template <typename T, int L, int V, int K, bool kVector>
__global__ void __launch_bounds__(kThreads, V <= 8 ? 4 : 3)
    tdx_moe_route_rows_kernel(const __grid_constant__ RouteParams p) {
  constexpr int kTokens = 32 / L;
  constexpr int kLog = (V == 4 ? 2 : V == 8 ? 3 : 4) + (L == 8 ? 3 : L == 16 ? 4 : 5);
  constexpr uint32_t kLow = (1u << kLog) - 1u;
  constexpr int S = V < 8 ? V : 8;                // words of the sorted list
  constexpr int R = K > L ? K / L : 1;            // places of the choice per lane
  extern __shared__ float sm[];
  griddep_launch_dependents();
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % L, first = lane - sub;   // lane within the token's, and the token's first lane
  const int E = p.E, per = p.per;
  const int run = 1 << p.group_shift, group = sub >> p.group_shift;   // lanes per group, and the lane's
  const int within = (sub & (run - 1)) * V;                             // its first expert, counted in the group
  const int c0 = group * per + within;
  const bool holds = group < p.n_group && within < per;
  griddep_wait();
  int* hist = clear_hist(p, sm);
  float* const stage = sm + warp * p.warp_floats;
  const bool biased = p.bias != nullptr;
  // the biases in the lanes' order, -inf past the end of a group. Logits there are 0 where scores are sigmoids:
  // the reciprocal of 1 + exp(inf) takes a slow path in the whole warp (384 experts, sigmoid: 41 against 56 us)
  __shared__ __align__(16) float bias_of[L * V];
  const float pad = p.sigmoid ? 0.0f : -INFINITY;
  if (biased || p.sigmoid) {
    if (threadIdx.x < L) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        bias_of[sub * V + i] = !holds || within + i >= per ? -INFINITY : biased ? p.bias[c0 + i] : 0.0f;
    }
    __syncthreads();
  }
  const bool exact_words = sizeof(T) == 2 && !p.sigmoid && !biased;
  // T and a step are below 2^31 each: token numbers fit 32 bits
  const uint32_t T_all = static_cast<uint32_t>(p.T), step = gridDim.x * warps * kTokens;
  uint32_t t = (blockIdx.x * warps + warp) * kTokens + lane / L;
  float next[V];
#pragma unroll
  for (int i = 0; i < V; ++i) next[i] = pad;
  if (t < T_all) load_logits<T, L, V>(static_cast<const T*>(p.logits) + t * p.ld, sub, c0, holds, E, kVector, pad, next);
  for (; t - lane / L < T_all; t += step) {
    const bool live = t < T_all;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    float f[V];   // logits, then keys
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = next[i];
    if constexpr (!kVector) {
      // from every L-th column to consecutive ones
      float* const token = stage + first * V;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) token[sub + i * L] = f[i];
      __syncwarp();
      if (p.n_group == 1) {
        read_lane(token + sub * V, f);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = holds && within + i < per ? token[c0 + i] : pad;
      }
    }
    if (t + step < T_all) load_logits<T, L, V>(row + step * p.ld, sub, c0, holds, E, kVector, pad, next);
    float m = -INFINITY, sum = 1.0f;
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = sigmoid_rn(f[i]);
      float bias[V];
      read_lane(bias_of + sub * V, bias);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __fadd_rn(f[i], bias[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, f[i]);
      m = lanes_max<L>(m);
      if (biased) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          f[i] = expf(__fadd_rn(f[i], -m));
          sum += f[i];
        }
        sum = lanes_sum<L>(sum);
        float bias[V];
        read_lane(bias_of + sub * V, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __fadd_rn(__fdiv_rn(f[i], sum), bias[i]);
      } else if (!p.renorm) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += __expf(f[i] - m);
        sum = lanes_sum<L>(sum);
      }
    }
    // a NaN among the keys (or +inf and -inf) shows in their sum
    float any = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) any += f[i];
    const unsigned odd = __ballot_sync(kAll, any != any);
    bool slow = L == 32 ? odd != 0 : ((odd >> first) & ((1u << (L & 31)) - 1u)) != 0;
    bool kept = holds;
    if (p.n_group > 1) {
      // a group's run of lanes shares its two best keys; a group is chosen if fewer than topk_group come
      // before it, each lane of the run comparing a part of the groups
      float k1 = -INFINITY, k2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        k2 = fmaxf(k2, fminf(k1, f[i]));
        k1 = fmaxf(k1, f[i]);
      }
      for (int o = 1; o < run; o <<= 1) {
        const float o1 = __shfl_xor_sync(kAll, k1, o), o2 = __shfl_xor_sync(kAll, k2, o);
        k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
        k1 = fmaxf(k1, o1);
      }
      const uint32_t mine = group_key(p, k1, k2, per > 1, m);
      int before = 0;
      for (int o = sub & (run - 1); o - (sub & (run - 1)) < p.n_group; o += run) {
        const uint32_t k = __shfl_sync(kAll, mine, first + (o << p.group_shift));
        if (o < p.n_group && (k > mine || (k == mine && o < group))) ++before;
      }
      for (int o = 1; o < run; o <<= 1) before += __shfl_xor_sync(kAll, before, o);
      kept &= before < p.topk_group;
    }
    uint32_t best[S];
    {
      uint32_t w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t u = __float_as_uint(__fadd_rn(f[i], 0.0f));   // -0 to +0
        const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
        w[i] = (k & ~kLow) | (kLow - static_cast<uint32_t>(c0 + i));
      }
      if constexpr (!kVector) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (within + i >= per) w[i] = 0;
      }
      best_words(w, best);
    }
    if (!kept) {
#pragma unroll
      for (int i = 0; i < S; ++i) best[i] = 0;
    }
    uint32_t got[R], top = 0;   // the words of the lane's places
#pragma unroll
    for (int r = 0; r < R; ++r) got[r] = 0;
    bool dry = false;
#pragma unroll
    for (int j = 0; j <= K; ++j) {
      top = lanes_top<L>(best[0]);
      if (j < K && sub == j % L) got[j < K ? j / L : 0] = top;
      if (best[0] == top) {
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) best[i] = best[i + 1];
        best[S - 1] = 0;
        if (V > S) dry |= best[0] == 0 && top != 0;
      }
    }
    if (V > S) slow |= __any_sync(kAll, dry);
    // the word of place j, K at most
    auto word = [&](int j) {
      uint32_t w = __shfl_sync(kAll, got[0], first + j % L);
      if (R > 1) {
        const uint32_t w1 = __shfl_sync(kAll, got[R - 1], first + j % L);
        if (j >= L) w = w1;
      }
      return j == K ? top : w;
    };
    const uint32_t left = word(p.k);   // the first word left out
    // what the gates are made of: the scores, or the logits
    auto gate_score = [&](int e) {
      const float x = to_float(row[e]);
      if (!p.sigmoid) return x;
      return x < -80.0f ? sigmoid_rn(x) : __fdividef(1.0f, 1.0f + __expf(-x));
    };
    int id[R];
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      id[r] = static_cast<int>(kLow - (got[r] & kLow));
      v[r] = 0.0f;
      if (live && !slow && sub + r * L < p.k) v[r] = gate_score(id[r]);
    }
    if (!exact_words) {
      bool open = false;   // places whose next one agrees in the leading bits
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int j = sub + r * L;
        uint32_t after = __shfl_sync(kAll, got[r], first + (sub + 1) % L);
        if (R > 1 && r + 1 < R) {
          const uint32_t over = __shfl_sync(kAll, got[R - 1], first);
          if (sub == L - 1) after = over;
        }
        if (j == p.k - 1) after = left;
        open |= live && j < p.k && after != 0 && (got[r] ^ after) <= kLow;
      }
      if (__any_sync(kAll, open)) {
        // Put the places and the first word left out in order by their exact keys. Should the second
        // word left out agree with it and with the last place, there may be more of them: route_row.
        const uint32_t next_top = lanes_top<L>(best[0]);
        const uint32_t second = p.k == K ? next_top : word(p.k + 1);
        const uint32_t end = word(p.k - 1);
        slow |= second != 0 && (end ^ left) <= kLow && (left ^ second) <= kLow;
        auto exact_key = [&](int e) {
          const float x = to_float(row[e]);
          float k = x;
          if (p.sigmoid) k = sigmoid_rn(x);
          else if (biased) k = __fdiv_rn(expf(__fadd_rn(x, -m)), sum);
          return ordered(biased ? __fadd_rn(k, p.bias[e]) : k);
        };
        const bool settle = live && !slow;
        uint32_t exact[R], exact_left = 0;
        const int id_left = static_cast<int>(kLow - (left & kLow));
        float v_left = 0.0f;
        if (settle && left != 0) {
          exact_left = exact_key(id_left);
          v_left = gate_score(id_left);
        }
        int place[R], nid[R], place_left = 0;
        float nv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          exact[r] = settle && sub + r * L < p.k ? exact_key(id[r]) : 0u;
          place[r] = exact_left > exact[r] || (exact_left == exact[r] && id_left < id[r]) ? 1 : 0;
          nid[r] = id[r];
          nv[r] = v[r];
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
          for (int j = 0; j < L && j + q * L < p.k; ++j) {
            const uint32_t o = __shfl_sync(kAll, exact[q], first + j);
            const int oid = __shfl_sync(kAll, id[q], first + j);
#pragma unroll
            for (int r = 0; r < R; ++r) place[r] += o > exact[r] || (o == exact[r] && oid < id[r]) ? 1 : 0;
            place_left += o > exact_left || (o == exact_left && oid < id_left) ? 1 : 0;
          }
#pragma unroll
        for (int q = 0; q < R; ++q)
          for (int j = 0; j < L && j + q * L < p.k; ++j) {
            const int at = __shfl_sync(kAll, place[q], first + j);
            const int oid = __shfl_sync(kAll, id[q], first + j);
            const float ov = __shfl_sync(kAll, v[q], first + j);
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (at == sub + r * L) {
                nid[r] = oid;
                nv[r] = ov;
              }
          }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool take = place_left == sub + r * L;
          id[r] = take ? id_left : nid[r];
          v[r] = take ? v_left : nv[r];
        }
      }
    }
    finish_row<L, R>(p, t, sub, live && !slow, id, v, m, sum, false, hist);
    for (unsigned rest = __ballot_sync(kAll, live && slow && sub == 0); rest != 0; rest &= rest - 1)
      route_row<T>(p, __shfl_sync(kAll, t, __ffs(rest) - 1), stage, hist);
  }
  add_hist(p, hist);
}

// Store V values of a row of E where load_logits finds them
template <typename T, int L, int V>
__device__ __forceinline__ void store_logits(T* x, int lane, int E, bool vector, const float (&v)[V]) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  const int c = lane * V;
  if (vector) {
    if (c >= E) return;
    if constexpr (kBytes >= 16) {
      constexpr int N = kVec<T>;
#pragma unroll
      for (int i = 0; i < V; i += N) {
        float w[N];
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = v[i + k];
        store_vec(x + c + i, w);
      }
    } else {
      static_assert(V == 4 && sizeof(T) == 2);
      store_vec(x + c, v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane + i * L < E) x[lane + i * L] = static_cast<T>(v[i]);
}

// L lanes per token, V consecutive experts per lane as forwards; slot r of a lane is the choice's place
// sub + r * L. What a chosen expert's logit receives is scattered into a row of shared memory and read
// back by the lanes that hold the row, so that dlogits are written in whole lines and softmax over the
// whole row needs no look at the chosen logits. Choices of the same expert add up in the order of their places.
// 4 E (softmax over the row: 8 E) bytes and 8 topk bytes a token: 32768 tokens, softmax over 64 experts 4.9 us
// (HBM 2.8), 128 experts 9.0 us (5.3), 500 experts 30 us (20; in lanes of consecutive experts, read one by one,
// 89), renormalised sigmoid over 256 12.9 us (5.5), there bound by the latency of a warp's steps for its one
// token: eight blocks per SM 13.0 us, four 16.7 (for 8 lanes a token more than the compiler's choice is slower:
// 6.3 against 4.9).
template <typename T, int L, int V>
__global__ void __launch_bounds__(kThreads, L == 32 ? (V <= 8 ? 8 : 4) : L == 16 ? 6 : 1)
    tdx_moe_route_bwd_kernel(const __grid_constant__ RouteParams p) {
  constexpr int kTokens = 32 / L;
  constexpr int R = kMoeMaxTopk > L ? kMoeMaxTopk / L : 1;
  __shared__ __align__(16) float rows[kWarps * 32 * V];
  griddep_launch_dependents();
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % L, first = lane - sub;
  float* const row = rows + (warp * 32 + first) * V;
  const int E = p.E;
  const bool dense = !p.sigmoid && !p.renorm;
  griddep_wait();
  const uint32_t T_all = static_cast<uint32_t>(p.T), step = gridDim.x * warps * kTokens;   // each below 2^31
  for (uint32_t t = (blockIdx.x * warps + warp) * kTokens + lane / L; t - lane / L < T_all; t += step) {
    const bool live = t < T_all;
    const int64_t at = static_cast<int64_t>(t) * p.k;
    const T* x = static_cast<const T*>(p.logits) + t * p.ld;
    float e[V];   // softmax over the row: logits, then exponentials
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = -INFINITY;
    if (dense && live) load_logits<T, L, V>(x, sub, sub * V, sub * V < E, E, p.vector, -INFINITY, e);
    int id[R];
    float d[R], v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = sub + r * L;
      id[r] = -1;
      d[r] = 0.0f;
      v[r] = -INFINITY;
      if (live && j < p.k) {
        id[r] = p.idx[at + j];
        if (id[r] < 0 || id[r] >= E) id[r] = -1;
      }
      if (id[r] >= 0) {
        d[r] = p.dgates[at + j] * p.scale;
        if (!dense) v[r] = to_float(x[id[r]]);
      }
    }
    // d: what the chosen score receives, then (but for softmax over the row) what its logit does
    float m = -INFINITY, inv = 0.0f;
    if (p.sigmoid) {
      float s[R], S = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = id[r] >= 0 ? sigmoid_rn(v[r]) : 0.0f;
        if (p.renorm) s[r] *= 0x1p40f;   // so that 1 / S is finite however small the scores
        S += s[r];
      }
      if (p.renorm) {
        // through the gates s / S, which are of size one
        float dot = 0.0f;
        S = lanes_sum<L>(S);
        const float one_over = S == 0.0f ? 0.0f : __frcp_rn(S);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r] *= one_over;
          dot += d[r] * s[r];
        }
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int r = 0; r < R; ++r) d[r] -= dot;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) d[r] = id[r] >= 0 ? d[r] * s[r] * sigmoid_rn(-v[r]) : 0.0f;
    } else if (p.renorm) {
#pragma unroll
      for (int r = 0; r < R; ++r) m = fmaxf(m, v[r]);
      m = lanes_max<L>(m);
      float S = 0.0f, dot = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v[r] = id[r] >= 0 && !(m == -INFINITY && v[r] == m) ? expf(v[r] - m) : 0.0f;
        S += v[r];
      }
      S = lanes_sum<L>(S);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v[r] = S == 0.0f ? 0.0f : v[r] / S;
        dot += d[r] * v[r];
      }
      dot = lanes_sum<L>(dot);
#pragma unroll
      for (int r = 0; r < R; ++r) d[r] = v[r] * (d[r] - dot);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, e[i]);
      m = lanes_max<L>(m);
      float S = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        e[i] = m == -INFINITY && e[i] == m ? 0.0f : __expf(e[i] - m);
        S += e[i];
      }
      S = lanes_sum<L>(S);
      inv = S == 0.0f ? 0.0f : 1.0f / S;
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(row + sub * V + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    // places that name one expert: the tag left there is another place's
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (id[r] >= 0) row[id[r]] = __int_as_float(sub + r * L);
    __syncwarp();
    bool twice = false;
#pragma unroll
    for (int r = 0; r < R; ++r) twice |= id[r] >= 0 && __float_as_int(row[id[r]]) != sub + r * L;
    if (__any_sync(kAll, twice)) {
      float add[R];
      bool lead[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        add[r] = d[r];
        lead[r] = true;
      }
#pragma unroll
      for (int q = 0; q < R; ++q)
        for (int j = 0; j < L; ++j) {
          const int oid = __shfl_sync(kAll, id[q], first + j);
          const float od = __shfl_sync(kAll, d[q], first + j);
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (oid == id[r] && oid >= 0) {
              if (j + q * L < sub + r * L) lead[r] = false;
              if (j + q * L > sub + r * L) add[r] += od;
            }
        }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        d[r] = add[r];
        if (!lead[r]) id[r] = -1;
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (id[r] >= 0) row[id[r]] = d[r];
    __syncwarp();
    float a[V];
    if (p.vector) {
      read_lane(row + sub * V, a);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = row[sub + i * L];
    }
    if (dense) {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        e[i] *= inv;
        dot = fmaf(a[i], e[i], dot);
      }
      dot = lanes_sum<L>(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = e[i] * (a[i] - dot);
    }
    if (live) store_logits<T, L, V>(static_cast<T*>(p.dlogits) + t * p.ld, sub, E, p.vector, a);
    __syncwarp();   // before the row is cleared
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

// Blocks for T tokens, `each` of them per warp. Few warps spread over the SMs, a block of one on each, before they
// share one: 128 tokens of 256 experts in groups 3.3 us, in blocks of eight warps 3.6.
struct RouteShape {
  unsigned grid, block;
};
RouteShape route_shape(int64_t T, int each, int blocks_per_sm) {
  const int64_t warps = (T + each - 1) / each, sms = sm_count() > 0 ? sm_count() : kRefSMs;
  const int64_t per_block = std::min<int64_t>(kWarps, (warps + sms - 1) / sms);
  const int64_t blocks = (warps + per_block - 1) / per_block;
  return {static_cast<unsigned>(std::min(blocks, sms * blocks_per_sm)), static_cast<unsigned>(per_block) * 32};
}

// log2 of the lanes that a group takes at V experts a lane
int group_lanes_log(const RouteParams& p, int V) {
  int log = 0;
  while ((V << log) < p.per) ++log;
  return log;
}

// Shared memory of a launch with at least `floats` per warp
size_t route_smem(RouteParams* p, unsigned block, int floats) {
  p->warp_floats = (std::max(2 * p->E, floats) + 3) & ~3;
  return static_cast<size_t>(block / 32) * p->warp_floats * sizeof(float) + (p->counts != nullptr ? p->E * sizeof(int) : 0);
}

template <typename T, int L, int V, int K>
tdx_status launch_route_k(RouteParams& p, cudaStream_t st) {
  constexpr int kBytes = std::min(16, V * static_cast<int>(sizeof(T)));
  p.vector = p.per % V == 0 && aligned(p.logits, kBytes) && (p.ld * static_cast<int64_t>(sizeof(T))) % kBytes == 0;
  p.group_shift = group_lanes_log(p, V);
  if (p.n_group == 1) p.group_shift = L == 8 ? 3 : L == 16 ? 4 : 5;
  const RouteShape at = route_shape(p.T, 32 / L, V <= 8 ? 4 : 3);
  const size_t smem = route_smem(&p, at.block, p.vector ? 0 : 32 * V);
  return p.vector ? launch_rows(tdx_moe_route_rows_kernel<T, L, V, K, true>, at.grid, at.block, smem, st, p)
                  : launch_rows(tdx_moe_route_rows_kernel<T, L, V, K, false>, at.grid, at.block, smem, st, p);
}

template <typename T, int L, int V>
tdx_status launch_route_v(RouteParams& p, cudaStream_t st) {
  if (p.k <= 4) return launch_route_k<T, L, V, 4>(p, st);
  return p.k <= 8 ? launch_route_k<T, L, V, 8>(p, st) : launch_route_k<T, L, V, 16>(p, st);
}

// Whether L lanes hold the row, V experts each and a power of two of lanes per group
bool route_fits(const RouteParams& p, int L, int V) {
  return p.n_group == 1 ? p.E <= L * V : p.n_group << group_lanes_log(p, V) <= L;
}

// The smallest layout that holds the row: the maxima, sums and addresses are the same instructions for four
// tokens of a warp as for one (32768 tokens, 64 experts 7.5 us, a warp per token 13.4). Up to a warp per
// scheduler a whole warp's maximum in one instruction is sooner there than shuffles: 1 token 2.0 / 2.4 us, 600
// tokens 2.4 / 2.5, but 1024 3.4 / 2.5.
template <typename T>
tdx_status launch_route(RouteParams& p, cudaStream_t st) {
  p.per = p.E / p.n_group;
  if (p.T <= 4 * sm_count() && route_fits(p, 32, 8)) return launch_route_v<T, 32, 8>(p, st);
  if (route_fits(p, 8, 4)) return launch_route_v<T, 8, 4>(p, st);
  if (route_fits(p, 8, 8)) return launch_route_v<T, 8, 8>(p, st);
  if (route_fits(p, 16, 8)) return launch_route_v<T, 16, 8>(p, st);
  if (route_fits(p, 32, 8)) return launch_route_v<T, 32, 8>(p, st);
  if (route_fits(p, 32, 16)) return launch_route_v<T, 32, 16>(p, st);
  const RouteShape at = route_shape(p.T, 1, 8);
  const size_t smem = route_smem(&p, at.block, 0);
  return launch_rows(tdx_moe_route_kernel<T>, at.grid, at.block, smem, st, p);
}

template <typename T, int L, int V>
tdx_status launch_route_bwd_v(RouteParams& p, cudaStream_t st) {
  constexpr int kBytes = std::min(16, V * static_cast<int>(sizeof(T)));
  p.vector = p.E % V == 0 && aligned(p.logits, kBytes) && aligned(p.dlogits, kBytes) &&
             (p.ld * static_cast<int64_t>(sizeof(T))) % kBytes == 0;
  const RouteShape at = route_shape(p.T, 32 / L, 8);
  return launch_rows(tdx_moe_route_bwd_kernel<T, L, V>, at.grid, at.block, 0, st, p);
}

template <typename T>
tdx_status launch_route_bwd(RouteParams& p, cudaStream_t st) {
  if (p.E <= 32) return launch_route_bwd_v<T, 8, 4>(p, st);
  if (p.E <= 64) return launch_route_bwd_v<T, 8, 8>(p, st);
  if (p.E <= 128) return launch_route_bwd_v<T, 16, 8>(p, st);
  return p.E <= 256 ? launch_route_bwd_v<T, 32, 8>(p, st) : launch_route_bwd_v<T, 32, 16>(p, st);
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
  return dtype == TDX_BF16 ? launch_route_bwd<bf16>(p, st) : launch_route_bwd<float>(p, st);
}

}  // extern "C"
