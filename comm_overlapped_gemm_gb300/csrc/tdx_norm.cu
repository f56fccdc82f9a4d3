// Root-mean-square norm of x + residual and its gradient (tdx_rmsnorm, tdx_rmsnorm_bwd).
#include <algorithm>

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
// Threads of the kernels for long rows. 256 / 512 / 1024: forwards 4000 x 32768 bf16 225 / 186 / 200 us, 4000 x
// 20000 to e4m3 117 / 101 / 189; backwards 5000 x 10000 fp32 882 / 262 / 185, 4000 x 32768 bf16 648 / 397 / 284
constexpr int kLong = 512, kLongBwd = 1024;
constexpr int kBwdParts = 304;   // most row groups whose partial weight gradients are added at the end, long rows

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
  float eps, inv_scale, inv_h;   // inv_h = 1 / H
};

// Sum (or largest magnitude) over the block; every thread gets it.
template <bool MAX, int kBlock>
__device__ float block_reduce(float v, float* sm) {
  v = MAX ? lanes_max_abs<32>(v) : warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = sm[0];
#pragma unroll
  for (int i = 1; i < kBlock / 32; ++i) r = MAX ? max_abs(r, sm[i]) : r + sm[i];
  return r;
}

// The e4m3 scale of a row, m / 448 from m = max|y| (1 where that is 0 or no number), and the factors that take y to
// codes, y * up * inv. The numbers of rows near the ends of fp32's range are first multiplied by a power of two, so
// that 448 / m stays finite and is no subnormal. Every thread computes this: the approximate quotient (2 ulp, for a
// divisor up to 2^126) keeps it short.
__device__ __forceinline__ float row_scale(float m, float* inv, float* up) {
  const float s = m * (1.0f / 448.0f);
  *inv = 1.0f;
  if (!(s > 0.0f)) return 1.0f;
  if (m < 1e-30f) *up = 0x1p100f;
  if (m > 1e30f) *up = 0x1p-100f;
  *inv = __fdividef(448.0f, m * *up);
  return s;
}

// A row held in registers, E of its elements per thread in 16-byte vectors: one read of x and residual,
// one reduction for the sum of squares and (kScaled: row scales are wanted) max|h * weight|, whose
// product with rstd is max|y|, one write of h and y.
// kLanes 8, 16, 32: that many lanes of a warp per row (short rows; the reduction is shuffles alone); 0: a
// block per row, whose reduction takes one barrier.
// Bound by HBM: 32768 x 7168 bf16 with the residual 268 us (7.0 TB/s, a plain copy's rate 281), 1000000 x
// 128 148 us (6.9 TB/s; with a warp per row of 128, half of its lanes idle, 200 us). 1024 x 7168 to e4m3 with
// row scales takes 10.4 us of 7.7: the launch's ramp and tail (a plain addition over as many bytes takes 9.0).
// Rows through a ring of cp.async stages in shared memory, as the gradient takes them, came out slower
// here (311 us): the many independent blocks keep more loads in flight than one block per SM does
// between two sums.
// Registers: 64 a thread for 32 bf16 elements, so that four blocks of 224 threads share an SM instead of three
// (1024 x 7168 to e4m3 11.2 / 11.7 us at the time; five, at 48 registers, spill: 13.8). y's address is taken after
// the reduction: before it, the row scales' instance spills (32768 x 7168 to e4m3 305 us, without 235).
// kSum: there may be a residual. Without one the row waits for its sum as it was read, not in fp32: 6960 x 7184
// bf16 93% of a copy's rate (in fp32, before the sums were taken two at a time and rsqrtf, 78%; now bound by issue
// slots, as are the codes there, 74%). Rows just above 1024 columns leave half of two warps idle: 48076 x 1040 bf16
// 61%.
template <typename T, typename O, int E, int kLanes, bool kSum, bool kScaled>
__global__ void __launch_bounds__(kLanes ? kThreads : 16384 / E, !kLanes && sizeof(T) == 2 && E == 32 ? 2 : 1)
    tdx_rmsnorm_rows_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = kVec<T>;
  constexpr int V = E / N;
  __shared__ float2 sm[32];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int width = kLanes ? kLanes : blockDim.x;                                       // threads of a row
  const int at = (kLanes ? threadIdx.x % (kLanes ? kLanes : 1) : threadIdx.x) * N;      // the thread's first column
  const int64_t t = kLanes ? static_cast<int64_t>(blockIdx.x) * (kThreads / (kLanes ? kLanes : 1)) +
                                 threadIdx.x / (kLanes ? kLanes : 1)
                           : blockIdx.x;
  const int H = t < p.T ? p.H : 0;   // a row past the end takes part in the shuffles only
  const T* x = static_cast<const T*>(p.x) + t * p.ld_x + at;
  const T* r = static_cast<const T*>(p.residual) + t * p.ld_r + at;
  const T* w = static_cast<const T*>(p.weight) + at;
  T* h = static_cast<T*>(p.h) + t * p.ld_h + at;
  uint4 qx[V], qr[V], qw[V];
  f32x2 v[V][N / 2];
  griddep_wait();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (at + i * width * N < H) {
      qx[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * width * N));
      if (kSum && p.residual != nullptr) qr[i] = __ldcs(reinterpret_cast<const uint4*>(r + i * width * N));
      qw[i] = *reinterpret_cast<const uint4*>(w + i * width * N);
    }
  }
  f32x2 ss2 = pair(0.0f, 0.0f);
  float m = 0.0f;   // max|h * weight|
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (at + i * width * N < H) {
      unpack(qx[i], v[i], T{});
      if (kSum && p.residual != nullptr) {
        f32x2 a[N / 2];
        unpack(qr[i], a, T{});
#pragma unroll
        for (int k = 0; k < N / 2; ++k) v[i][k] = add2(v[i][k], a[k]);
        if (p.h != nullptr) store_vec(h + i * width * N, v[i]);
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) ss2 = fma2(v[i][k], v[i][k], ss2);
      if (kScaled) {
        f32x2 g[N / 2];
        unpack(qw[i], g, T{});
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const f32x2 hw = mul2(v[i][k], g[k]);
          m = max_abs(m, max_abs(fabsf(first(hw)), fabsf(second(hw))));
        }
      }
    }
  }
  float ss = first(ss2) + second(ss2);
  ss = lanes_sum<kLanes ? kLanes : 32>(ss);
  if (kScaled) m = lanes_max_abs<kLanes ? kLanes : 32>(m);
  if (!kLanes) {
    if (lane == 0) sm[warp] = make_float2(ss, m);
    __syncthreads();
    const float2 a = lane < width / 32 ? sm[lane] : make_float2(0.0f, 0.0f);
    ss = warp_sum(a.x);
    if (kScaled) m = lanes_max_abs<32>(a.y);
  }
  O* y = static_cast<O*>(p.y) + t * p.ld_y + at;
  const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
  if (at == 0 && H > 0 && p.rstd != nullptr) p.rstd[t] = rstd;
  // The thread's i-th vectors of h and of the weight
  auto operands = [&](int i, f32x2 (&g)[N / 2]) {
    if (!kSum) {
      // the row again (the compiler is kept from holding on to it)
      asm volatile("" : "+r"(qx[i].x), "+r"(qx[i].y), "+r"(qx[i].z), "+r"(qx[i].w));
      unpack(qx[i], v[i], T{});
    }
    unpack(qw[i], g, T{});
  };
  float inv = p.inv_scale, up = 1.0f;
  if (kScaled) {
    // Where the products have kept well within fp32's range, as those of ordinary rows do, max|y| is m * rstd
    // and y / scale is h * weight * (448 / m). Other rows (masked to the type's lowest value, of zeros, of large
    // weights) take both from y itself, which costs a second reduction.
    const float s = m * rstd * (1.0f / 448.0f);
    const bool left = H > 0 && !(m > 1e-30f && m < 1e30f && s > 0.0f);
    if (!left) {
      inv = __fdividef(448.0f, m);
      if (at == 0 && H > 0) p.row_scale[t] = s;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at + i * width * N < H) {
          f32x2 g[N / 2];
          operands(i, g);
#pragma unroll
          for (int k = 0; k < N / 2; ++k) g[k] = mul2(mul2(v[i][k], g[k]), pair(inv, inv));
          store_vec(y + i * width * N, g);
        }
      }
    }
    if (kLanes ? !__any_sync(0xFFFFFFFFu, left) : !left) return;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (at + i * width * N < H) {
        f32x2 g[N / 2];
        operands(i, g);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          g[k] = mul2(mul2(v[i][k], pair(rstd, rstd)), g[k]);
          a = max_abs(a, max_abs(fabsf(first(g[k])), fabsf(second(g[k]))));
        }
      }
    }
    a = lanes_max_abs<kLanes ? kLanes : 32>(a);
    if (!kLanes) {
      __syncthreads();   // the sums are read
      if (lane == 0) sm[warp].y = a;
      __syncthreads();
      a = lanes_max_abs<32>(lane < width / 32 ? sm[lane].y : 0.0f);
    }
    if (!left) return;
    const float sa = row_scale(a, &inv, &up);
    if (at == 0) p.row_scale[t] = sa;
  }
  // y = h * rstd * weight in this order: h * weight may be infinite where y is not
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (at + i * width * N < H) {
      f32x2 g[N / 2];
      operands(i, g);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        g[k] = mul2(mul2(v[i][k], pair(rstd, rstd)), g[k]);
        if (kScaled) g[k] = mul2(g[k], pair(up, up));
        if (sizeof(O) == 1) g[k] = mul2(g[k], pair(inv, inv));
      }
      store_vec(y + i * width * N, g);
    }
  }
}

// Rows too long for that: one block per row, a pass for the sum of squares, a pass for the largest |y|
// where the row's scale is wanted, a pass that stores; all but the first read the row from L1 / L2.
template <typename T, typename O>
__global__ void __launch_bounds__(kLong) tdx_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = kVec<T>;
  __shared__ float sm[kLong / 32];
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
  for (int c = threadIdx.x * N; c < p.H; c += kLong * N) {
    float v[N];
    load_h(c, v);
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = block_reduce<false, kLong>(ss, sm);
  const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
  if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[t] = rstd;
  float inv = p.inv_scale, up = 1.0f;
  bool within = false;   // as in the kernel above
  if (p.row_scale != nullptr) {
    float m = 0.0f;
    for (int c = threadIdx.x * N; c < p.H; c += kLong * N) {
      float v[N], g[N];
      load_h(c, v);
      load_vec(w + c, g);
#pragma unroll
      for (int i = 0; i < N; ++i) m = max_abs(m, fabsf(v[i] * g[i]));
    }
    m = block_reduce<true, kLong>(m, sm);
    float s = m * rstd * (1.0f / 448.0f);
    within = m > 1e-30f && m < 1e30f && s > 0.0f;
    inv = __fdividef(448.0f, m);
    if (!within) {
      m = 0.0f;
      for (int c = threadIdx.x * N; c < p.H; c += kLong * N) {
        float v[N], g[N];
        load_h(c, v);
        load_vec(w + c, g);
#pragma unroll
        for (int i = 0; i < N; ++i) m = max_abs(m, fabsf(v[i] * rstd * g[i]));
      }
      s = row_scale(block_reduce<true, kLong>(m, sm), &inv, &up);
    }
    if (threadIdx.x == 0) p.row_scale[t] = s;
  }
  for (int c = threadIdx.x * N; c < p.H; c += kLong * N) {
    float v[N], g[N];
    load_h(c, v);
    load_vec(w + c, g);
    if (h != nullptr) store_vec(h + c, v);
    if (within) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] * g[i] * inv;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = v[i] * rstd * g[i];
        if (sizeof(O) == 1) v[i] = v[i] * up * inv;
      }
    }
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

// Rows through a ring of kStages rows in shared memory, filled by cp.async: every thread copies the vectors
// that it reads itself, so that the ring needs no barrier and the loads of the rows to come run on
// through the row's sum. A thread keeps the sums of dweight of its E columns in registers over all its
// rows and stores them once, [blocks][H] fp32 for tdx_rmsnorm_dweight_kernel. kLanes as above.
// Bound by HBM (8 bytes an element in bf16 with dres): 16381 x 8192 157 us with the sums' second kernel
// (6.8 TB/s, a plain copy's rate 161), 100001 x 1024 120 us (123), 8000 x 16384 161 us (157), 262144 x 128
// 45 us (40). Ring depth 2 / 3 / 4 at 16381 x 8192: 158 (32 columns a thread) / 157 / 158 us. Two blocks of
// 512 threads per SM, at 64 registers, spill: 223 us. Spills that stay: 48 to 72 bytes in the fp32 instances for up to
// 256 columns (64 columns 89% of a copy's rate; in bf16, without any, 93%), 28 in the bf16 one for more than 8192.
template <typename T, int E, int kStages, int kMaxThreads, int kBlocks, int kLanes>
__global__ void __launch_bounds__(kMaxThreads, kBlocks)
    tdx_rmsnorm_bwd_rows_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int N = kVec<T>;
  constexpr int V = E / N;
  extern __shared__ uint4 ring[];   // [stage][dy, h, dres][vector][thread]
  __shared__ float sm[2][16];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kGroups = kLanes ? kThreads / (kLanes ? kLanes : 1) : 1;   // rows that a block has in hand
  const int width = kLanes ? kLanes : blockDim.x;
  const int group = kLanes ? threadIdx.x / (kLanes ? kLanes : 1) : 0;
  const int at = (threadIdx.x - group * width) * N;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const T* dy = static_cast<const T*>(p.dy) + at;
  const T* h = static_cast<const T*>(p.h) + at;
  const T* dr = static_cast<const T*>(p.dres) + at;
  const bool res = p.dres != nullptr;
  uint4* mine = ring + threadIdx.x;
  const uint32_t dst = smem_u32(mine);
  griddep_wait();
  auto fetch = [&](int64_t t, int s) {
    if (t < p.T) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at + i * width * N < p.H) {
          const uint32_t d = dst + (s * 3 * V + i) * blockDim.x * 16;
          cp_async16(d, dy + t * p.ld_dy + i * width * N);
          cp_async16(d + V * blockDim.x * 16, h + t * p.ld_h + i * width * N);
          if (res) cp_async16(d + 2 * V * blockDim.x * 16, dr + t * p.ld_dres + i * width * N);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(first + s * step, s);
  // 32 columns a thread and 512 threads: the weight waits in shared memory, behind the ring (in registers
  // it spills: 8000 x 16384 226 against 161 us)
  constexpr bool kWeightApart = kMaxThreads * E > 8192 && kLanes == 0;
  uint4* const apart = mine + kStages * 3 * V * blockDim.x;
  uint4 qw[V];
  float acc[V][N];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    qw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (at + i * width * N < p.H)
      qw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.weight) + at + i * width * N);
    if (kWeightApart) apart[i * blockDim.x] = qw[i];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[i][k] = 0.0f;
  }
  int s = 0, flip = 0;
  float next_rstd = first < p.T ? p.rstd[first] : 0.0f;
  // all groups of a warp go round as often as its first: their shuffles are shared
  for (int64_t t = first; t - (kLanes ? group % (32 / (kLanes ? kLanes : 32)) : 0) < p.T; t += step) {
    const float rstd = next_rstd;
    next_rstd = t + step < p.T ? p.rstd[t + step] : 0.0f;
    cp_async_wait<kStages - 1>();
    uint4 qd[V], qh[V], qr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (at + i * width * N < p.H && t < p.T) {
        const uint4* q = mine + (s * 3 * V + i) * blockDim.x;
        qd[i] = q[0];
        qh[i] = q[V * blockDim.x];
        if (res) qr[i] = q[2 * V * blockDim.x];
      } else {
        qd[i] = qh[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float d[N], v[N], g[N];
      unpack(qd[i], d, T{});
      unpack(qh[i], v, T{});
      unpack(kWeightApart ? apart[i * blockDim.x] : qw[i], g, T{});
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float n = v[k] * rstd;
        dot = fmaf(d[k] * g[k], n, dot);
        acc[i][k] = fmaf(d[k], n, acc[i][k]);
      }
    }
    fetch(t + kStages * step, s);   // the stage is read
    dot = lanes_sum<kLanes ? kLanes : 32>(dot);
    if (!kLanes) {
      if (lane == 0) sm[flip][warp] = dot;
      __syncthreads();
      dot = warp_sum(lane < width / 32 ? sm[flip][lane] : 0.0f);
      flip ^= 1;
    }
    const float mean = dot / static_cast<float>(p.H);
    T* dx = static_cast<T*>(p.dx) + t * p.ld_dx + at;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (at + i * width * N < p.H && t < p.T) {
        float d[N], v[N], g[N];
        unpack(qd[i], d, T{});
        unpack(qh[i], v, T{});
        unpack(kWeightApart ? apart[i * blockDim.x] : qw[i], g, T{});
#pragma unroll
        for (int k = 0; k < N; ++k) d[k] = rstd * (d[k] * g[k] - v[k] * rstd * mean);
        if (res) {
          unpack(qr[i], v, T{});
#pragma unroll
          for (int k = 0; k < N; ++k) d[k] += v[k];
        }
        store_vec(dx + i * width * N, d);
      }
    }
    s = s + 1 == kStages ? 0 : s + 1;
  }
  cp_async_wait<0>();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
  if (kLanes) {
    // the groups' sums, added in the order of the groups
    float* all = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at + i * width * N < p.H) store_vec(all + group * p.H + at + i * width * N, acc[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += kThreads) {
      float a = 0.0f;
      for (int i = 0; i < kGroups; ++i) a += all[i * p.H + c];
      out[c] = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at + i * width * N < p.H) store_vec(out + at + i * width * N, acc[i]);
  }
}

// Rows too long for the ring: a block takes rows b, b + grid, ... and adds up dy * n of its columns in shared memory.
template <typename T>
__global__ void __launch_bounds__(kLongBwd) tdx_rmsnorm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int N = kVec<T>;
  extern __shared__ float dw[];
  __shared__ float sm[kLongBwd / 32];
  griddep_wait();
  for (int c = threadIdx.x * N; c < p.H; c += kLongBwd * N)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[c + i] = 0.0f;
  const T* w = static_cast<const T*>(p.weight);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + t * p.ld_dy;
    const T* h = static_cast<const T*>(p.h) + t * p.ld_h;
    const float rstd = p.rstd[t];
    float dot = 0.0f;
    for (int c = threadIdx.x * N; c < p.H; c += kLongBwd * N) {
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
    const float mean = block_reduce<false, kLongBwd>(dot, sm) / static_cast<float>(p.H);
    const T* dr = p.dres ? static_cast<const T*>(p.dres) + t * p.ld_dres : nullptr;
    T* dx = static_cast<T*>(p.dx) + t * p.ld_dx;
    for (int c = threadIdx.x * N; c < p.H; c += kLongBwd * N) {
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
  for (int c = threadIdx.x * N; c < p.H; c += kLongBwd * N)
#pragma unroll
    for (int i = 0; i < N; ++i) out[c + i] = dw[c + i];
}

// dweight[c] = the sum of column c's partial sums (5 MB at most up to H = 8192, 10 up to 16384, in L2): warp w adds
// the row groups w, w + 32, ... of 64 columns, the warps' sums follow in order.
__global__ void __launch_bounds__(1024) tdx_rmsnorm_dweight_kernel(const float* part, float* dweight, int parts, int H) {
  __shared__ float2 sm[32][33];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 64 + lane * 2;
  float2 a = make_float2(0.0f, 0.0f);
  griddep_wait();
  if (c < H) {
#pragma unroll 10
    for (int b = warp; b < parts; b += 32) {
      const float2 v = *reinterpret_cast<const float2*>(part + static_cast<int64_t>(b) * H + c);
      a.x += v.x;
      a.y += v.y;
    }
  }
  sm[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < H) {
    for (int i = 1; i < 32; ++i) {
      a.x += sm[i][lane].x;
      a.y += sm[i][lane].y;
    }
    *reinterpret_cast<float2*>(dweight + c) = a;
  }
}

// Largest dynamic shared memory of a kernel, raised once per device (calls may come from several threads)
template <typename K>
bool raise_smem(K kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return true;
}

template <typename T, typename O, bool kScaled, int E, int kLanes>
tdx_status launch_norm_lanes(const NormParams& p, cudaStream_t st) {
  const int rows = kThreads / kLanes;
  return launch_rows(tdx_rmsnorm_rows_kernel<T, O, E, kLanes, true, kScaled>,
                     static_cast<unsigned>((static_cast<int64_t>(p.T) + rows - 1) / rows), kThreads, 0, st, p);
}

template <typename T, typename O, bool kScaled, int E, bool kSum>
tdx_status launch_norm_block(const NormParams& p, cudaStream_t st) {
  const unsigned block = static_cast<unsigned>((p.H + 32 * E - 1) / (32 * E) * 32);
  return launch_rows(tdx_rmsnorm_rows_kernel<T, O, E, 0, kSum, kScaled>, p.T, block, 0, st, p);
}

template <typename T, typename O, bool kScaled>
tdx_status launch_norm_t(const NormParams& p, cudaStream_t st) {
  if (p.H <= 64) return launch_norm_lanes<T, O, kScaled, 8, 8>(p, st);
  if (p.H <= 128) return launch_norm_lanes<T, O, kScaled, 8, 16>(p, st);
  if (p.H <= 256) return launch_norm_lanes<T, O, kScaled, 8, 32>(p, st);
  if (p.H <= 512) return launch_norm_lanes<T, O, kScaled, 16, 32>(p, st);
  if (p.H <= 1024) return launch_norm_lanes<T, O, kScaled, 32, 32>(p, st);
  if (p.H <= 16384) {
    // 32 elements a thread carry more loads per block of bf16 rows (32768 x 7168 with the residual 268 us, with 16
    // 293); fp32 rows take 16 (48076 x 1040 without a residual 80% of a copy's rate, with 32 60%), as do up to one
    // row per SM (1 x 8192 bf16 2.0 us, with 32 2.2)
    if constexpr (sizeof(T) == 2) {
      if (p.T > sm_count())
        return p.residual != nullptr ? launch_norm_block<T, O, kScaled, 32, true>(p, st)
                                     : launch_norm_block<T, O, kScaled, 32, false>(p, st);
    }
    return p.residual != nullptr ? launch_norm_block<T, O, kScaled, 16, true>(p, st)
                                 : launch_norm_block<T, O, kScaled, 16, false>(p, st);
  }
  return launch_rows(tdx_rmsnorm_kernel<T, O>, p.T, kLong, 0, st, p);
}

template <typename T>
tdx_status launch_norm(tdx_dtype out, const NormParams& p, cudaStream_t st) {
  switch (out) {
    case TDX_BF16: return launch_norm_t<T, bf16, false>(p, st);
    case TDX_FP32: return launch_norm_t<T, float, false>(p, st);
    default:
      return p.row_scale != nullptr ? launch_norm_t<T, e4m3, true>(p, st) : launch_norm_t<T, e4m3, false>(p, st);
  }
}

// Blocks per SM of the gradient's kernel, as many as its registers and shared memory leave room for: 512 threads
// where a block takes a row, 16 elements a thread (24224 x 2064 bf16: 93% of a copy's rate with three blocks of 160
// threads, 69% with two)
constexpr int bwd_block(int H, int e) { return (H + 32 * e - 1) / (32 * e) * 32; }
constexpr int bwd_blocks(int H) {
  return H <= 256 ? 4 : H <= 512 ? 2 : H <= 1024 ? 1 : H <= 8192 ? 512 / bwd_block(H, 16) : 1;
}
// Most row groups whose partial sums of dweight are added at the end: what the workspace holds
constexpr int bwd_most_parts(int H) { return H <= 16384 ? 152 * bwd_blocks(H) : kBwdParts; }

template <typename T, int E, int kStages, int kMaxThreads, int kBlocks, int kLanes>
tdx_status launch_bwd_rows(const NormBwdParams& p, int* parts, cudaStream_t st) {
  static std::atomic<bool> done[64];
  // the ring, and the weight where a thread has 32 columns of a long row
  constexpr int kRows = kStages * 3 + (kMaxThreads * E > 8192 && kLanes == 0 ? 1 : 0);
  constexpr int kMost = kRows * E * static_cast<int>(sizeof(T)) * kMaxThreads;
  const auto kernel = tdx_rmsnorm_bwd_rows_kernel<T, E, kStages, kMaxThreads, kBlocks, kLanes>;
  if (kMost > 48 * 1024 && !raise_smem(kernel, kMost, done)) return TDX_ERR_CUDA;
  const int block = kLanes ? kThreads : bwd_block(p.H, E);
  const int rows = kLanes ? kThreads / (kLanes ? kLanes : 1) : 1;
  const int64_t want = (static_cast<int64_t>(p.T) + rows - 1) / rows;
  const int most = std::min(bwd_most_parts(p.H), bwd_blocks(p.H) * (sm_count() > 0 ? sm_count() : kRefSMs));
  *parts = static_cast<int>(want < most ? want : most);
  return launch_rows(kernel, *parts, block, static_cast<size_t>(kRows) * E * sizeof(T) * block, st, p);
}

template <typename T>
tdx_status launch_norm_bwd(const NormBwdParams& p, int* parts, cudaStream_t st) {
  if (p.H <= 64) return launch_bwd_rows<T, 8, 2, kThreads, 4, 8>(p, parts, st);
  if (p.H <= 128) return launch_bwd_rows<T, 8, 2, kThreads, 4, 16>(p, parts, st);
  if (p.H <= 256) return launch_bwd_rows<T, 8, 2, kThreads, 4, 32>(p, parts, st);
  if (p.H <= 512) return launch_bwd_rows<T, 16, 2, kThreads, 2, 32>(p, parts, st);
  if (p.H <= 1024) return launch_bwd_rows<T, 32, 2, kThreads, 1, 32>(p, parts, st);
  if (p.H <= 8192) return launch_bwd_rows<T, 16, sizeof(T) == 2 ? 3 : 2, 512, 1, 0>(p, parts, st);
  if constexpr (sizeof(T) == 2) {
    if (p.H <= 16384) return launch_bwd_rows<T, 32, 2, 512, 1, 0>(p, parts, st);
  }
  static std::atomic<bool> done[64];
  const size_t smem = static_cast<size_t>(p.H) * sizeof(float);
  if (!raise_smem(tdx_rmsnorm_bwd_kernel<T>, 32768 * static_cast<int>(sizeof(float)), done)) return TDX_ERR_CUDA;
  *parts = std::min(p.T, bwd_most_parts(p.H));
  return launch_rows(tdx_rmsnorm_bwd_kernel<T>, *parts, kLongBwd, smem, st, p);
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
  return dtype == TDX_FP8_E4M3 || H > (1 << 28) ? TDX_ERR_UNSUPPORTED : TDX_OK;
}

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
  if (!known(o.out_dtype) || !(o.eps >= 0.0f) || !std::isfinite(o.eps) || !usable_scale(o.out_scale))
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
  p.inv_h = 1.0f / static_cast<float>(H);
  p.inv_scale = o.out_dtype == TDX_FP8_E4M3 ? 1.0f / o.out_scale : 1.0f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == TDX_BF16 ? launch_norm<bf16>(o.out_dtype, p, st) : launch_norm<float>(o.out_dtype, p, st);
}

tdx_status tdx_rmsnorm_bwd_workspace_size(int T, int H, tdx_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return TDX_ERR_INVALID_ARG;
  const tdx_status s = check_sizes(T, H, dtype);
  if (s != TDX_OK) return s;
  if (H > 32768) return TDX_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(T < 1 ? 1 : std::min(T, bwd_most_parts(H))) * H * sizeof(float);
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
  int parts = 0;
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
    s = dtype == TDX_BF16 ? launch_norm_bwd<bf16>(p, &parts, st) : launch_norm_bwd<float>(p, &parts, st);
    if (s != TDX_OK) return s;
  }
  return launch_rows(tdx_rmsnorm_dweight_kernel, (H + 63) / 64, 1024, 0, st,
                     static_cast<const float*>(part), dweight, parts, H);
}

}  // extern "C"
