// Shared by the row-wise operators (norm, routing, gated SiLU): 16-byte loads and converting
// stores of bf16 / fp32 / e4m3 values, warp and block sums, the launch with programmatic
// dependent launch, and host-side argument checks.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/tdx.h"
#include "tdx_internal.h"
#include "tdx_ptx.cuh"

namespace tdx {

using bf16 = __nv_bfloat16;
struct e4m3 {
  uint8_t bits;
};

// Elements of T in 16 bytes
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8], bf16) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4], float) {
  v[0] = __uint_as_float(q.x);
  v[1] = __uint_as_float(q.y);
  v[2] = __uint_as_float(q.z);
  v[3] = __uint_as_float(q.w);
}
// Two fp32 values in a register pair: one instruction for both (each rounded as the scalar one rounds)
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float first(f32x2 a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float second(f32x2 a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <int N, typename T>
__device__ __forceinline__ void unpack(const uint4& q, f32x2 (&v)[N], T) {
  float f[2 * N];
  unpack(q, f, T{});
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[kVec<T>]) {
  unpack(*reinterpret_cast<const uint4*>(p), v, T{});
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Store N (4 or 8) consecutive values rounded to the output type
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store_vec(e4m3* p, const float (&v)[8]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3(v[0], v[1], v[2], v[3]), pack_e4m3(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store_vec(e4m3* p, const float (&v)[4]) {
  *reinterpret_cast<uint32_t*>(p) = pack_e4m3(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }

template <int N, typename O>
__device__ __forceinline__ void store_vec(O* p, const f32x2 (&v)[N]) {
  float f[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[2 * i] = first(v[i]);
    f[2 * i + 1] = second(v[i]);
  }
  store_vec(p, f);
}

// Sum and maximum over groups of L consecutive lanes (a power of two); every lane of the warp takes part
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// The larger of two magnitudes (no sign bit); a NaN is larger than any of them
__device__ __forceinline__ float max_abs(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
template <int L>
__device__ __forceinline__ float lanes_max_abs(float v) {
  if constexpr (L == 32) return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = max_abs(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) { return lanes_sum<32>(v); }
__device__ __forceinline__ float warp_max(float v) { return lanes_max<32>(v); }

// ------------------------------------------------------------------------------------ host side
// Launch with programmatic dependent launch: the grid may be scheduled before the stream's previous
// kernel has ended, and every kernel here calls griddep_wait before it touches global memory.
template <typename... KArgs, typename... Args>
tdx_status launch_rows(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? TDX_OK : TDX_ERR_CUDA;
}

inline bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
// A scale that the kernels may divide by: it and its reciprocal are positive and finite
inline bool usable_scale(float v) { return v > 0.0f && std::isfinite(v) && std::isfinite(1.0f / v); }
inline size_t bytes_of(tdx_dtype d) { return d == TDX_BF16 ? 2 : d == TDX_FP8_E4M3 ? 1 : 4; }
inline bool known(tdx_dtype d) { return d == TDX_BF16 || d == TDX_FP8_E4M3 || d == TDX_FP32; }

// Resolve a row stride (0 = dense) and check it: at least `len` elements, whole 16-byte steps
inline tdx_status row_stride(int64_t ld, int64_t len, size_t elt, int64_t* out) {
  if (ld == 0) ld = len;
  if (ld < len || ld > (INT64_C(1) << 40)) return TDX_ERR_INVALID_ARG;
  *out = ld;
  return (ld * static_cast<int64_t>(elt)) % 16 == 0 ? TDX_OK : TDX_ERR_ALIGNMENT;
}

int sm_count();   // SMs of the current device, 0 if unknown

}  // namespace tdx
