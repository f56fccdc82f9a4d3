// The product kernel behind tdx_linear, tdx_linear_bwd, tdx_grouped_gemm and tdx_grouped_gemm_bwd:
// D = A @ B with fp32 accumulators in Tensor Memory and an epilogue of scales, bias, activation,
// residual and one rounding.
//
// Forms. A is M x K, B is K x N; either may lie in memory with K or with its other dimension
// contiguous, and the tensor cores take both, so no operand is ever transposed by a pass of its own:
//   NN  A rows along K, B rows along N      (the layer itself)
//   NT  A rows along K, B stored N x K      (input gradient: dz @ weights^T)
//   TN  A stored K x M, B rows along N      (weight gradient: inputs^T @ dz)
// Groups. kFlat: one product. kRows: the M rows fall into E runs, run e multiplied by B[e]. kSums:
// the K rows of both operands fall into E runs, run e summed into output e.
//
// Roles (12 warps, one CTA per SM, persistent over tiles):
//   warp 0 lane 0  TMA loads of 128-byte K slices into a ring of shared-memory slots
//   warp 1 lane 0  tcgen05.mma into one of two accumulators; commits free slots, hand over accumulators
//   warp 2         kSums: a run's last slice also holds rows of the next run (the tail); they are cleared in
//                  shared memory, in both operands (0 times a foreign infinity would still be a NaN), in a slot
//                  of its own that is loaded early in the tile: with tails in the ring every tile waited 1.4 us
//   warps 4-11     epilogue: Tensor Memory -> registers -> output, while the next tile is multiplied
//
// Pairs (kPair): two CTAs run one 2-SM MMA stream on a 256 x 256 tile, each staging its 128 rows of A
// and half of B. Single CTAs take 128 x BN tiles; when they are fewer than the SMs a cluster of `split`
// CTAs shares a tile's K slices, and the partial accumulators are added through distributed shared
// memory in rank order, so no workspace is needed and the bits do not change from call to call.
//
// Every wait on a barrier is bounded; one that runs out sets *status (if given) and ends the kernel's work.
#pragma once

#include <atomic>
#include <type_traits>

#include "tdx_actmath.cuh"
#include "tdx_linear.h"
#include "tdx_rows.cuh"

namespace tdx {

constexpr int kLinStages = 6;
constexpr int kStoreBytes = 4096;   // an epilogue warp's staging: 32 rows of 128 bytes
constexpr int kTailAfter = 8;       // whole slices of a tile that are loaded in front of its tail


template <bool FP8, Form FORM, Group GROUP, bool PAIR>
struct LinCfg {
  static constexpr int ELT = FP8 ? 1 : 2;
  static constexpr int BN = lin_block_n(FP8, PAIR);
  static constexpr int BK = 128 / ELT;                 // K per slot
  static constexpr int UMMA_K = 32 / ELT;
  static constexpr int BOX_N = 128 / ELT;              // columns of a box of 128-byte rows
  static constexpr int BOX_BYTES = BK * 128;           // box of BK rows (operand with K not contiguous)
  static constexpr bool A_MN = FORM == TN;             // A's rows lie along M
  static constexpr bool B_MN = FORM != NT;             // B's rows lie along N
  static constexpr int A_BOXES = A_MN ? kBM / BOX_N : 1;
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int N_CTA = PAIR ? BN / 2 : BN;     // columns of B this CTA stages
  static constexpr int B_BOXES = B_MN ? N_CTA / BOX_N : N_CTA / 128;
  static constexpr int B_BOX_STEP = B_MN ? BOX_BYTES : 128 * 128;
  static constexpr int B_BYTES = N_CTA * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TM = PAIR ? 2 * kBM : kBM;      // rows of a tile
  static constexpr int TMEM_COLS = 2 * BN;
  // run ends and, for kRows, tiles in front of each run
  static constexpr int TABLE = GROUP == kFlat ? 0 : (GROUP == kRows ? 2 : 1) * (kMoeMaxExperts + 1) + 3;   // ints
  // staging for the output's TMA stores, but for the e4m3 kernel of single CTAs, whose slots are larger
  static constexpr int STORE = STAGE_BYTES > 32768 ? 0 : kNumEpiWarps * kStoreBytes;
  static constexpr int OTHER = STORE + 64 + TABLE * 4 + (2 * kLinStages + 8) * 8;
  static constexpr int FIT = (227 * 1024 - OTHER) / STAGE_BYTES;
  static constexpr int SLOTS = FIT < kLinStages ? FIT : kLinStages;
  static constexpr int STAGES = GROUP == kSums ? SLOTS - 1 : SLOTS;   // of the ring; kSums: one slot is the tails'
  static constexpr int NUM_BARS = 2 * STAGES + 8;      // full and empty per slot; accumulators; drain; tail
  static constexpr int SMEM_BYTES = SLOTS * STAGE_BYTES + STORE + NUM_BARS * 8 + 64 + TABLE * 4;
  static constexpr int PART_LD = BN + 4;               // row pitch of a partial: 16 bytes past the banks' period
  static constexpr uint32_t IDESC = (1u << 4) | ((FP8 ? 0u : 1u) << 7) | ((FP8 ? 0u : 1u) << 10) |
                                    ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                                    (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(TM >> 4) << 24);
  static_assert(!FP8 || FORM == NN, "e4m3 operands: the forward product only");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(PAIR || kBM * PART_LD * 4 <= SLOTS * STAGE_BYTES, "a partial fits the slots");
};

// ------------------------------------------------------------------------------------ bounded waits
template <uint64_t LIMIT>
static __device__ __noinline__ bool lin_wait_slow(uint32_t* status, uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 0u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > LIMIT) {
        if (status != nullptr) *status = TDX_ERR_TIMEOUT;
        *abort_flag = 1;
        return false;
      }
    }
  }
}
template <uint64_t LIMIT = kLinTimeoutNs>
__device__ __forceinline__ bool lin_wait(uint32_t* status, uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || lin_wait_slow<LIMIT>(status, bar, parity, abort_flag);
}

// ------------------------------------------------------------------------------------------- tiles
struct LinTile {
  int e;            // expert (0 without groups)
  int m0, mend;     // first row of this CTA's tile, end of its rows
  int nt;           // tile column
  int k0;           // first K index
  int klen;         // K indexes of the whole tile
  int kb0, kb1;     // this CTA's slices
};

// Position `pos` of tm x tn tiles: columns in groups of gn; inside a group rows outer, columns inner, so
// that the tiles at work at one time share few rows of A and few columns of B
__device__ __forceinline__ void lin_raster(int pos, int tm, int tn, int gn, int* mt, int* nt) {
  const int per = tm * gn, full = tn / gn;
  const int g = pos / per;
  const int w = g < full ? gn : tn - full * gn;
  const int q = pos - g * per;
  *mt = q / w;
  *nt = g * gn + (q - *mt * w);
}

template <class C, Group GROUP, bool PAIR>
__device__ __forceinline__ LinTile lin_tile(const LinParams& p, const int* off, const int* cum, int it, int crank) {
  LinTile t;
  int mt;
  t.k0 = 0;
  t.klen = p.K;
  if constexpr (GROUP == kRows) {
    const int q = it / p.tiles_n;
    int lo = 0, hi = p.E;   // cum[lo] <= q < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= q) lo = mid;
      else hi = mid;
    }
    t.e = lo;
    lin_raster(it - cum[lo] * p.tiles_n, cum[lo + 1] - cum[lo], p.tiles_n, p.group_n, &mt, &t.nt);
    t.m0 = off[lo] + mt * C::TM;
    t.mend = off[lo + 1];
  } else {
    int pos = it;
    t.e = 0;
    if constexpr (GROUP == kSums) {
      const int per = p.tiles_m * p.tiles_n;
      t.e = it / per;
      pos = it - t.e * per;
      t.k0 = off[t.e];
      t.klen = off[t.e + 1] - off[t.e];
    }
    lin_raster(pos, p.tiles_m, p.tiles_n, p.group_n, &mt, &t.nt);
    t.m0 = mt * C::TM;
    t.mend = p.M;
  }
  const int nkb = (t.klen + C::BK - 1) / C::BK;
  if constexpr (PAIR) {
    t.m0 += crank * kBM;
    t.kb0 = 0;
    t.kb1 = nkb;
  } else {
    t.kb0 = static_cast<int>(static_cast<int64_t>(nkb) * crank / p.split);
    t.kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (crank + 1) / p.split);
  }
  return t;
}

// One warp: the runs' ends as given, clamped to [0, rows] and never descending, and the count of tiles
// (of tile_rows rows) in front of each run, where cum is not NULL
__device__ __forceinline__ void lin_table(const int32_t* offsets, int E, int rows, int tile_rows, int* off, int* cum) {
  const int lane = threadIdx.x & 31;
  int32_t v[(kMoeMaxExperts + 32) / 32];
#pragma unroll
  for (int i = 0; i < (kMoeMaxExperts + 32) / 32; ++i) {
    const int e = i * 32 + lane;
    v[i] = e <= E ? min(max(offsets[e], 0), rows) : 0;
  }
  int last = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < (kMoeMaxExperts + 32) / 32; ++i) {
    if (i * 32 > E) break;
    int hi = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, hi, o);
      if (lane >= o) hi = max(hi, up);
    }
    hi = max(hi, last);
    int before = __shfl_up_sync(0xFFFFFFFFu, hi, 1);
    if (lane == 0) before = last;
    const int e = i * 32 + lane;
    // run e - 1 ends here
    int n = e > 0 && e <= E ? (hi - before + tile_rows - 1) / tile_rows : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) n += up;
    }
    if (e <= E) {
      off[e] = hi;
      if (cum != nullptr) cum[e] = tiles + n;
    }
    last = __shfl_sync(0xFFFFFFFFu, hi, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
}

// ---------------------------------------------------------------------------------------- epilogue
struct LinRow {
  int64_t out, res, z;   // element offsets of the row
  float scale;
};

template <class C, Group GROUP>
__device__ __forceinline__ LinRow lin_row(const LinParams& p, const LinTile& t, int row, float tile_scale) {
  LinRow r;
  r.out = static_cast<int64_t>(row) * p.ld_out + (GROUP == kSums ? t.e * p.out_step : 0);
  r.res = static_cast<int64_t>(row) * p.ld_res;
  r.z = static_cast<int64_t>(row) * p.ld_z;
  r.scale = p.row_scale != nullptr ? tile_scale * p.row_scale[row] : tile_scale;
  return r;
}

// Of the epilogue's steps the forward product (NN) alone has scales of rows, bias, z and activation, the weight
// gradient (TN) alone the addition to its output; the others' instances do without their code.
template <Form FORM>
struct LinSteps {
  static constexpr bool kForward = FORM == NN, kResidual = FORM != TN, kAccumulate = FORM == TN;
};

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// N values in bf16 at o, the first 8 alone unless `both`; 16 go out as one 32-byte store where the address
// allows it: a sector of L2 is then written once, not half by half
template <int N>
__device__ __forceinline__ void store_bf16(bf16* o, const float (&v)[N], bool both, bool wide) {
  const uint4 a = pack8(v);
  if (N == 16 && both) {
    const uint4 b = pack8(v + N - 8);
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(a.x), "r"(a.y), "r"(a.z),
                   "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                   : "memory");
    } else {
      st_v4(o, a);
      st_v4(o + 8, b);
    }
  } else {
    st_v4(o, a);
  }
}
// v += N values of bf16 at b
template <int N>
__device__ __forceinline__ void add_bf16(float (&v)[N], const bf16* b, bool both) {
#pragma unroll
  for (int h = 0; h < N; h += 8) {
    if (h > 0 && !both) break;
    float w[8];
    load_vec(b + h, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[h + i] += w[i];
  }
}

// Columns col .. col + N (8, or 16 of which the last 8 count if `both`) of one row: v the accumulators (SWIGLU: of
// the gate), u those of the other half. v becomes the values to round; z is stored.
template <Form FORM, int N>
__device__ __forceinline__ void lin_values(const LinParams& p, const LinRow& r, int col, bool both, float (&v)[N],
                                           float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= r.scale;
  if constexpr (LinSteps<FORM>::kForward) {
    if (p.bias != nullptr) add_bf16(v, p.bias + col, both);
    if (p.z != nullptr) store_bf16(p.z + r.z + col, v, both, p.wide_z);
    if (p.act != TDX_ACT_NONE) {
      act_forward(p.act, p.out_type == TDX_FP32, v);
      if (p.gated) {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] *= r.scale;
        if (p.bias != nullptr) add_bf16(u, p.bias + p.cols + col, both);
        if (p.z != nullptr) store_bf16(p.z + r.z + p.cols + col, u, both, p.wide_z);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= u[i];
      }
    }
  }
  if constexpr (LinSteps<FORM>::kResidual) {
    if (p.residual != nullptr) add_bf16(v, p.residual + r.res + col, both);
  }
}

// Round them and store them
template <Form FORM, int N>
__device__ __forceinline__ void lin_store(const LinParams& p, const LinRow& r, int col, bool both, float (&v)[N]) {
  if (p.out_type == TDX_BF16) {
    bf16* o = static_cast<bf16*>(p.out) + r.out + col;
    if (LinSteps<FORM>::kAccumulate && p.accumulate) add_bf16(v, o, both);
    store_bf16(o, v, both, p.wide);
  } else if (p.out_type == TDX_FP32) {
    float* o = static_cast<float*>(p.out) + r.out + col;
#pragma unroll
    for (int h = 0; h < N; h += 4) {
      if (h >= 8 && !both) break;
      float4 w = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
      if (LinSteps<FORM>::kAccumulate && p.accumulate) {
        const float4 old = *reinterpret_cast<const float4*>(o + h);
        w = make_float4(w.x + old.x, w.y + old.y, w.z + old.z, w.w + old.w);
      }
      *reinterpret_cast<float4*>(o + h) = w;
    }
  } else if constexpr (LinSteps<FORM>::kForward) {
#pragma unroll
    for (int h = 0; h < N; h += 8) {
      if (h > 0 && !both) break;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[h + i] * p.inv_out_scale;
      store_vec(static_cast<e4m3*>(p.out) + r.out + col + h, w);
    }
  }
}

__device__ __forceinline__ void st_shared_v4(uint8_t* row, int unit, int lane, uint4 q) {
  *reinterpret_cast<uint4*>(row + ((unit ^ (lane & 7)) * 16)) = q;
}

// TMA store of a staged box (coordinates innermost first), or its addition to fp32 values as they are (rounded to
// nearest, by L2: nothing is read back here), in this thread's bulk group
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 32 columns' values of a row plus the bias of their columns, and to z where it is kept; `n` of the columns exist
__device__ __forceinline__ void lin_bias_z(const LinParams& p, const LinRow& lr, int col, int n, bool row_ok, f32x2 (&v)[16]) {
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (8 * i >= n) break;
      f32x2 w[4];
      unpack(*reinterpret_cast<const uint4*>(p.bias + col + 8 * i), w, bf16{});
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * i + k] = add2(v[4 * i + k], w[k]);
    }
  }
  if (p.z != nullptr && row_ok) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (16 * i >= n) break;
      float f[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[2 * k] = first(v[8 * i + k]);
        f[2 * k + 1] = second(v[8 * i + k]);
      }
      store_bf16(p.z + lr.z + col + 16 * i, f, 16 * i + 8 < n, p.wide_z);
    }
  }
}

// The short epilogues, over a warp's columns [begin, last) of a tile that go out in boxes of 128-byte rows: 32
// columns at a time (the accumulators behind `last` are read, not stored), values in pairs. STEPS 0: scaled, perhaps with a
// row added (RES: the residual, or the output as it is, on its way ahead of its use), rounded; 1: bias, z and an
// approximate activation too; 2: SWIGLU, whose other half lies `other` columns on. The general loop takes some four
// times the instructions: 8192 x 512 x 8192 68 us with it, 57 with STEPS 0; 8192 x 1024 x 8192 with bias and GELU_TANH 125
// and 103 with 1, with SWIGLU 95 and 86 with 2.
template <bool F32, bool RES, int STEPS>
__device__ __forceinline__ void lin_short(const LinParams& p, const LinRow& lr, const bf16* add, uint32_t d, bool none,
                                          bool row_ok, int n0, int begin, int last, uint8_t* stage, int warp_row, int z,
                                          int other) {
  const int lane = threadIdx.x & 31;
  uint8_t* stage_row = stage + lane * 128;
  const f32x2 scale = pair(lr.scale, lr.scale);
  uint4 res[4];
  auto fetch = [&](int c) {
    const uint4* at = reinterpret_cast<const uint4*>(add + n0 + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row_ok && c + 8 * i < last) res[i] = at[i];
  };
  auto load = [&](uint32_t at, uint32_t (&r)[32]) {
    if (none) {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0u;
    } else {
      tmem_ld_32x32b_x32(at, r);
    }
  };
  if (RES) fetch(begin);
#pragma unroll 1
  for (int c = begin; c < last; c += 32) {
    uint32_t r[32], q[32];
    f32x2 v[16];
    __syncwarp();
    load(d + c, r);
    if (STEPS == 2) {
      load(d + other + c, q);
      tmem_ld_wait(q);
    }
    tmem_ld_wait(r);
    const int in_box = F32 ? 0 : c & 32;
    if (in_box == 0) {
      if (lane == 0) bulk_wait_read_all();   // the staging's last store has been read
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = mul2(pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), scale);
    if (STEPS > 0) {
      lin_bias_z(p, lr, n0 + c, last - c, row_ok, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = act_pair(STEPS == 2 ? TDX_ACT_SILU : p.act, v[i]);
    }
    if (STEPS == 2) {
      f32x2 u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = mul2(pair(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1])), scale);
      lin_bias_z(p, lr, p.cols + n0 + c, last - c, row_ok, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], u[i]);
    }
    if (RES) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x2 w[4];
        unpack(res[i], w, bf16{});
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * i + k] = add2(v[4 * i + k], w[k]);
      }
      if (c + 32 < last) fetch(c + 32);
    }
    // 16-byte units of a row, permuted as the 128-byte swizzle has them
#pragma unroll
    for (int i = 0; i < 16; i += F32 ? 2 : 4) {
      uint4 w;
      if (F32)
        w = make_uint4(__float_as_uint(first(v[i])), __float_as_uint(second(v[i])), __float_as_uint(first(v[i + 1])),
                       __float_as_uint(second(v[i + 1])));
      else
        w = make_uint4(pack_bf16(first(v[i]), second(v[i])), pack_bf16(first(v[i + 1]), second(v[i + 1])),
                       pack_bf16(first(v[i + 2]), second(v[i + 2])), pack_bf16(first(v[i + 3]), second(v[i + 3])));
      st_shared_v4(stage_row, F32 ? i / 2 : in_box / 8 + i / 4, lane, w);
    }
    if (F32 || in_box == 32 || c + 32 >= last) {
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&p.tm_c, smem_u32(stage), n0 + c - in_box, warp_row, z, F32 && p.accumulate);
        bulk_commit();
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ kernel
template <bool FP8, Form FORM, Group GROUP, bool PAIR, Sum SUM>
__global__ void __launch_bounds__(kNumThreads, 1) tdx_linear_kernel(const __grid_constant__ LinParams p) {
  using C = LinCfg<FP8, FORM, GROUP, PAIR>;
  constexpr int BN = C::BN;
  extern __shared__ __align__(1024) uint8_t smem[];   // checked below: swizzled boxes lie on 1024-byte boundaries
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::SLOTS * C::A_BYTES;
  uint8_t* staging = smem + C::SLOTS * C::STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + C::STORE);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);   // [0] Tensor Memory base, [1] abort
  int* off = reinterpret_cast<int*>(misc + 16);
  int* cum = GROUP == kRows ? off + kMoeMaxExperts + 1 : nullptr;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + C::STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * C::STAGES), tempty0 = smem_u32(bars + 2 * C::STAGES + 2);
  const uint32_t drain_bar = smem_u32(bars + 2 * C::STAGES + 4);
  // the tail's slot: loads landed (leader: and the peer's slot cleared), cleared, multiplied
  const uint32_t tail_in = smem_u32(bars + 2 * C::STAGES + 5), tail_full = tail_in + 8, tail_empty = tail_in + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = PAIR ? 2 : p.split;   // CTAs per cluster
  const int crank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = !PAIR || crank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(tail_in, PAIR && leader ? 2 : 1);
    mbar_init(tail_full, 1);
    mbar_init(tail_empty, 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, PAIR ? 2 * kNumEpiWarps : kNumEpiWarps);
    }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.tm_a);
    tma_prefetch_map(&p.tm_b);
    if (p.tma_out) tma_prefetch_map(&p.tm_c);
  }
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0 && p.status != nullptr) *p.status = TDX_ERR_CUDA;
    return;   // every CTA alike
  }
  if (warp == kMmaWarp) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&misc[0]), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&misc[0]), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (p.overlap != kOverlapSecond) griddep_wait();
  if (p.overlap == kOverlapFirst) griddep_launch_dependents();
  if constexpr (GROUP != kFlat) {
    if (warp == kCopyWarp0) lin_table(p.offsets, p.E, GROUP == kRows ? p.M : p.K, C::TM, off, cum);
  }
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const int cid = blockIdx.x / S, ncl = gridDim.x / S;
  const int items = GROUP == kRows ? cum[p.E] * p.tiles_n : p.items;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, tails = 0;   // parity of the tail slot's use
      bool stop = false;
      const uint64_t keep_a = policy_of(p.keep_a), keep_b = policy_of(p.keep_b);
      const uint32_t leader_full0 = PAIR ? mapa_shared(full0, 0) : full0;
      const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
      for (int it = cid; it < items && !stop; it += ncl) {
        const LinTile t = lin_tile<C, GROUP, PAIR>(p, off, cum, it, crank);
        // What stays the same over the tile's slices: this thread's pace is what small tiles wait for (a slice takes
        // it 240 cycles; with this inside 296, with a loop over boxes of few rows 568).
        const int n0 = t.nt * (LinSteps<FORM>::kForward && p.gated ? BN / 2 : BN);
        int n[C::B_BOXES];   // first columns of the boxes of B (SWIGLU: gate columns, then the other half's)
#pragma unroll
        for (int j = 0; j < C::B_BOXES; ++j) {
          const int c = (PAIR ? crank * C::N_CTA : 0) + j * (C::B_MN ? C::BOX_N : 128);
          n[j] = LinSteps<FORM>::kForward && p.gated && c >= BN / 2 ? p.cols + n0 + c - BN / 2 : n0 + c;
        }
        const int z = GROUP == kRows ? t.e : 0;
        // A tile of few rows loads only them: rows that a box fills with zeros past the end of A cost as much as
        // real ones (1 x 8192 x 8192: streaming B alone 23 us, with boxes of 8 or 16 rows of A 23, of 64 rows 31, of
        // 128 rows 33). The accumulators of the rows behind are never read.
        const bool few = !PAIR && !C::A_MN && t.mend - t.m0 <= p.few_rows;
        const CUtensorMap* map_a = few ? &p.tm_few : &p.tm_a;
        const uint32_t bytes = few ? p.few_rows * 128 + C::B_BYTES : C::STAGE_BYTES;
        int k = t.k0 + t.kb0 * C::BK;
        // The loads of slice kb into a slot. A tail is counted on this CTA's own barrier, a pair's other slices on
        // the leader's. Two instances of the code: with the choice made per load in one loop, the loop and not the
        // tensor cores set the pace (one run of 2048 rows, 2048 x 57344: 379 us against 272).
        auto load = [&](auto is_tail, uint32_t bar, uint32_t a, uint32_t b, int k) {
          constexpr bool kOwn = !PAIR || decltype(is_tail)::value;
          if constexpr (C::A_MN) {
#pragma unroll
            for (int j = 0; j < C::A_BOXES; ++j) {
              if constexpr (kOwn) tma_load_2d_hint(a + j * C::BOX_BYTES, &p.tm_a, bar, t.m0 + j * C::BOX_N, k, keep_a);
              else tma_load_2d_pair_hint(a + j * C::BOX_BYTES, &p.tm_a, bar, t.m0 + j * C::BOX_N, k, keep_a);
            }
          } else if constexpr (kOwn) {
            tma_load_2d_hint(a, map_a, bar, k, t.m0, keep_a);
          } else {
            tma_load_2d_pair_hint(a, &p.tm_a, bar, k, t.m0, keep_a);
          }
#pragma unroll
          for (int j = 0; j < C::B_BOXES; ++j) {
            const uint32_t dst = b + j * C::B_BOX_STEP;
            const int x = C::B_MN ? n[j] : k, y = C::B_MN ? k : n[j];
            if constexpr (kOwn) tma_load_3d_hint(dst, &p.tm_b, bar, x, y, z, keep_b);
            else tma_load_3d_pair_hint(dst, &p.tm_b, bar, x, y, z, keep_b);
          }
        };
        const bool tail = GROUP == kSums && t.kb1 > t.kb0 && t.kb1 * C::BK > t.klen;
        const int whole = tail ? t.kb1 - 1 : t.kb1;
        // whole slices to the ring up to slice `to`
        int kb = t.kb0;
        auto ring = [&](int to) {
          for (; kb < to && !stop; ++kb) {
            if (!lin_wait(p.status, empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
              stop = true;
              return;
            }
            if constexpr (!PAIR) mbar_arrive_expect_tx(full0 + 8 * stage, bytes);
            else if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * C::STAGE_BYTES);
            load(std::false_type{}, leader_full0 + 8 * stage, a0 + stage * C::A_BYTES, b0 + stage * C::B_BYTES, k);
            k += C::BK;
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        };
        if constexpr (GROUP == kSums) {
          if (tail) {
            // The tail goes to a slot of its own early in the tile, so that it is cleared long before its turn at the
            // end, but late enough that the last tile's tail has been multiplied.
            ring(min(whole, t.kb0 + kTailAfter));
            if (!stop && lin_wait(p.status, tail_empty, tails ^ 1u, abort_flag)) {
              mbar_arrive_expect_tx(tail_in, C::STAGE_BYTES);
              load(std::true_type{}, tail_in, a0 + C::STAGES * C::A_BYTES, b0 + C::STAGES * C::B_BYTES, t.k0 + whole * C::BK);
              tails ^= 1u;
            } else {
              stop = true;
            }
          }
        }
        ring(whole);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0 && leader) {
      int stage = 0, local = 0;
      uint32_t phase = 0, tails = 0;
      bool stop = false;
      const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
      for (int it = cid; it < items && !stop; it += ncl, ++local) {
        const LinTile t = lin_tile<C, GROUP, PAIR>(p, off, cum, it, crank);
        int acc = local & 1;
        if (!lin_wait(p.status, tempty0 + 8 * acc, ((local >> 1) & 1) ^ 1u, abort_flag)) break;
        tc_fence_after();
        uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
        int start = t.kb0;   // first slice in the accumulator
        // Other kinds than kOnce: the epilogue takes what is summed so far, slices from kb on are summed anew. kSegments
        // goes on with the other accumulator; kLongSegments with the same, as the epilogue has the other one in use:
        // its turn passes without a product.
        auto next_segment = [&](int kb) {
          for (int turn = 0; turn < (SUM == kLongSegments ? 2 : 1); ++turn) {
            if constexpr (PAIR) tc_commit_pair_multicast(tfull0 + 8 * acc, static_cast<uint16_t>(0x3));
            else tc_commit(tfull0 + 8 * acc);
            ++local;
            acc = local & 1;
            if (!lin_wait(p.status, tempty0 + 8 * acc, ((local >> 1) & 1) ^ 1u, abort_flag)) return false;
          }
          tc_fence_after();
          d = tmem_base + static_cast<uint32_t>(acc * BN);
          start = kb;
          return true;
        };
        // slice kb, once `full` is: into the accumulator, and its slot is free when that is done
        auto multiply = [&](int kb, uint32_t full, uint32_t parity, uint32_t a, uint32_t b, uint32_t empty) {
          if (!lin_wait(p.status, full, parity, abort_flag)) return false;
          tc_fence_after();
          const int in_segment = kb - (SUM == kOnce ? t.kb0 : start);
#pragma unroll
          for (int k = 0; k < C::BK / C::UMMA_K; ++k) {
            const uint64_t ad = C::A_MN ? smem_desc(a + k * C::UMMA_K * 128, C::BOX_BYTES, 1024, 2u)
                                        : smem_desc(a + k * 32, 16, 1024, 2u);
            const uint64_t bd = C::B_MN ? smem_desc(b + k * C::UMMA_K * 128, C::BOX_BYTES, 1024, 2u)
                                        : smem_desc(b + k * 32, 16, 1024, 2u);
            const uint32_t accum = in_segment > 0 || k > 0 ? 1u : 0u;
            if constexpr (PAIR) {
              if constexpr (FP8) umma_f8_pair(d, ad, bd, C::IDESC, accum);
              else umma_bf16_pair(d, ad, bd, C::IDESC, accum);
            } else {
              if constexpr (FP8) umma_f8(d, ad, bd, C::IDESC, accum);
              else umma_bf16(d, ad, bd, C::IDESC, accum);
            }
          }
          if constexpr (PAIR) tc_commit_pair_multicast(empty, static_cast<uint16_t>(0x3));
          else tc_commit(empty);
          return true;
        };
        const bool tail = GROUP == kSums && t.kb1 > t.kb0 && t.kb1 * C::BK > t.klen;
        const int whole = tail ? t.kb1 - 1 : t.kb1;
        int kb = t.kb0;
        auto ring = [&](int to) {
          for (; kb < to; ++kb) {
            if (!multiply(kb, full0 + 8 * stage, phase, a0 + stage * C::A_BYTES, b0 + stage * C::B_BYTES, empty0 + 8 * stage)) {
              stop = true;
              break;
            }
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        };
        if constexpr (SUM == kOnce) {
          ring(whole);
        } else {
          while (kb < whole && !stop) {
            ring(min(whole, start + p.segment));
            if (!stop && kb < t.kb1 && kb == start + p.segment) stop = !next_segment(kb);
          }
        }
        if constexpr (GROUP == kSums) {
          if (tail && !stop) {
            stop = !multiply(whole, tail_full, tails, a0 + C::STAGES * C::A_BYTES, b0 + C::STAGES * C::B_BYTES, tail_empty);
            tails ^= 1u;
          }
        }
        if (stop) break;
        if constexpr (PAIR) tc_commit_pair_multicast(tfull0 + 8 * acc, static_cast<uint16_t>(0x3));
        else tc_commit(tfull0 + 8 * acc);
      }
      // every MMA issued has completed once this barrier flips
      if constexpr (PAIR) tc_commit_pair(drain_bar);
      else tc_commit(drain_bar);
      int none = 0;
      lin_wait(p.status, drain_bar, 0, &none);
    }
  } else if (GROUP == kSums && warp == kCopyWarp0) {
    uint32_t tails = 0;
    for (int it = cid; it < items; it += ncl) {
      const LinTile t = lin_tile<C, GROUP, PAIR>(p, off, cum, it, crank);
      const int valid = t.klen - (t.kb1 - 1) * C::BK;
      if (t.kb1 == t.kb0 || valid >= C::BK) continue;
      // tiles without a tail go by unseen: this may wait for as long as they take (a loader that gave up sets the flag)
      const bool ok = lin_wait<kLinTailTimeoutNs>(p.status, tail_in, tails, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tails ^= 1u;
      // a K row is one 128-byte line of every box (the swizzle permutes 16-byte units inside a line)
      const int units = (C::BK - valid) * 8;
      for (int i = lane; i < units; i += 32) {
        const int at = valid * 128 + i * 16;
#pragma unroll
        for (int j = 0; j < C::A_BOXES; ++j)
          *reinterpret_cast<uint4*>(sA + C::STAGES * C::A_BYTES + j * C::BOX_BYTES + at) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < C::B_BOXES; ++j)
          *reinterpret_cast<uint4*>(sB + C::STAGES * C::B_BYTES + j * C::BOX_BYTES + at) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
      __syncwarp();
      // The second CTA of a pair tells the leader, whose arrival (after both) releases the slice. (Two arrivals on
      // every slice's barrier, one of them remote, cost 1 us a slice: 1583 us for 32749 rows of 2048 and 7168
      // columns over 16 experts.)
      if (lane == 0) {
        if (leader) mbar_arrive(tail_full);
        else mbar_arrive_cluster(mapa_shared(tail_in, 0));
      }
    }
  } else if (warp >= kEpiWarp0) {
    const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int local = 0;
    for (int it = cid; it < items; it += ncl, ++local) {
      const LinTile t = lin_tile<C, GROUP, PAIR>(p, off, cum, it, crank);
      const bool none = t.kb0 == t.kb1;   // nothing was multiplied: zeros
      const int in_tile = quarter * 32 + lane, row = t.m0 + in_tile;
      const bool row_ok = row < t.mend;
      const int width = LinSteps<FORM>::kForward && p.gated ? BN / 2 : BN;
      const int n0 = t.nt * width, first = half * (width / 2), last = min(first + width / 2, p.cols - n0);
      bool ok = true;
      auto release = [&](int acc) {   // the accumulator may be overwritten
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(mapa_shared(tempty0 + 8 * acc, 0));
          else mbar_arrive(tempty0 + 8 * acc);
        }
      };
      // The columns that this warp sums are those it reads again below, as its own stores alone are ordered before its
      // loads: of a gated tile a quarter of the gates and the same of the other half; of a cluster's partial its half.
      const bool apart = p.gated && (PAIR || S == 1);
      const int base = apart ? half * (BN / 4) : half * (BN / 2), skip = apart ? BN / 4 : 0;
      auto full = [&] {
        return __all_sync(0xFFFFFFFFu, lin_wait(p.status, tfull0 + 8 * (local & 1), (local >> 1) & 1, abort_flag));
      };
      if constexpr (SUM == kSegments) {
        // The tensor cores truncate every addition to an accumulator, always toward zero. Of bf16 products of one sign
        // a sum loses 8e-7 at K = 1024, 6.5e-5 at 16384, 3.4e-4 at 65536 and 6e-3 at 2^20; of normal inputs its error
        // is 1e-6, 1.9e-5, 7.6e-5 and 1.2e-3, against 1e-7 to 9e-7 for sums rounded to nearest. A result that stays
        // fp32 takes the sum of segments of kLinSegment slices, added here in fp32 (7e-7 to 1e-6 at all of these); the
        // last one's accumulator gets the total.
        const int segments = (t.kb1 - t.kb0 + p.segment - 1) / p.segment;
        if (segments > 1) {
          float sum[BN / 2];
#pragma unroll 1
          for (int g = 0; g < segments && ok; ++g, local += g < segments) {
            ok = full();
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = tmem_base + static_cast<uint32_t>((local & 1) * BN) + lanes + base;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < BN / 2; i += 16) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(at + i + (i >= BN / 4 ? skip : 0), r);
              tmem_ld_wait(r);
#pragma unroll
              for (int k = 0; k < 16; ++k) sum[i + k] = g == 0 ? __uint_as_float(r[k]) : sum[i + k] + __uint_as_float(r[k]);
            }
            if (g + 1 < segments) {
              release(local & 1);
            } else {
#pragma unroll
              for (int i = 0; i < BN / 2; i += 16) {
                uint32_t r[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(sum[i + k]);
                tmem_st_32x32b_x16(at + i + (i >= BN / 4 ? skip : 0), r);
              }
              tmem_st_wait();
            }
          }
        } else {
          ok = full();
        }
      } else {
        ok = full();
      }
      if constexpr (SUM == kLongSegments) {
        // In a result of 8 or 16 bits (half a step 4e-3) that shows past some 65536 of K alone. Its segments are so long
        // that their additions need not overlap the next one's products: the sums so far wait in the other
        // accumulator, and the last segment's gets the total. In instances of their own, as small tiles wait for the
        // others' code: 1 x 4096 x 8192 14.5 us, 14.7 with this in them; 131072 rows, 64 experts of 2048 x 2048, 733 us
        // with these, 719 with the others'.
        const int all = t.kb1 - t.kb0;   // left: slices from the present segment's first on
#pragma unroll 1
        for (int left = all; ok && all > p.segment && left > 0; left -= p.segment) {
          const bool last = left <= p.segment;
          tc_fence_after();
          const uint32_t mine = tmem_base + static_cast<uint32_t>((local & 1) * BN) + lanes + base;
          const uint32_t other = tmem_base + static_cast<uint32_t>((~local & 1) * BN) + lanes + base;
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < BN / 2; i += 16) {
            const uint32_t c = i + (i >= BN / 4 ? skip : 0);
            uint32_t r[16], q[16];
            tmem_ld_32x32b_x16(mine + c, r);
            tmem_ld_wait(r);
            if (left < all) {
              tmem_ld_32x32b_x16(other + c, q);
              tmem_ld_wait(q);
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(q[k]) + __uint_as_float(r[k]));
            }
            tmem_st_32x32b_x16((last ? mine : other) + c, r);
          }
          tmem_st_wait();
          if (left < all) release(~local & 1);   // the turn that passed
          if (!last) {
            release(local & 1);
            for (int turn = 0; turn < 2 && ok; ++turn) {
              ++local;
              ok = full();
            }
          }
        }
      }
      if (!ok) break;
      const int acc = local & 1;
      tc_fence_after();
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN) + lanes;
      if (!PAIR && S > 1) {
        // this CTA's partial, into the ring (its slots are free: every MMA of the tile has completed)
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32(d + c, r);
          tmem_ld_wait(r);
          if (t.m0 + in_tile < t.mend) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 q = make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]),
                                     __uint_as_float(r[i + 3]));
              if (none) q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              *reinterpret_cast<float4*>(part + in_tile * C::PART_LD + c + i) = q;
            }
          }
        }
        break;   // one tile per cluster
      }
      float scale = p.alpha;
      if (GROUP == kRows && p.expert_scale != nullptr) scale *= p.expert_scale[t.e];
      LinRow lr = {};
      if (row_ok) lr = lin_row<C, GROUP>(p, t, row, scale);
      // rows of 128 bytes go out through shared memory as TMA stores, which drop what lies past the output's
      // edges; not where the tile's rows end inside this warp's 32 and the next run's follow
      const int warp_row = t.m0 + quarter * 32;
      const bool box = C::STORE > 0 && p.tma_out && warp_row + (GROUP == kRows ? 31 : 0) < t.mend;
      uint8_t* stage_row = staging + (warp - kEpiWarp0) * kStoreBytes + lane * 128;
      const int box_cols = p.out_type == TDX_BF16 ? 64 : 32, z = GROUP == kSums ? t.e : 0;
      uint8_t* stage = staging + (warp - kEpiWarp0) * kStoreBytes;
      const bf16* add = LinSteps<FORM>::kResidual && p.residual != nullptr ? p.residual + lr.res : nullptr;
      if (LinSteps<FORM>::kAccumulate && p.accumulate) add = static_cast<const bf16*>(p.out) + lr.out;
      auto run = [&](auto f32, auto res, auto steps) {
        lin_short<decltype(f32)::value, decltype(res)::value, decltype(steps)::value>(
            p, lr, add, d, none, row_ok, n0, first, last, stage, warp_row, z, BN / 2);
      };
      using S0 = std::integral_constant<int, 0>;
      if (box && p.steps == 0 && p.out_type == TDX_FP32 && (LinSteps<FORM>::kAccumulate || add == nullptr)) {
        run(std::true_type{}, std::false_type{}, S0{});
      } else if (box && p.steps == 0 && p.out_type == TDX_BF16) {
        if (add != nullptr) run(std::false_type{}, std::true_type{}, S0{});
        else run(std::false_type{}, std::false_type{}, S0{});
      } else if (LinSteps<FORM>::kForward && SUM == kOnce && box && p.steps == 1 && add == nullptr) {
        run(std::false_type{}, std::false_type{}, std::integral_constant<int, LinSteps<FORM>::kForward ? 1 : 0>{});
      } else if (LinSteps<FORM>::kForward && SUM == kOnce && box && p.steps == 2 && add == nullptr) {
        run(std::false_type{}, std::false_type{}, std::integral_constant<int, LinSteps<FORM>::kForward ? 2 : 0>{});
      } else
      // a rolled loop over 16 columns: unrolled over the tile its code came from L2 anew with every tile
#pragma unroll 1
      for (int c = first; c < last; c += 16) {
        uint32_t r[16], q[16];
        float v[16], u[16];
        __syncwarp();
        tmem_ld_32x32b_x16(d + c, r);
        if (LinSteps<FORM>::kForward && p.gated) {
          tmem_ld_32x32b_x16(d + BN / 2 + c, q);
          tmem_ld_wait(q);
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = none ? 0.0f : __uint_as_float(q[i]);
        }
        tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = none ? 0.0f : __uint_as_float(r[i]);
        const int col = n0 + c, in_box = c & (box_cols - 1);
        const bool both = c + 8 < last;
        if (box && in_box == 0) {
          if (lane == 0) bulk_wait_read_all();   // the staging's last store has been read
          __syncwarp();
        }
        if (row_ok) {
          lin_values<FORM>(p, lr, col, both, v, u);
          if (!box) {
            lin_store<FORM>(p, lr, col, both, v);
          } else if (p.out_type == TDX_BF16) {
            // 16-byte units of a row, permuted as the 128-byte swizzle has them
            st_shared_v4(stage_row, in_box / 8, lane, pack8(v));
            st_shared_v4(stage_row, in_box / 8 + 1, lane, pack8(v + 8));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4(stage_row, in_box / 4 + k, lane,
                           make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                                      __float_as_uint(v[4 * k + 3])));
          }
        }
        if (box && (in_box + 16 == box_cols || c + 16 >= last)) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&p.tm_c, smem_u32(stage), col - in_box, warp_row, z, LinSteps<FORM>::kAccumulate && p.accumulate);
            bulk_commit();
          }
        }
      }
      release(acc);
    }
    if (lane == 0) bulk_wait_read_all();   // the stores read this CTA's shared memory
  }

  griddep_launch_dependents();
  __syncthreads();
  if (!PAIR && S > 1) {
    cluster_sync_all();   // every partial of the tile is written
    if (cid < items && warp >= kEpiWarp0 && !*abort_flag) {
      const LinTile t = lin_tile<C, GROUP, PAIR>(p, off, cum, cid, crank);
      const int width = p.gated ? BN / 2 : BN;
      const int n0 = t.nt * width, groups = width / 8;
      const int rows = min(kBM, t.mend - t.m0);
      float scale = p.alpha;
      if (GROUP == kRows && p.expert_scale != nullptr) scale *= p.expert_scale[t.e];
      const uint32_t part = smem_u32(smem);
      const int units = ((rows - crank + S - 1) / S) * groups;   // rows crank, crank + S, ...
      for (int i = threadIdx.x - kEpiWarp0 * 32; i < units; i += kEpiThreads) {
        const int r = crank + (i / groups) * S, c = (i % groups) * 8;
        if (n0 + c >= p.cols) continue;
        float v[8] = {}, u[8] = {};
        for (int s = 0; s < S; ++s) {
          const uint32_t at = mapa_shared(part + (r * C::PART_LD + c) * 4, s);
          const float4 a = ld_cluster_f4(at), b = ld_cluster_f4(at + 16);
          v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
          v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
          if (LinSteps<FORM>::kForward && p.gated) {
            const float4 x = ld_cluster_f4(at + BN / 2 * 4), y = ld_cluster_f4(at + BN / 2 * 4 + 16);
            u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
            u[4] += y.x; u[5] += y.y; u[6] += y.z; u[7] += y.w;
          }
        }
        const LinRow lr = lin_row<C, GROUP>(p, t, t.m0 + r, scale);
        lin_values<FORM>(p, lr, n0 + c, false, v, u);
        lin_store<FORM>(p, lr, n0 + c, false, v);
      }
    }
  }
  if (*abort_flag) {
    // loads that nothing waited for are given ample time to land before the shared memory is given up
    for (int i = 0; i < 256; ++i) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync_all();   // no CTA leaves while its peer may read from it, load into it or arrive on it
  else __syncthreads();
  if (p.overlap == kOverlapSecond) griddep_wait();   // see LinParams
  if (warp == kMmaWarp) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------------------------------------- host
template <bool FP8, Form FORM, Group GROUP, bool PAIR, Sum SUM>
tdx_status launch_linear_t(const LinParams& p, int want, cudaStream_t stream) {
  using C = LinCfg<FP8, FORM, GROUP, PAIR>;
  auto* kernel = tdx_linear_kernel<FP8, FORM, GROUP, PAIR, SUM>;
  // per device: raised shared-memory limit and, for pairs, the clusters that are resident together
  static std::atomic<int> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TDX_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.blockDim = dim3(kNumThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  int most = dev >= 0 && dev < 64 ? ready[dev].load(std::memory_order_relaxed) : 0;
  if (most == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return TDX_ERR_CUDA;
    most = sm_count();
    if (PAIR) {
      cfg.gridDim = dim3(2 * most, 1, 1);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return TDX_ERR_CUDA;
      most = n;
    }
    if (most <= 0) return TDX_ERR_CUDA;
    if (dev >= 0 && dev < 64) ready[dev].store(most, std::memory_order_relaxed);
  }
  // `want` clusters of work; with a split one cluster per tile, else persistent
  const int clusters = !PAIR && p.split > 1 ? want : (want < most ? want : most);
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * (PAIR ? 2 : p.split), 1, 1);
  cfg.attrs = attr;
  cfg.numAttrs = PAIR || p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? TDX_OK : TDX_ERR_CUDA;
}

template <bool FP8, Form FORM, Group GROUP, Sum SUM>
tdx_status launch_linear_g(const LinParams& p, bool pair, int want, cudaStream_t stream) {
  return pair ? launch_linear_t<FP8, FORM, GROUP, true, SUM>(p, want, stream)
              : launch_linear_t<FP8, FORM, GROUP, false, SUM>(p, want, stream);
}

}  // namespace tdx
