// Host side of tdx_linear, tdx_linear_bwd, tdx_grouped_gemm and tdx_grouped_gemm_bwd: argument checks,
// tensor maps, the choice of tiles and the launches.
#include <algorithm>

#include "tdx_linear.h"
#include "tdx_rows.cuh"

namespace tdx {

tdx_linear_opts linear_defaults() {
  tdx_linear_opts o;
  std::memset(&o, 0, sizeof(o));
  o.out_dtype = TDX_BF16;
  o.act = TDX_ACT_NONE;
  o.alpha = 1.0f;
  o.out_scale = 1.0f;
  o.dw_dtype = TDX_BF16;
  return o;
}

namespace {

constexpr int kMostSize = 1 << 30;
constexpr int64_t kMostBytes = INT64_C(1) << 40;   // a tensor map's strides stay below

// An operand's matrices as the kernel loads them: `rows` x `cols` elements with `cols` contiguous,
// E of them `step` elements apart
struct Operand {
  const void* p;
  int64_t rows, cols, ld, step;
  int E;
};

bool map_of(CUtensorMap* m, const Operand& o, bool fp8, int rank, int box_rows) {
  const uint64_t elt = fp8 ? 1 : 2;
  const uint64_t dims[3] = {static_cast<uint64_t>(o.cols), static_cast<uint64_t>(std::max<int64_t>(o.rows, 1)),
                            static_cast<uint64_t>(o.E)};
  const uint64_t strides[2] = {o.ld * elt, (o.E > 1 ? o.step : o.ld) * elt};
  const uint32_t box[3] = {static_cast<uint32_t>(128 / elt), static_cast<uint32_t>(box_rows), 1};
  return encode_map(m, o.p, static_cast<int>(elt), rank, dims, strides, box);
}

// How a product of about `tiles256` pair or `tiles1` single tiles of `nkb` K slices runs: in pairs, or on single
// CTAs, a tile's K slices over clusters of `split`
struct Shape {
  bool pair;
  int split;
};

// Microseconds, as measured over 1 .. 4096 rows, 512 .. 8192 of K and of N: a launch's fixed part; one K slice (128
// bytes of K) of a pair's and of a single CTA's tile; a persistent kernel's last epilogue; the addition of a tile's
// partials, once and for each 128 rows of each CTA; what a second wave of clusters adds.
constexpr float kLaunch = 5.0f, kPairSlice = 0.30f, kSingleSlice = 0.27f, kSingleSliceE4m3 = 0.33f;
constexpr float kPairEnd = 1.5f, kSingleEnd = 1.0f, kFold = 2.2f, kFoldRows = 1.8f, kFoldRowsCta = 0.7f, kWave = 3.0f;

Shape choose(bool fp8, int64_t tiles256, int64_t tiles1, int64_t most1, int nkb, float rows) {
  const int sms = sm_count() > 0 ? sm_count() : kRefSMs;
  auto waves = [](int64_t tiles, int at_once) { return static_cast<float>((tiles + at_once - 1) / at_once); };
  Shape best = {true, 1};
  float t = kLaunch + waves(tiles256, sms / 2) * nkb * kPairSlice + kPairEnd;
  const float slice = fp8 ? kSingleSliceE4m3 : kSingleSlice;
  for (int s = 1; s <= kMostSplit; ++s) {
    if (s > 1 && (s > nkb || most1 * s > 4 * sms)) break;
    float one = kLaunch + waves(tiles1, sms) * nkb * slice + kSingleEnd;
    if (s > 1) {
      const float w = waves(tiles1, lin_clusters(s));
      one = kLaunch + w * ((nkb + s - 1) / s * slice + kFold + rows / 128.0f * (kFoldRows + s * kFoldRowsCta)) + (w - 1) * kWave;
    }
    if (one < t) {
      t = one;
      best = {false, s};
    }
  }
  return best;
}

tdx_status stride_ok(int64_t ld, int64_t len, size_t elt, int64_t* out) {
  const tdx_status s = row_stride(ld, len, elt, out);
  if (s != TDX_OK) return s;
  return *out * static_cast<int64_t>(elt) < kMostBytes ? TDX_OK : TDX_ERR_UNSUPPORTED;
}

// Elements from one expert's matrix (K rows of ld) to the next one's; 0 where there is no next one
tdx_status expert_step(int E, int K, int64_t ld, int64_t elt, int64_t* step) {
  *step = 0;
  if (E <= 1) return TDX_OK;
  if (ld > kMostBytes / K || K * ld * elt >= kMostBytes) return TDX_ERR_UNSUPPORTED;
  *step = K * ld;
  return TDX_OK;
}

// The run of one product: p holds sizes (M, K, cols, E, offsets) and the epilogue
tdx_status run(Form form, Group group, bool fp8, LinParams& p, const Operand& a, const Operand& b, cudaStream_t st) {
  const int bk = fp8 ? 128 : 64;
  const int64_t rows = p.M, E = p.E;
  int64_t t256, t1, most1, most256;
  const int w256 = p.gated ? 128 : 256, w1 = p.gated ? lin_block_n(fp8, false) / 2 : lin_block_n(fp8, false);
  const int64_t n256 = (p.cols + w256 - 1) / w256, n1 = (p.cols + w1 - 1) / w1;
  int64_t k = p.K;
  if (group == kRows) {
    // tiles of E runs of unknown lengths: at most one part tile more per run that has rows
    const int64_t runs = std::min(E, rows);
    most256 = (rows + runs * 255) / 256 * n256;
    most1 = (rows + runs * 127) / 128 * n1;
    t256 = std::max<int64_t>(std::min((rows / 256 + (runs + 1) / 2) * n256, most256), 1);
    t1 = std::max<int64_t>(std::min((rows / 128 + (rows > runs * 64 ? (runs + 1) / 2 : runs)) * n1, most1), 1);
  } else {
    most256 = t256 = (rows + 255) / 256 * n256 * E;
    most1 = t1 = (rows + 127) / 128 * n1 * E;
    if (group == kSums) k = (k + E - 1) / E;
  }
  const int nkb = static_cast<int>((k + bk - 1) / bk);
  const int64_t tile_rows = group == kRows ? (rows + std::min(E, rows) - 1) / std::min(E, rows) : rows;
  const Shape shape = choose(fp8, t256, t1, most1, nkb, static_cast<float>(std::min<int64_t>(tile_rows, 128)));
  const int64_t most = shape.pair ? most256 : most1;
  if (most + kMoeMaxExperts * std::max(n1, n256) >= INT64_C(0x7FFFFFFF)) return TDX_ERR_UNSUPPORTED;
  const int bn = lin_block_n(fp8, shape.pair);
  const int width = p.gated ? bn / 2 : bn;
  const int tm = lin_tile_rows(shape.pair);
  p.tiles_n = (p.cols + width - 1) / width;
  p.tiles_m = group == kRows ? 0 : (p.M + tm - 1) / tm;
  p.items = group == kRows ? 0 : static_cast<int>(most);
  p.group_n = std::min(p.tiles_n, shape.pair ? 8 : 16);
  p.split = shape.split;
  // an operand that one tile alone reads is streamed through L2, others are kept there
  p.keep_a = p.tiles_n > 1 ? 1 : 0;
  p.keep_b = group == kRows ? (rows > std::min(E, rows) * tm ? 1 : 0) : (p.tiles_m > 1 ? 1 : 0);
  const int b_rows = form == NT ? 128 : bk;
  if (!map_of(&p.tm_a, a, fp8, 2, form == TN ? bk : kBM) || !map_of(&p.tm_b, b, fp8, 3, b_rows)) return TDX_ERR_CUDA;
  p.few_rows = std::min(kFewRows, p.M);
  if (form != TN && !map_of(&p.tm_few, a, fp8, 2, p.few_rows)) return TDX_ERR_CUDA;
  const int64_t out = static_cast<int64_t>(bytes_of(p.out_type));
  p.wide = aligned(p.out, 32) && p.ld_out * out % 32 == 0 && p.out_step * out % 32 == 0;
  p.wide_z = aligned(p.z, 32) && p.ld_z % 16 == 0 && (!p.gated || p.cols % 16 == 0);
  // a warp's columns of a tile (half of them) are whole 128-byte rows; strides as tensor maps take them
  p.tma_out = p.out_type != TDX_FP8_E4M3 && width / 2 * out >= 128 && p.ld_out * out < kMostBytes &&
              p.out_step * out < kMostBytes;
  const bool bare = p.bias == nullptr && p.z == nullptr && p.act == TDX_ACT_NONE;
  const bool approximate = p.act == TDX_ACT_RELU || p.act == TDX_ACT_GELU_TANH || p.act == TDX_ACT_SILU;
  p.steps = bare ? 0 : p.out_type != TDX_BF16 ? -1 : p.gated ? 2 : approximate ? 1 : -1;
  if (p.tma_out) {
    const uint64_t dims[3] = {static_cast<uint64_t>(p.cols), static_cast<uint64_t>(p.M),
                              static_cast<uint64_t>(group == kSums ? p.E : 1)};
    const uint64_t strides[2] = {static_cast<uint64_t>(p.ld_out * out),
                                 static_cast<uint64_t>((group == kSums && E > 1 ? p.out_step : p.ld_out) * out)};
    const uint32_t box[3] = {static_cast<uint32_t>(128 / out), 32, 1};
    if (!encode_map(&p.tm_c, p.out, p.out_type == TDX_FP32 ? 4 : 2, 3, dims, strides, box)) return TDX_ERR_CUDA;
  }
  // index: NN, NT, TN, NN of e4m3
  static LinLaunch* const launch[2][4] = {
      {launch_linear_nn, launch_linear_nt, launch_linear_tn, launch_linear_e4m3},
      {launch_linear_nn_long, launch_linear_nt_long, launch_linear_tn_long, launch_linear_e4m3_long}};
  // more slices in a tile than one segment, fp32; in a CTA's part of it, others (kSums: a run may have all rows)
  p.segment = p.out_type == TDX_FP32 ? kLinSegment : kLongSegment / bk;
  const int most_k = p.out_type == TDX_FP32 || group == kSums ? p.K : p.K / p.split;
  const bool longer = (most_k + bk - 1) / bk > p.segment;
  return launch[longer][fp8 ? 3 : form](group, shape.pair, p, static_cast<int>(most), st);
}

bool act_known(tdx_activation a) { return a >= TDX_ACT_NONE && a <= TDX_ACT_SWIGLU; }

// The forward product; E = 0: the linear layer, else grouped
tdx_status forward(const void* A, const int32_t* offsets, const void* B, const void* bias, const void* residual,
                   const float* row_scale, const float* expert_scale, void* C, void* z, int M, int K, int N, int E,
                   tdx_dtype dtype, const tdx_linear_opts* opts, void* stream) {
  const tdx_linear_opts o = opts ? *opts : linear_defaults();
  if (M < 0 || K <= 0 || N <= 0 || !known(dtype) || !known(o.out_dtype) || !act_known(o.act)) return TDX_ERR_INVALID_ARG;
  // tensors of M = 0 rows have no address
  if (B == nullptr || (M > 0 && (A == nullptr || C == nullptr)) || !std::isfinite(o.alpha) || !usable_scale(o.out_scale))
    return TDX_ERR_INVALID_ARG;
  const bool gated = o.act == TDX_ACT_SWIGLU, fp8 = dtype == TDX_FP8_E4M3;
  if (gated && N % 2 != 0) return TDX_ERR_INVALID_ARG;
  if (dtype == TDX_FP32 || M > kMostSize || K > kMostSize || N > kMostSize) return TDX_ERR_UNSUPPORTED;
  LinParams p;
  std::memset(&p, 0, sizeof(p));
  const int64_t cols = gated ? N / 2 : N, elt = fp8 ? 1 : 2, out = static_cast<int64_t>(bytes_of(o.out_dtype));
  int64_t ld_a, ld_b;
  tdx_status s;
  if ((s = stride_ok(o.ld_a, K, elt, &ld_a)) != TDX_OK || (s = stride_ok(o.ld_b, N, elt, &ld_b)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_c, cols, out, &p.ld_out)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_residual, cols, 2, &p.ld_res)) != TDX_OK) return s;
  if ((s = row_stride(o.ld_z, N, 2, &p.ld_z)) != TDX_OK) return s;
  if (K * elt % 16 != 0 || cols * elt % 16 != 0 || cols * 2 % 16 != 0 || cols * out % 16 != 0) return TDX_ERR_ALIGNMENT;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(bias, 16) || !aligned(residual, 16) ||
      !aligned(z, 16) || !aligned(row_scale, 4) || !aligned(expert_scale, 4) || !aligned(offsets, 4) ||
      !aligned(o.device_status, 4))
    return TDX_ERR_ALIGNMENT;
  int64_t step;
  if ((s = expert_step(E, K, ld_b, elt, &step)) != TDX_OK) return s;
  if (M == 0) return TDX_OK;
  p.M = M;
  p.K = K;
  p.cols = static_cast<int>(cols);
  p.E = E > 0 ? E : 1;
  p.offsets = offsets;
  p.gated = gated ? 1 : 0;
  p.act = o.act;
  p.out_type = o.out_dtype;
  p.alpha = o.alpha;
  p.inv_out_scale = 1.0f / o.out_scale;
  p.row_scale = row_scale;
  p.expert_scale = expert_scale;
  p.bias = static_cast<const bf16*>(bias);
  p.residual = static_cast<const bf16*>(residual);
  p.z = static_cast<bf16*>(z);
  p.out = C;
  p.status = o.device_status;
  return run(NN, E > 0 ? kRows : kFlat, fp8, p, {A, M, K, ld_a, 0, 1}, {B, K, N, ld_b, step, p.E},
             static_cast<cudaStream_t>(stream));
}

// Both gradients; E = 0: the linear layer, else grouped
tdx_status backward(const void* dz, const void* A, const int32_t* offsets, const void* B, const void* dres, void* dA,
                    void* dB, int M, int K, int N, int E, tdx_dtype dtype, const tdx_linear_opts* opts, void* stream) {
  const tdx_linear_opts o = opts ? *opts : linear_defaults();
  if (M < 0 || K <= 0 || N <= 0 || !known(dtype) || !known(o.out_dtype) || !known(o.dw_dtype) || !act_known(o.act))
    return TDX_ERR_INVALID_ARG;
  if ((dA != nullptr && B == nullptr) || o.act != TDX_ACT_NONE || !std::isfinite(o.alpha) || o.accumulate < 0 ||
      o.accumulate > 1)
    return TDX_ERR_INVALID_ARG;
  // tensors of M = 0 rows have no address
  if (M > 0 && (dz == nullptr || (dA == nullptr && dB == nullptr) || (dB != nullptr && A == nullptr) ||
                (dres != nullptr && dA == nullptr)))
    return TDX_ERR_INVALID_ARG;
  if (dtype != TDX_BF16 || o.out_dtype == TDX_FP8_E4M3 || o.dw_dtype == TDX_FP8_E4M3 || M > kMostSize ||
      K > kMostSize || N > kMostSize)
    return TDX_ERR_UNSUPPORTED;
  int64_t ld_a, ld_b, ld_z, ld_da, ld_res;
  tdx_status s;
  if ((s = stride_ok(o.ld_a, K, 2, &ld_a)) != TDX_OK || (s = stride_ok(o.ld_b, N, 2, &ld_b)) != TDX_OK ||
      (s = stride_ok(o.ld_z, N, 2, &ld_z)) != TDX_OK || (s = row_stride(o.ld_residual, K, 2, &ld_res)) != TDX_OK ||
      (s = row_stride(o.ld_c, K, bytes_of(o.out_dtype), &ld_da)) != TDX_OK)
    return s;
  if (K % 8 != 0 || N % 8 != 0) return TDX_ERR_ALIGNMENT;
  if (!aligned(dz, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(dres, 16) || !aligned(dA, 16) ||
      !aligned(dB, 16) || !aligned(offsets, 4) || !aligned(o.device_status, 4))
    return TDX_ERR_ALIGNMENT;
  int64_t step;
  if ((s = expert_step(E, K, ld_b, 2, &step)) != TDX_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LinParams p;
  std::memset(&p, 0, sizeof(p));
  p.E = E > 0 ? E : 1;
  p.offsets = offsets;
  p.act = TDX_ACT_NONE;
  p.alpha = o.alpha;
  p.inv_out_scale = 1.0f;
  p.status = o.device_status;
  const bool both = dA != nullptr && dB != nullptr && M > 0;
  if (dA != nullptr && M > 0) {
    LinParams q = p;
    q.overlap = both ? kOverlapFirst : kOverlapNone;
    q.M = M;
    q.cols = K;
    q.K = N;
    q.residual = static_cast<const bf16*>(dres);
    q.ld_res = ld_res;
    q.out = dA;
    q.ld_out = ld_da;
    q.out_type = o.out_dtype;
    if ((s = run(NT, E > 0 ? kRows : kFlat, false, q, {dz, M, N, ld_z, 0, 1}, {B, K, N, ld_b, step, p.E}, st)) != TDX_OK)
      return s;
  }
  if (dB != nullptr) {
    LinParams q = p;
    q.M = K;
    q.cols = N;
    q.K = M;
    q.out = dB;
    q.ld_out = ld_b;
    q.out_step = step;
    q.out_type = o.dw_dtype;
    q.accumulate = o.accumulate;
    q.overlap = both ? kOverlapSecond : kOverlapNone;
    // without rows nothing is loaded; the maps want an address all the same
    const void* rows_a = M > 0 ? A : dB;
    const void* rows_z = M > 0 ? dz : dB;
    return run(TN, E > 0 ? kSums : kFlat, false, q, {rows_a, M, K, ld_a, 0, 1}, {rows_z, M, N, ld_z, 0, 1}, st);
  }
  return TDX_OK;
}

}  // namespace
}  // namespace tdx

using namespace tdx;

extern "C" {

tdx_status tdx_linear_opts_default(tdx_linear_opts* opts) {
  if (opts == nullptr) return TDX_ERR_INVALID_ARG;
  *opts = linear_defaults();
  return TDX_OK;
}

tdx_status tdx_linear(const void* A, const void* B, const void* bias, const void* residual, const float* row_scale,
                      void* C, void* z, int M, int K, int N, tdx_dtype dtype, const tdx_linear_opts* opts,
                      void* stream) {
  return forward(A, nullptr, B, bias, residual, row_scale, nullptr, C, z, M, K, N, 0, dtype, opts, stream);
}

tdx_status tdx_linear_bwd(const void* dz, const void* A, const void* B, const void* dres, void* dA, void* dB, int M,
                          int K, int N, tdx_dtype dtype, const tdx_linear_opts* opts, void* stream) {
  return backward(dz, A, nullptr, B, dres, dA, dB, M, K, N, 0, dtype, opts, stream);
}

tdx_status tdx_grouped_gemm(const void* X, const int32_t* offsets, const void* B, const float* row_scale,
                            const float* expert_scale, void* Y, void* z, int R, int K, int N, int E, tdx_dtype dtype,
                            const tdx_linear_opts* opts, void* stream) {
  if (E <= 0 || offsets == nullptr) return TDX_ERR_INVALID_ARG;
  if (E > kMoeMaxExperts) return TDX_ERR_UNSUPPORTED;
  return forward(X, offsets, B, nullptr, nullptr, row_scale, expert_scale, Y, z, R, K, N, E, dtype, opts, stream);
}

tdx_status tdx_grouped_gemm_bwd(const void* dY, const void* X, const int32_t* offsets, const void* B, void* dX,
                                void* dB, int R, int K, int N, int E, tdx_dtype dtype, const tdx_linear_opts* opts,
                                void* stream) {
  if (E <= 0 || offsets == nullptr) return TDX_ERR_INVALID_ARG;
  if (E > kMoeMaxExperts) return TDX_ERR_UNSUPPORTED;
  return backward(dY, X, offsets, B, nullptr, dX, dB, R, K, N, E, dtype, opts, stream);
}

}  // extern "C"
