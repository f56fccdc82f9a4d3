// Shared by the product kernel's instances and their host side.
#pragma once

#include <cuda_bf16.h>

#include "../../include/tdx.h"
#include "tdx_internal.h"

namespace tdx {

enum Form { NN, NT, TN };                 // see tdx_linear.cuh
enum Group { kFlat, kRows, kSums };
// A tile's sum over K: on the tensor cores alone; in segments of kLinSegment slices, for fp32 results; in segments of
// kLongSegment of K, for others
enum Sum { kOnce, kSegments, kLongSegments };
// Longest waits: for a slice, a sum or an epilogue; and for a tail, which waits for the tiles in front of its own
constexpr uint64_t kLinTimeoutNs = 4000000000ull, kLinTailTimeoutNs = 60000000000ull;
constexpr int kLinSegment = 14, kLongSegment = 65536;
constexpr int kMostSplit = 8;    // CTAs of a cluster that share a tile, the portable limit
constexpr int kFewRows = 16;   // most rows of the small boxes of A

// Tile columns: pairs 256. Single CTAs 128, and 256 for e4m3, whose 128-column boxes would not split
// a 128-column tile into gate and up halves.
constexpr int lin_block_n(bool fp8, bool pair) { return pair || fp8 ? 256 : 128; }
constexpr int lin_tile_rows(bool pair) { return pair ? 2 * kBM : kBM; }

// Two products of one call that read nothing of each other's: the first lets the second be launched as soon as it has
// itself waited for the stream's earlier work, so the second, which then need not wait for anything, takes the SMs
// that the first leaves idle; before it ends it waits for the first, so that what follows in the stream
// waits for both.
enum Overlap { kOverlapNone, kOverlapFirst, kOverlapSecond };

struct LinParams {
  CUtensorMap tm_a, tm_b;   // operands
  CUtensorMap tm_few;       // A in boxes of few rows
  CUtensorMap tm_c;         // output in boxes of 32 rows of 128 bytes
  int M, K;                 // output rows, summed length (kRows: M, kSums: K over all runs)
  int cols;                 // output columns: those of the product, or half of them for SWIGLU
  int E;
  const int32_t* offsets;
  int tiles_m, tiles_n, items, group_n;
  int few_rows;             // rows of tm_few's boxes: kFewRows, or all rows of a smaller A
  int split;                // CTAs that share a tile's K slices (single CTAs)
  int segment;              // K slices of a segment
  int keep_a, keep_b;       // L2 policies of the operands' loads (policy_of)
  int gated;                // act == TDX_ACT_SWIGLU
  tdx_activation act;
  tdx_dtype out_type;
  int accumulate;
  float alpha, inv_out_scale;
  const float* row_scale;
  const float* expert_scale;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* z;
  void* out;
  int64_t ld_out, ld_res, ld_z;
  int64_t out_step;         // kSums: elements between two experts' outputs
  int tma_out;              // output through tm_c (bf16 or fp32; whole 128-byte columns per warp)
  int wide, wide_z;         // output and z in 32-byte stores: 32-byte aligned rows
  int steps;                // a short epilogue's (lin_short) where tma_out is set: 0, 1, 2, or -1 for none
  int overlap;
  uint32_t* status;
};

// Instances by operand type, form and group; each form's in a file of its own, those that add segments in another. `want`: clusters of work.
using LinLaunch = tdx_status(Group g, bool pair, const LinParams& p, int want, cudaStream_t stream);
LinLaunch launch_linear_nn, launch_linear_nt, launch_linear_tn, launch_linear_e4m3;
LinLaunch launch_linear_nn_long, launch_linear_nt_long, launch_linear_tn_long, launch_linear_e4m3_long;

// Clusters of `split` single CTAs (2 .. kMostSplit) that are resident together on the current device
int lin_clusters(int split);

}  // namespace tdx
