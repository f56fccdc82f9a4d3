/*
 * tdx.h -- C ABI of the tile-pipelined collective+GEMM library (sm_103a): AllGather+GEMM,
 * GEMM+ReduceScatter, GEMM+AllReduce, the mixture-of-experts AllToAll dispatch + grouped GEMM and
 * grouped GEMM + combine, the row-wise operators around these products (root-mean-square norm,
 * routing to experts, gated SiLU, with their gradients), and the products that need no communication:
 * the linear layer, the products grouped by expert and the sum of a token's expert rows, with their
 * gradients.
 *
 * What the operations are. The Triton-distributed article on cronfeed.work ("Triton-distributed
 * is turning communication into compiler territory"), section "The first move was to expose the
 * overlap", describes an AllGather that moves row shards into place feeding a GEMM, split into
 * chunks so that the GEMM computes on one chunk while another is still moving, and the mirror
 * operation GEMM-plus-ReduceScatter; communication and computation thread blocks of one kernel
 * are coordinated through symmetric memory and signals. Section "DITRON adds three levels of
 * tiling" adds that collectives such as AllGather and ReduceScatter are broken into chunks, paired
 * with compute tiles, and synchronised (AllToAll and AllReduce among them; the AllToAll entry
 * points are further down). This library implements these kernels for one GPU: the W ranks are
 * logical, i.e. W shard buffers (W partial products for ReduceScatter / AllReduce, W token sets
 * for the AllToAll) in one device's memory; the "network" is a chunk producer that copies shard
 * chunks into a symmetric gathered buffer and releases one flag per chunk, and the GEMM tiles
 * acquire those flags before they read a chunk.
 *
 * Conventions for every entry point:
 *  - Ownership: every tensor and the workspace are device memory owned by the caller. The library
 *    allocates nothing per call and keeps no pointer after a call returns.
 *  - Layout: all matrices are dense and row-major with no padding (row pitch = columns * element
 *    size). Each row pitch must be a multiple of 16 bytes and each pointer 16-byte aligned.
 *  - Asynchrony: calls are stream-ordered on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and return before the work runs. The returned status covers host-side validation and
 *    launch errors only. Errors found on the device (a bounded wait that timed out, a stale epoch)
 *    are recorded in the workspace's status word; read them with tdx_read_device_status. Kernels
 *    never trap: a failed wait makes the kernel stop issuing work, drain what it started and exit.
 *  - Threading: a workspace is used by one call at a time (calls that overlap on the GPU and share a
 *    workspace race). Different workspaces may be used concurrently.
 *  - A tensor without elements may be NULL, as an empty tensor's address is.
 *  - No fallback: shapes the kernels cannot tile return TDX_ERR_UNSUPPORTED; nothing runs on the CPU.
 */
#ifndef TDX_H_
#define TDX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TDX_OK = 0,
  TDX_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, W out of range, bad enum */
  TDX_ERR_UNSUPPORTED = 2,   /* valid request the kernels do not implement (dtype combination, tiling) */
  TDX_ERR_ALIGNMENT = 3,     /* pointer not 16-byte aligned or row pitch not a multiple of 16 bytes */
  TDX_ERR_WORKSPACE = 4,     /* workspace null, misaligned (256 B) or smaller than tdx_workspace_size */
  TDX_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed (launch, tensor map, memset) */
  TDX_ERR_TIMEOUT = 6,       /* device: a bounded wait on a flag or pipeline barrier ran out */
  TDX_ERR_STALE_EPOCH = 7    /* device: a flag already held an epoch >= the call's epoch */
} tdx_status;

typedef enum { TDX_BF16 = 0, TDX_FP8_E4M3 = 1, TDX_FP32 = 2 } tdx_dtype;

/* tdx_opts.epoch value selecting epochs kept on the device (see tdx_opts). */
#define TDX_EPOCH_DEVICE 0xFFFFFFFFu

typedef enum {
  TDX_FUSED = 0,          /* producer and consumer overlapped in one persistent kernel (default) */
  TDX_GEMM_ONLY = 1,      /* AG: GEMM on an already gathered buffer, no flag waits, no copies.
                             RS: every rank's partial tile computed and read out of Tensor Memory,
                             no partial buffer, no rank chain; only rank W-1's partial is stored,
                             rounded to bf16, into the output (the GEMM alone, for measurements) */
  TDX_MOVE_ONLY = 2,      /* AG: chunk copies and flag releases only. RS: the rank-order
                             read-add-write chain over the running-sum buffer with zero partials */
  TDX_CONSUMER_ONLY = 3   /* AG: consumers wait on flags that no producer releases (fault tests) */
} tdx_mode;

typedef enum {
  TDX_PRODUCER_SM = 0,          /* chunk copies by producer warps of the persistent kernel */
  TDX_PRODUCER_COPY_ENGINE = 1  /* not offered (TDX_ERR_UNSUPPORTED): copies issued outside the kernel
                                   that its consumers wait on need not run while it holds every SM */
} tdx_producer;

/* Per-call options. Pass NULL for all defaults; tdx_opts_default fills the same values. */
typedef struct tdx_opts {
  int self_rank;             /* AG: rank whose shard is local; arrival order self, self+1, ... (default 0) */
  int chunk_rows;            /* AG: rows per chunk and per flag; must divide M_local (default min(128, M_local)) */
  tdx_dtype out_dtype;       /* AG: TDX_BF16 (default) or TDX_FP32. RS: TDX_BF16 only */
  const float* scale_a;      /* host array [W]: per-shard (AG) / per-A_r (RS) / per source rank (MoE)
                                e4m3 dequantisation scales (NULL = 1) */
  const float* scale_b;      /* host array: AG [1] B's scale; RS [W] the B_r scales; MoE [E] the
                                experts' scales; e4m3 only (NULL = 1) */
  tdx_mode mode;             /* default TDX_FUSED */
  tdx_producer producer;     /* default TDX_PRODUCER_SM */
  uint32_t epoch;            /* 0: the library clears the flags on `stream` and uses epoch 1.
                                >0: flags are not cleared; the caller passes strictly increasing
                                epochs on one workspace (after tdx_workspace_init).
                                TDX_EPOCH_DEVICE: the epochs are kept in the workspace itself: a
                                call uses the epoch of the last completed call on that workspace
                                plus one and stores it when its kernel finishes. Nothing is cleared
                                and the host tracks nothing, so the same captured call replays
                                correctly in a CUDA graph. Start from a workspace zeroed by
                                tdx_workspace_init, and do not mix with caller epochs on one
                                workspace without re-initialising it (a flag left at a higher
                                epoch is reported as TDX_ERR_STALE_EPOCH). */
  uint64_t timeout_ns;       /* bound of every device-side wait (default 2e9 ns) */
  uint32_t perturb_seed;     /* test only: !=0 injects pseudo-random delays in producers/epilogues */
  void* trace;               /* optional device buffer of tdx_trace_size() bytes, or NULL */
  int num_sms;               /* largest persistent grid; 0 = every SM of the device (a plan with a
                                grid-wide fold takes as many CTAs as give each the same number of
                                work items; small AllGathers split K to fill this many CTAs) */
  int split_k;               /* AG: K splits reduced in fixed order (0 = library choice, 1 = none) */
  int block_n;               /* GEMM tile width 64/128/256, or 512 on 2-SM pairs (cluster 3; one
                                512-column accumulator per CTA, two MMAs per K step; bf16 and e4m3
                                AllGather / ReduceScatter / AllReduce). 0 = library choice */
  int reduce_mode;           /* fixed-order reduction of RS ranks / AG K splits: 0 = library choice,
                                1 = chained (element c adds its partial to the running sum of
                                elements 0..c-1 and hands it on), 2 = slotted (each element stores its
                                partial; the last to arrive folds them in order 0..L-1), 3 = slotted
                                with a grid-wide fold (once every CTA has stored its partials, all
                                CTAs fold 1/grid of every tile each, slots in order 0..L-1; single
                                CTAs and fp32 partials only). All give the same bits. */
  int cluster;               /* how CTAs cooperate on the GEMM: 0 = library choice, 1 = single CTAs,
                                3 = pairs running one 2-SM MMA stream on a 256 x 256 tile (each CTA
                                stages its 128 rows of A and half of B in its own shared memory;
                                needs tile width 256 and an even number of 128-row M-tiles).
                                2 (pairs sharing B through multicast loads) is not offered:
                                TDX_ERR_UNSUPPORTED. */
  int bf16_partials;         /* ReduceScatter / AllReduce: 0 (default) = each rank's partial enters
                                the fold in fp32; 1 = each partial is rounded once to bf16 (RNE, the
                                type a rank would send) before the fp32 fold, which halves the
                                partial-slot traffic. Needs the slotted reduction (reduce_mode 0 or 2);
                                AllGather: must be 0. */
} tdx_opts;

/* Fill *opts with the defaults above. Returns TDX_ERR_INVALID_ARG if opts is NULL. */
tdx_status tdx_opts_default(tdx_opts* opts);

/* Bytes of workspace needed by one call. op = 0: AllGather+GEMM (M_local_or_M = rows per shard);
 * op = 1: GEMM+ReduceScatter, op = 2: GEMM+AllReduce (M_local_or_M = rows of every A_r). The workspace holds the status
 * word, the chunk flags, the symmetric gathered buffer G (AG, (W*M_local) x K of `dtype`) and the
 * fp32 running-sum buffer with its rank-chain flags (RS, and AG with split K). Writes *bytes.
 * After a call the running-sum region holds the last call's fp32 sums (chained: ranks/splits
 * 0..L-2 of every tile) or partials (slotted: one slot per rank/split). */
tdx_status tdx_workspace_size(int op, int W, int M_local_or_M, int K, int N, tdx_dtype dtype,
                              const tdx_opts* opts, size_t* bytes);

/* Zero the control region of a workspace (status word, flags, counters) on `stream`. Call once
 * after allocating a workspace, and again after a call reported a device-side error. */
tdx_status tdx_workspace_init(void* workspace, size_t bytes, void* stream);

/* AllGather+GEMM: C = concat_r(shards[r]) @ B, the shards gathered in rank order 0..W-1.
 * (Triton-distributed article, section "The first move was to expose the overlap": the AllGather
 * moves shards into place, split into chunks, and the GEMM consumes each chunk once it has arrived.)
 *  shards     host array of W device pointers; shards[r] is M_local x K of `dtype`, row-major.
 *             Any addresses; shards at one stride (shards[r] = shards[0] + r * pitch, as in a
 *             symmetric heap) let tiles of small shards read them with fewer, larger loads (a
 *             performance difference only).
 *  B          device, K x N of `dtype`, row-major.
 *  C          device, (W*M_local) x N, row-major, of opts->out_dtype (bf16 or fp32). Row
 *             r*M_local + i of C is row i of shards[r] times B, whatever the arrival order.
 *  workspace  device, 256-byte aligned, workspace_bytes >= tdx_workspace_size(0, ...) with the
 *             same shapes and opts (else TDX_ERR_WORKSPACE). After the call its gathered buffer
 *             holds concat_r(shards[r]) and every chunk flag holds the epoch.
 *  W          logical ranks, 1..16. M_local, K, N >= 0 (M_local or N == 0: nothing is launched;
 *             K == 0: C is filled with zeros).
 *  dtype      TDX_BF16, or TDX_FP8_E4M3 with per-tensor scales: C = scale_a[r]*scale_b*(shard @ B).
 * Accumulation is fp32 on the tensor cores; the output is rounded once, to nearest even. */
tdx_status tdx_ag_gemm(const void* const* shards, const void* B, void* C, void* workspace,
                       size_t workspace_bytes, int W, int M_local, int K, int N, tdx_dtype dtype,
                       const tdx_opts* opts, void* stream);

/* GEMM+ReduceScatter: S = sum_{r=0}^{W-1} A_parts[r] @ B_parts[r], out_shards[j] = rows
 * [j*M/W, (j+1)*M/W) of S. (Same article and section: "GEMM-plus-ReduceScatter"; section "DITRON
 * adds three levels of tiling" lists ReduceScatter among the collectives split into chunks.)
 *  A_parts    host array of W device pointers, each M x K of `dtype`, row-major.
 *  B_parts    host array of W device pointers, each K x N of `dtype`, row-major.
 *  out_shards host array of W device pointers, each (M/W) x N bf16 row-major.
 *  workspace  device, 256-byte aligned, workspace_bytes >= tdx_workspace_size(1, ...) with the
 *             same shapes and opts (else TDX_ERR_WORKSPACE).
 *  W          1..16, and M must be a multiple of W.
 *  dtype      TDX_BF16, or TDX_FP8_E4M3 with per-rank scales: P_r = scale_a[r]*scale_b[r]*(A_r @ B_r).
 * Rank r's fp32 partial tile is added to the running sum of ranks 0..r-1 in that fixed order,
 * ((P_0 + P_1) + P_2) + ..., whatever the timing, so the result is identical run to run; the sum
 * is rounded once to bf16 (nearest even). */
tdx_status tdx_gemm_rs(const void* const* A_parts, const void* const* B_parts,
                       void* const* out_shards, void* workspace, size_t workspace_bytes,
                       int W, int M, int K, int N, tdx_dtype dtype,
                       const tdx_opts* opts, void* stream);

/* Size of the library's built-in scratch array used by tdx_ag_gemm_noalloc: 16 MiB per device. */
#define TDX_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

/* AllGather+GEMM for callers that cannot allocate device memory themselves: for example code that
 * runs inside a host framework which owns every device allocation and exposes no allocator to it
 * (a plugin of an inference runtime with a fixed memory budget), or a latency-critical caller that
 * cannot accept the device-wide synchronisation cudaMalloc may cause. The pages have no
 * counterpart of this entry point; it is a convenience of this library.
 *
 * Computes exactly what tdx_ag_gemm computes (same shards, B, C, W, M_local, K, N, dtype and opts
 * meaning), but instead of a caller-owned workspace it uses a scratch array that the library
 * declares statically in device memory: TDX_NOALLOC_SCRATCH_BYTES on every GPU that loads the
 * library, held until the process exits. The call itself allocates nothing (no cudaMalloc, no
 * cudaFree, no allocating library routine).
 *  - Limit: problems whose tdx_workspace_size(0, W, M_local, K, N, dtype, opts) exceeds
 *    TDX_NOALLOC_SCRATCH_BYTES are rejected with TDX_ERR_WORKSPACE before anything is launched
 *    (the small-M and tiny AllGather shapes fit; W=8 x 1024 x 8192 bf16 does not).
 *  - First call on a device: it looks up the device address of the scratch array (with that
 *    device current) and caches it with the ID of the current CUDA context; make this first call
 *    before any stream capture. The cached address belongs to that context: after the device's
 *    context is destroyed and re-created (for example by cudaDeviceReset), the next call looks the
 *    address up again, and that call too should come before any stream capture.
 *  - Every argument is checked before anything is enqueued: a call that returns an error has
 *    launched nothing and left the scratch array untouched.
 *  - Shared state: every call on a device uses the same array, which keeps the previous call's
 *    contents. Each call clears, on `stream`, the status word and the flags that must start at
 *    zero (opts->epoch is ignored; epoch 1 is used). Calls that overlap on the GPU (different
 *    streams, or different host threads) race on the array: serialise them.
 *  - opts->producer must be TDX_PRODUCER_SM (else TDX_ERR_UNSUPPORTED).
 *  - device_status: optional device pointer to 8 uint32 words. If not NULL, the call copies the
 *    scratch's status word and details (see tdx_read_device_status) there on `stream` once the
 *    kernel has finished; if NULL, device-side errors of this call are not reported. */
tdx_status tdx_ag_gemm_noalloc(const void* const* shards, const void* B, void* C,
                               int W, int M_local, int K, int N, tdx_dtype dtype,
                               const tdx_opts* opts, uint32_t* device_status, void* stream);

/* GEMM+AllReduce: every rank r receives the whole S = sum_{r'} A_parts[r'] @ B_parts[r'] in
 * out_full[r]. (Triton-distributed article, section "DITRON adds three levels of tiling": AllReduce is
 * among the collectives broken into chunks and paired with compute tiles.) Realised as the chunked
 * ReduceScatter above fused with an AllGather: the element that completes a tile's fixed-order fold
 * ((P_0 + P_1) + ...) rounds the tile once to bf16 and writes it into every rank's output, so all W
 * outputs are bit-identical.
 *  A_parts, B_parts, workspace, dtype, scales: as tdx_gemm_rs (workspace sized with op = 2).
 *  out_full   host array of W device pointers, each M x N bf16 row-major. M need not be a multiple
 *             of W. */
tdx_status tdx_gemm_ar(const void* const* A_parts, const void* const* B_parts, void* const* out_full,
                       void* workspace, size_t workspace_bytes, int W, int M, int K, int N, tdx_dtype dtype,
                       const tdx_opts* opts, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Mixture-of-experts AllToAll dispatch + grouped GEMM.
 * (Triton-distributed article, section "DITRON adds three levels of tiling": AllToAll is among the
 * collectives broken into chunks and paired with compute tiles; the tokens routed to each expert of
 * a mixture-of-experts model are known only at run time, so its device-level tiles are sized
 * dynamically.)
 *
 * W ranks; rank s holds T tokens X[s] (T x H of `dtype`, row-major) and their routing topk_idx[s]
 * (T x topk int32 expert ids in [0, E)). Rank rho owns experts rho*E/W .. (rho+1)*E/W - 1. The
 * dispatch sends every (s, t, j) row X[s][t] to expert topk_idx[s][t][j]; the receive side (one
 * buffer for all ranks, in the workspace) groups the W*T*topk rows by expert, experts ascending,
 * and inside an expert by source rank then token, ascending. Expert e's rows are multiplied by its
 * weights B_experts[e] (H x F); Y keeps the dispatched row order:
 *   Y[dest[s][t][j]] = round_bf16(X[s][t] @ B_experts[topk_idx[s][t][j]]),
 * for e4m3 inputs multiplied first by scale_a[s] * scale_b[e] (fp32, in the epilogue).
 * The layout (counts, offsets, row of every pair, GEMM tile table) is computed on the device; the
 * dispatch copies the receive buffer in 128-row chunks, each released by a flag, while the GEMM
 * tiles of the experts whose rows have arrived already run.
 *  X              host array of W device pointers, each T x H of `dtype` (16-byte aligned).
 *  topk_idx       host array of W device pointers, each T x topk int32. Ids outside [0, E) make the
 *                 call do nothing further and record TDX_ERR_INVALID_ARG in the device status.
 *  B_experts      device pointer, E x H x F of `dtype` (expert e's weights at e*H*F).
 *  Y              device pointer, (W*T*topk) x F bf16 (for either input type), the dispatched order.
 *  dest           device pointer, W x T x topk int32 (output): the row of Y of every (s, t, j).
 *  expert_offsets optional device pointer, E + 1 int32 (output): expert e's rows are
 *                 [expert_offsets[e], expert_offsets[e+1]).
 *  workspace      caller-owned device memory of tdx_moe_workspace_size() bytes, 256-byte aligned,
 *                 zeroed once by tdx_workspace_init; it holds the status word, chunk flags, the
 *                 layout tables and the receive buffer ((W*T*topk) x H of `dtype`).
 *  dtype          TDX_BF16, or TDX_FP8_E4M3 with per-tensor scales: opts->scale_a host array [W]
 *                 (one per source rank's tokens), opts->scale_b host array [E] (one per expert's
 *                 weights); NULL = 1. e4m3 needs tile width 128 or 256.
 *  H and F rows of 16-byte multiples (bf16: multiples of 8; e4m3: H and F multiples of 16);
 *  1 <= topk <= E <= 512; W <= 16.
 *  opts: epoch, timeout_ns, perturb_seed, trace, num_sms, block_n and mode (TDX_FUSED, TDX_GEMM_ONLY:
 *  the receive buffer is assumed filled by an earlier call with the same routing, TDX_MOVE_ONLY:
 *  dispatch only) apply; other cooperation options must keep their defaults. */
tdx_status tdx_moe_workspace_size(int W, int T, int H, int F, int E, int topk, tdx_dtype dtype,
                                  const tdx_opts* opts, size_t* bytes);
tdx_status tdx_moe_dispatch_gemm(const void* const* X, const int32_t* const* topk_idx, const void* B_experts,
                                 void* Y, int32_t* dest, int32_t* expert_offsets, void* workspace,
                                 size_t workspace_bytes, int W, int T, int H, int F, int E, int topk,
                                 tdx_dtype dtype, const tdx_opts* opts, void* stream);
/* Plan of one MoE call (16 words to info): [0] tile width, [1] N-tiles, [2] tile-table capacity,
 * [3] 128-row chunks of the dispatched rows (one flag each), [4] dispatched rows W*T*topk, byte
 * offsets in the workspace of [5] chunk flags (uint32 per chunk), [6] tile count + invalid-routing
 * words, [7] expert offsets (int32 [E+1]), [8] source of every dispatched row (int32, s*T + t),
 * [9] tile table (int32x4 {first row, end row of the expert, expert, 0}), [10] receive buffer
 * (dispatch) / expert outputs Z (combine, (W*T*topk) x H bf16 in dispatched order), [11] total
 * workspace bytes, [12] 128-byte K blocks, [13] per-(token, N-tile) arrival counters (combine; 0
 * for the dispatch), [14] dispatched row of every token slot (combine, int32 W x T x topk; 0),
 * [15] CTA cooperation in use: 1 single CTAs, 3 2-SM pairs on two 128-row tiles of one expert
 * (chosen by default for tile width 256 when the experts average at least 8 tiles; the tile table
 * then pads every expert to an even count with an empty tile). opts.cluster: 0 library choice,
 * 1 single, 3 pairs (2: TDX_ERR_UNSUPPORTED). */
tdx_status tdx_moe_plan_info(int W, int T, int H, int F, int E, int topk, tdx_dtype dtype,
                             const tdx_opts* opts, int64_t* info);

/* ---------------------------------------------------------------------------------------------
 * Mixture-of-experts grouped GEMM + AllToAll combine (the reverse of the dispatch above; same
 * article section: AllToAll is chunked and paired with compute tiles).
 *
 * Hd holds the dispatched rows ((W*T*topk) x F bf16) in the order tdx_moe_dispatch_gemm lays out
 * for the same routing topk_idx (grouped by expert, then source rank, then token). Expert e's rows
 * are multiplied by B_experts[e] (F x H) into expert outputs Z, rounded once to bf16 (the type a
 * rank sends back), kept in the workspace in dispatched order; then every token is combined on its
 * source rank with its gates:
 *   out[s][t] = round_bf16( sum_{j=0}^{topk-1} gates[s][t][j] * Z[row of (s, t, j)] ),
 * the sum in slot order j (fp32 fused multiply-adds). A token's combine runs as soon as the tiles
 * holding all its rows are stored (an arrival counter per (token, N-tile); the last arriver folds),
 * so the combine overlaps the GEMM and the result does not depend on timing.
 *  Hd         device pointer, (W*T*topk) x F bf16 (16-byte aligned).
 *  topk_idx   host array of W device pointers, each T x topk int32 expert ids in [0, E).
 *  B_experts  device pointer, E x F x H bf16.
 *  gates      host array of W device pointers, each T x topk fp32.
 *  out        host array of W device pointers, each T x H bf16 (output).
 *  workspace  tdx_moe_combine_workspace_size() bytes, 256-byte aligned, zeroed once by
 *             tdx_workspace_init (layout tables, counters, Z).
 *  F, H multiples of 8; topk <= 16; 1 <= topk <= E <= 512; bf16 only. opts.mode: TDX_FUSED,
 *  TDX_GEMM_ONLY (Z only, no combine), TDX_MOVE_ONLY (combine only, from the Z of an earlier
 *  call with the same routing). */
tdx_status tdx_moe_combine_workspace_size(int W, int T, int F, int H, int E, int topk, tdx_dtype dtype,
                                          const tdx_opts* opts, size_t* bytes);
tdx_status tdx_moe_gemm_combine(const void* Hd, const int32_t* const* topk_idx, const void* B_experts,
                                const float* const* gates, void* const* out, void* workspace,
                                size_t workspace_bytes, int W, int T, int F, int H, int E, int topk,
                                tdx_dtype dtype, const tdx_opts* opts, void* stream);
/* Plan of one combine call: the 16 words of tdx_moe_plan_info, [10] = Z, [13] and [14] set. */
tdx_status tdx_moe_combine_plan_info(int W, int T, int F, int H, int E, int topk, tdx_dtype dtype,
                                     const tdx_opts* opts, int64_t* info);

/* ---------------------------------------------------------------------------------------------
 * The row-wise operators around the products: root-mean-square norm, routing to experts, gated
 * SiLU, each with its gradient. They read one tensor per operand; W ranks whose tensors lie in one
 * buffer, rank after rank, are one call on W*T rows. All arithmetic is fp32, with the approximate
 * functions that each operator names; every output is rounded once (RNE; e4m3 saturates at +-448).
 * e4m3 codes are those of the value times its scale's fp32 reciprocal, not of an exact quotient: a
 * value within the arithmetic's own rounding of the middle between two codes may take either.
 * Except tdx_rmsnorm_bwd they need no workspace, and they record nothing in a device status word: ids
 * and indexes read on the device are bounds-checked there. Rows of 0 elements are invalid; 0 rows
 * launch nothing (tdx_rmsnorm_bwd still zeroes dweight), and their tensors may be NULL. Row strides are
 * in elements, 0 = dense; a stride below the row's length is TDX_ERR_INVALID_ARG. Unless said otherwise
 * pointers are 16-byte aligned and rows and strides are multiples of 16 bytes (TDX_ERR_ALIGNMENT).
 *
 * Root-mean-square norm of x + residual:
 *   h = x + residual (x alone if residual is NULL), rstd = 1 / sqrt(mean(h^2) + eps),
 *   y = h * rstd * weight; the sum h is normalised before it is rounded to `dtype` for h_out. The
 *   inverse root is rsqrtf (2 ulp).
 *  x, residual, h_out  device, T x H of `dtype` (TDX_BF16 or TDX_FP32). residual optional; h_out (the
 *             residual stream for the next layer) optional, only with residual. h_out may be x or
 *             residual itself (same stride); otherwise outputs overlap no input.
 *  weight     device, H of `dtype`.
 *  y          device, T x H of opts->out_dtype (TDX_BF16, TDX_FP32 or TDX_FP8_E4M3).
 *  row_scale  device, T fp32 (4-byte aligned), e4m3 output only: row t is stored as
 *             y[t] / row_scale[t] with row_scale[t] = max|y[t]| / 448 (1 if that is 0 or NaN). NULL: e4m3
 *             output is y / opts->out_scale, one scale per tensor as the e4m3 products take it.
 *  rstd       optional, T fp32 (4-byte aligned), for tdx_rmsnorm_bwd.
 * A row holding a NaN or an infinity gives the NaNs the formula gives; others are not touched.
 * H <= 2^28 (TDX_ERR_UNSUPPORTED beyond). */
typedef struct tdx_norm_opts {
  tdx_dtype out_dtype;       /* default TDX_BF16 */
  float eps;                 /* default 1e-6; finite, >= 0 */
  float out_scale;           /* default 1; positive and finite, as its reciprocal */
  int64_t ld_x, ld_residual, ld_h, ld_y;   /* row strides (tdx_rmsnorm_bwd: ld_x of dy, ld_residual
                                of dres, ld_h of h, ld_y of dx) */
} tdx_norm_opts;
tdx_status tdx_norm_opts_default(tdx_norm_opts* opts);
tdx_status tdx_rmsnorm(const void* x, const void* residual, const void* weight, void* h_out, void* y,
                       float* row_scale, float* rstd, int T, int H, tdx_dtype dtype,
                       const tdx_norm_opts* opts, void* stream);

/* Its gradient: with g = dy * weight and n = h * rstd,
 *   dx = rstd * (g - n * mean(g * n)) + dres,   dweight = sum_t dy[t] * n[t].
 * dx is the gradient of x and of residual alike; dres (optional) is the one that reaches h_out.
 *  dy, h, dres, dx  device, T x H of `dtype`; dx may be dy or dres itself (same stride).
 *  rstd       device, T fp32, as the forward call left it.
 *  dweight    device, H fp32 (16-byte aligned), overwritten. Partial sums over rows are added in a
 *             fixed order: the bits do not change from call to call.
 *  workspace  tdx_rmsnorm_bwd_workspace_size() bytes, 256-byte aligned; needs no initialisation.
 * H <= 32768 (TDX_ERR_UNSUPPORTED beyond). */
tdx_status tdx_rmsnorm_bwd_workspace_size(int T, int H, tdx_dtype dtype, size_t* bytes);
tdx_status tdx_rmsnorm_bwd(const void* dy, const void* h, const void* weight, const float* rstd,
                           const void* dres, void* dx, float* dweight, void* workspace,
                           size_t workspace_bytes, int T, int H, tdx_dtype dtype,
                           const tdx_norm_opts* opts, void* stream);

/* Routing of T tokens to topk of E experts, in the layout tdx_moe_dispatch_gemm and
 * tdx_moe_gemm_combine read (T x topk int32 ids, T x topk fp32 gates).
 *   score s = softmax(x) over the E logits of a row, or sigmoid(x) = 1 / (1 + exp(-x));
 *   key = s + bias (the bias steers the choice only and has no gradient); softmax without a bias
 *   compares the logits themselves, whose order is the same.
 *   Groups: E / n_group consecutive experts form a group; its score is the largest key
 *   (group_top 1) or the sum of the two largest (group_top 2; softmax without a bias: of
 *   exp(x - max)); only the experts of the topk_group best groups remain.
 *   The topk largest keys are taken in descending order; equal keys (and groups) go to the lowest
 *   index; a NaN key comes after every other.
 *   gate_j = scale * s_j / (renorm ? sum of the chosen s : 1), 0 where that sum is 0 or, with softmax
 *   scores, the logits it runs over are all -inf. With softmax scores a NaN or a +inf among a row's logits
 *   makes all its gates NaN, chosen or not; with sigmoid scores a NaN shows where it enters.
 * Gates, and the gradient's softmax, take approximate exponentials and quotients: within
 * 2^-24 * (64 + E / 16 + 2 d) of their values, d the spread of the row's logits.
 * Every step up to the keys rounds to fp32 as written, so ids do not depend on the kernel (but for the
 * order in which the sum of softmax scores with a bias is taken).
 *  logits     device, T x E of `dtype` (TDX_BF16 or TDX_FP32), aligned to the element, any stride.
 *  bias       optional, E fp32 (4-byte aligned).
 *  topk_idx   device, T x topk int32 (4-byte aligned); gates: T x topk fp32 (4-byte aligned).
 *  counts     optional, E int32 (4-byte aligned): the number of tokens sent to each expert is ADDED
 *             (for balancing the bias over the calls of a step; clear it when the step begins).
 *  1 <= topk <= 16, topk <= topk_group * (E / n_group), E <= 512, n_group <= 32 dividing E. */
typedef enum { TDX_SCORE_SOFTMAX = 0, TDX_SCORE_SIGMOID = 1 } tdx_score;
typedef struct tdx_route_opts {
  tdx_score score;           /* default TDX_SCORE_SOFTMAX */
  int n_group, topk_group;   /* default 1, 1 (no groups) */
  int group_top;             /* 1 or 2; default 1 */
  int renorm;                /* default 1 */
  float scale;               /* default 1; finite */
  int64_t ld_logits;         /* row stride of logits (and, backwards, of dlogits) */
} tdx_route_opts;
tdx_status tdx_route_opts_default(tdx_route_opts* opts);
tdx_status tdx_moe_route(const void* logits, const float* bias, int32_t* topk_idx, float* gates,
                         int32_t* counts, int T, int E, int topk, tdx_dtype dtype,
                         const tdx_route_opts* opts, void* stream);

/* Its gradient: dlogits = the gradient of sum(gates * dgates) by the logits, the chosen ids held
 * fixed (score, renorm and scale as in the forward call; groups and bias play no part). All of
 * dlogits (T x E of `dtype`) is written. An id outside [0, E) contributes nothing. */
tdx_status tdx_moe_route_bwd(const void* logits, const int32_t* topk_idx, const float* dgates,
                             void* dlogits, int T, int E, int topk, tdx_dtype dtype,
                             const tdx_route_opts* opts, void* stream);

/* Gated SiLU between two products (the experts' or a dense block's):
 *   out[r] = g * sigmoid(g) * u,  g = c * y[r][0 .. I), u = c * y[r][I .. 2I).
 * fp32 results take the exact exp and quotient (within 2^-20 of the value); bf16 and e4m3 ones approximate
 * ones, within 2^-22 * (4 + |g|) of it before their own rounding. sigmoid(g) is 0 from g = -88.8 down.
 *  y          device, R x 2I of `dtype` (TDX_BF16 or TDX_FP32).
 *  out        device, R x I of opts->out_dtype (TDX_BF16, TDX_FP32, or TDX_FP8_E4M3 stored as
 *             out / opts->out_scale, the one scale an e4m3 product takes).
 *  row_scale  optional, fp32 scales of the rows (c = 1 if NULL), for rows whose product was taken of
 *             tokens scaled one by one (tdx_rmsnorm's row_scale). With opts->topk = 0 row r takes
 *             row_scale[r]; with opts->topk = k the R rows are those of R / k tokens in the order of
 *             dest (R int32, as tdx_moe_dispatch_gemm writes it): row dest[i] takes row_scale[i / k],
 *             and a row that dest does not name is not written. Entries outside [0, R) are skipped.
 *  dest       given exactly when opts->topk > 0. Both 4-byte aligned. */
typedef struct tdx_act_opts {
  tdx_dtype out_dtype;       /* default TDX_BF16 */
  float out_scale;           /* default 1; positive and finite, as its reciprocal */
  int topk;                  /* slots per token for row_scale and dest; default 0; divides R */
  int64_t ld_y, ld_out;      /* row strides (backwards: of y and dy, and of dout) */
} tdx_act_opts;
tdx_status tdx_act_opts_default(tdx_act_opts* opts);
tdx_status tdx_swiglu(const void* y, void* out, const float* row_scale, const int32_t* dest, int R,
                      int I, tdx_dtype dtype, const tdx_act_opts* opts, void* stream);

/* Its gradient (c = 1): dy[r] = { dout * u * s * (1 + g * (1 - s)), dout * g * s }, s = sigmoid(g).
 *  y, dy      device, R x 2I of `dtype`; dy may be y itself. dout: R x I of `dtype`. */
tdx_status tdx_swiglu_bwd(const void* y, const void* dout, void* dy, int R, int I, tdx_dtype dtype,
                          const tdx_act_opts* opts, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Products without communication, with their gradients: the linear layer (tdx_linear), the products
 * grouped by expert over ragged rows (tdx_grouped_gemm) and the sum of a token's expert rows
 * (tdx_moe_combine). W ranks whose tensors lie in one buffer, rank after rank, are one call.
 * Products of bf16 or e4m3 operands are accumulated in fp32 on the tensor cores, in one fixed order
 * for given sizes; the epilogue is fp32 and every output is rounded once (RNE; e4m3 saturates at
 * +-448). No call needs a workspace but tdx_linear_act_bwd. Pointers are 16-byte aligned, rows and
 * strides multiples of 16 bytes (TDX_ERR_ALIGNMENT); fp32 vectors named "scale" and offsets 4-byte.
 * Row strides are in elements, 0 = dense; below the row's length: TDX_ERR_INVALID_ARG. Outputs overlap
 * no input unless said so. Sizes K, N, E, H, topk are at least 1; M, R or T of 0 launch nothing but
 * the zeroing that the formula asks for, and tensors of that many rows may then be NULL, as an empty
 * tensor's address is. A wait inside a kernel that runs out (4 s for what
 * takes milliseconds) ends that kernel's work and sets opts->device_status. */
typedef enum {
  TDX_ACT_NONE = 0,
  TDX_ACT_RELU = 1,
  TDX_ACT_GELU = 2,        /* x * Phi(x), Phi the normal distribution function */
  TDX_ACT_GELU_TANH = 3,   /* 0.5 x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) */
  TDX_ACT_SILU = 4,        /* x * sigmoid(x) */
  TDX_ACT_SWIGLU = 5       /* columns [0, N/2) are gates: silu(x[i]) * x[N/2 + i], N/2 output columns */
} tdx_activation;

typedef struct tdx_linear_opts {
  tdx_dtype out_dtype;       /* forward: of C or Y (TDX_BF16, the default, TDX_FP32 or TDX_FP8_E4M3);
                                backward: of dA or dX (TDX_BF16 or TDX_FP32) */
  tdx_activation act;        /* default TDX_ACT_NONE */
  float alpha;               /* multiplies the product (the scales of e4m3 operands); default 1, finite */
  float out_scale;           /* e4m3 output is stored as C / out_scale; default 1; positive and
                                finite, as its reciprocal */
  tdx_dtype dw_dtype;        /* backward: of dB (TDX_BF16, the default, or TDX_FP32) */
  int accumulate;            /* backward: 1 adds to dB as it is (the sum is fp32, then rounded to
                                dw_dtype); default 0 overwrites it */
  int64_t ld_a, ld_b;        /* row strides of A or X; of B (and of dB) */
  int64_t ld_c;              /* of C or Y; backward: of dA or dX */
  int64_t ld_residual;       /* of residual; tdx_linear_bwd: of dres */
  int64_t ld_z;              /* of z; backward: of dz or dY (tdx_linear_act_bwd: of z and dz) */
  uint32_t* device_status;   /* optional device word, set to TDX_ERR_TIMEOUT if a wait ran out and
                                otherwise left as it is. NULL: nothing tells that outputs are
                                incomplete; one word may serve any number of calls */
} tdx_linear_opts;
tdx_status tdx_linear_opts_default(tdx_linear_opts* opts);

/* Linear layer:  v = alpha * row_scale[m] * (A @ B) + bias,  C = act(v) + residual.
 *  A          device, M x K of `dtype` (TDX_BF16 or TDX_FP8_E4M3); B: K x N of `dtype`.
 *  bias       optional, N bf16. residual: optional, as C but bf16; C may be residual itself where it
 *             is bf16 (same stride).
 *  row_scale  optional, M fp32: the scales of A's rows (tdx_rmsnorm's row_scale).
 *  C          device, M x N of opts->out_dtype (M x N/2 for TDX_ACT_SWIGLU).
 *  z          optional, M x N bf16: v, for tdx_linear_act_bwd (C takes act(v) of the unrounded v).
 * N is a multiple of 8 (bf16) or 16 (e4m3), for TDX_ACT_SWIGLU N/2 is; for e4m3 outputs the output's
 * columns are multiples of 16.
 * Activations take approximate exponentials for bf16 and e4m3 outputs, within 2^-22 * (4 + |x|) of the
 * value (TDX_ACT_GELU_TANH: |x| the exponent's size, 1.6 |x + 0.045 x^3|), and exact ones for fp32; a
 * sigmoid below 2^-128 is 0. The tensor cores truncate their sums' additions, so sums over K (and of a
 * gradient's rows or columns) are added up in fp32 from segments: fp32 results of at most 896 (bf16;
 * e4m3 1792), others of at most 65536. */
tdx_status tdx_linear(const void* A, const void* B, const void* bias, const void* residual,
                      const float* row_scale, void* C, void* z, int M, int K, int N, tdx_dtype dtype,
                      const tdx_linear_opts* opts, void* stream);

/* Gradient of the activation and the bias:  dz = dy * act'(z),  dbias = sum_m dz[m] (unrounded).
 *  dy         device, M x N bf16 (M x N/2 for TDX_ACT_SWIGLU; opts->ld_c is its stride).
 *  z, dz      device, M x N bf16; dz may be z itself or, but for TDX_ACT_SWIGLU, dy (same stride). For
 *             TDX_ACT_NONE z and dz may be NULL (dz is dy); else dz may be NULL where dbias is not.
 *  dbias      optional, N fp32, overwritten; partial sums over rows are added in a fixed order.
 *  workspace  tdx_linear_act_bwd_workspace_size() bytes, 256-byte aligned, for dbias only; needs no
 *             initialisation.
 *  dtype      TDX_BF16. */
tdx_status tdx_linear_act_bwd_workspace_size(int M, int N, tdx_dtype dtype, const tdx_linear_opts* opts,
                                             size_t* bytes);
tdx_status tdx_linear_act_bwd(const void* dy, const void* z, void* dz, float* dbias, void* workspace,
                              size_t workspace_bytes, int M, int N, tdx_dtype dtype,
                              const tdx_linear_opts* opts, void* stream);

/* Gradients of the product:  dA = alpha * dz @ B^T + dres,  dB = alpha * A^T @ dz (+ dB).
 *  dz         device, M x N bf16; A: M x K bf16 (needed for dB); B: K x N bf16 (needed for dA).
 *  dres       optional, M x K bf16, with dA only; dA may be dres itself where it is bf16 (same stride).
 *  dA         optional, M x K of opts->out_dtype. dB: optional, K x N of opts->dw_dtype. One of the two.
 *  dtype      TDX_BF16. opts->act must be TDX_ACT_NONE. */
tdx_status tdx_linear_bwd(const void* dz, const void* A, const void* B, const void* dres, void* dA,
                          void* dB, int M, int K, int N, tdx_dtype dtype, const tdx_linear_opts* opts,
                          void* stream);

/* Products grouped by expert: rows offsets[e] .. offsets[e+1]-1 of X times B[e],
 *   v = alpha * row_scale[r] * expert_scale[e] * (X[r] @ B[e]),  Y[r] = act(v).
 * Rows in front of offsets[0] and from offsets[E] on are left as they are in Y and z.
 *  X          device, R x K of `dtype` (TDX_BF16 or TDX_FP8_E4M3), rows grouped by expert, as
 *             tdx_moe_dispatch_gemm lays them out.
 *  offsets    device, E + 1 int32, ascending (its expert_offsets). Entries are read on the device, taken
 *             into [0, R] and raised to the largest entry before them.
 *  B          device, E x K x N of `dtype`, expert e's at e * K * ld_b.
 *  row_scale  optional, R fp32; expert_scale: optional, E fp32.
 *  Y, z       as C and z of tdx_linear. E <= 512. */
tdx_status tdx_grouped_gemm(const void* X, const int32_t* offsets, const void* B, const float* row_scale,
                            const float* expert_scale, void* Y, void* z, int R, int K, int N, int E,
                            tdx_dtype dtype, const tdx_linear_opts* opts, void* stream);

/* Their gradients:  dX[r] = alpha * dY[r] @ B[e]^T,  dB[e] = alpha * X_e^T @ dY_e (+ dB[e]) over the
 * expert's rows; 0 (+ dB[e]) for an expert without rows. Rows of no expert are left as they are in dX.
 *  dY         device, R x N bf16; X: R x K bf16 (needed for dB); B: E x K x N bf16 (needed for dX).
 *  dX         optional, R x K of opts->out_dtype. dB: optional, E x K x N of opts->dw_dtype, expert e's at
 *             e * K * ld_b. One of the two. dtype TDX_BF16, opts->act TDX_ACT_NONE. */
tdx_status tdx_grouped_gemm_bwd(const void* dY, const void* X, const int32_t* offsets, const void* B,
                                void* dX, void* dB, int R, int K, int N, int E, tdx_dtype dtype,
                                const tdx_linear_opts* opts, void* stream);

/* Sum of a token's expert rows:  out[t] = sum_j gates[t][j] * Z[dest[t][j]], j ascending in fp32. With
 * gates NULL (all 1) it is the gradient of the dispatch by the tokens.
 *  Z          device, R x H of `dtype` (TDX_BF16 or TDX_FP32).
 *  dest       device, T x topk int32 (4-byte aligned), as tdx_moe_dispatch_gemm writes it. An entry outside
 *             [0, R) adds nothing.
 *  gates      optional, T x topk fp32 (4-byte aligned).
 *  out        device, T x H of opts->out_dtype (TDX_BF16 or TDX_FP32). 1 <= topk <= 16. */
typedef struct tdx_combine_opts {
  tdx_dtype out_dtype;       /* default TDX_BF16 */
  int64_t ld_z, ld_out;      /* row strides of Z (and dZ), of out (and dout) */
} tdx_combine_opts;
tdx_status tdx_combine_opts_default(tdx_combine_opts* opts);
tdx_status tdx_moe_combine(const void* Z, const int32_t* dest, const float* gates, void* out, int R, int T,
                           int H, int topk, tdx_dtype dtype, const tdx_combine_opts* opts, void* stream);

/* Its gradient:  dZ[dest[t][j]] = gates[t][j] * dout[t],  dgates[t][j] = sum_h dout[t][h] * Z[dest[t][j]][h].
 * With gates NULL it is the dispatch itself: each token's row copied to its experts' rows.
 *  dout       device, T x H of `dtype`; Z, dZ: R x H of `dtype`. dZ: optional; rows that dest does not name
 *             are left as they are. It may be Z itself (same stride). dest names a row once at most: of two
 *             writers of one row either may stay.
 *  dgates     optional (then Z is needed), T x topk fp32 (4-byte aligned), 0 for an entry outside [0, R).
 *  One of dZ and dgates is given. */
tdx_status tdx_moe_combine_bwd(const void* dout, const void* Z, const int32_t* dest, const float* gates,
                               void* dZ, float* dgates, int R, int T, int H, int topk, tdx_dtype dtype,
                               const tdx_combine_opts* opts, void* stream);

/* Synchronise `stream`, then read the workspace's device status word into *out (TDX_OK, or the
 * first device-side error since tdx_workspace_init). If detail is not NULL it receives 8 words:
 * [0] status, [1] role that failed (1 flag wait, 2 pipeline wait, 3 chain wait, 4 producer,
 * 5 MoE routing layout: [4] the first invalid expert id seen, [5] E), [2] CTA index, [3] flag/barrier
 * index, [4] value observed, [5] value expected, [6..7] reserved. An invalid MoE routing is reported
 * as TDX_ERR_INVALID_ARG here (the ids are only read on the device). */
tdx_status tdx_read_device_status(const void* workspace, void* stream, tdx_status* out,
                                  uint32_t* detail);

/* Introspection for tests and tools: the tiling and workspace layout a call with these arguments
 * uses. Writes 22 words to info: [0] tile width BN, [1] chain length L (RS: W; AG: K splits),
 * [2] M-tiles, [3] N-tiles, [4] tiles T, [5] K blocks (128 bytes of K each, one ring slot),
 * [6] chunk rows, [7] chunks per rank,
 * byte offsets in the workspace of [8] chunk flags (uint32 [W * chunks], index rank*chunks + c),
 * [9] chunk piece counters, [10] chain flags (uint32 [(L-1) * T], index c*T + tile), [11] gathered
 * buffer G, [12] fp32 running-sum / partial-slot buffer, [13] total workspace bytes, [14] reduce
 * mode in use (1 chained, 2 slotted, 0 none), [15] offset of the per-tile arrival counters,
 * [16] CTA cooperation in use (1 single, 3 2-SM pair), [17] ReduceScatter
 * raster: N-tiles per group (within a rank the tiles are taken group by group, M-tiles, then the
 * group's N-tiles), [18] ReduceScatter rank block:
 * that many positions of a rank's tile order are processed for ranks 0..W-1 before the next block
 * (positions count tiles, or tile pairs when [16] >= 2), [19] 1 if AllGather tiles read A straight
 * from the shards (shards smaller than a 128-row tile: a tile covers 128/M_local whole shards, each
 * loaded from its own buffer, or all in one load when the shards sit at one stride, so no tile waits
 * on the gathered copy, which still completes G and its flags), else 0, [20] bytes per element of the running-sum / partial-slot buffer (4 fp32,
 * 2 bf16 partials), [21] how the slotted fold is shared (single CTAs, fp32 partials; depends on the
 * device's SM count and opts.num_sms): 0 the last arriver folds the tile; 1 every work item is in
 * one wave of the persistent grid, and each element of a tile waits for the tile's L partials and
 * folds 1/L of it; 2 several waves but fewer tiles than CTAs (or reduce_mode 3): after a grid
 * barrier every CTA folds 1/grid of all tiles. */
tdx_status tdx_plan_info(int op, int W, int M_local_or_M, int K, int N, tdx_dtype dtype,
                         const tdx_opts* opts, int64_t* info);

/* Bytes of the optional trace buffer (opts->trace) for a call on `grid` CTAs taking `items` work
 * items and releasing `chunks` chunk flags (AllGather: W * chunks per rank; MoE dispatch: the 128-row
 * chunks of the dispatched rows; 0 otherwise). Layout, in 32-bit words:
 *  [0..3]  {grid, items, chain length, tiles};
 *  then per CTA 12 statistics words {ns spent waiting on chunk flags, number of flag waits, ns
 *          spent waiting on rank-chain flags, items taken, then seven phase stamps, each the low 32
 *          bits of the GPU's nanosecond global timer: kernel entry, set-up done (barriers, Tensor
 *          Memory), all operand loads of the CTA's first item issued, all MMAs of its first item
 *          issued, last MMA completed, epilogue done with the CTA's own items, epilogue done (shared
 *          folds included); the MMA stamps are 0 for the second CTA of a 2-SM pair, the load and
 *          MMA stamps 0 for a CTA without items; then one word 0};
 *  then the producer section: one count of released chunks, then `chunks` words: word k holds the
 *          flag index (AllGather: rank * chunks per rank + chunk) of the k-th chunk released by the
 *          call, whichever CTA released it. The count must be zero when the call starts (pass a
 *          zero-filled buffer); every other word is written by the kernel;
 *  then per CTA, in order, the work items it took, one word each: (chain element << 24) | tile id,
 *          tile id = m_tile * N-tiles + n_tile. CTA b takes items b, b + grid, b + 2*grid, ... (CTA
 *          pairs: pair b/2 takes items b/2, b/2 + grid/2, ...). */
size_t tdx_trace_size(int grid, int items, int chunks);

/* Static description of a status code. Never NULL. */
const char* tdx_status_string(tdx_status s);

/* Library version, (major << 16) | minor. */
uint32_t tdx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TDX_H_ */
