/*
 * exact_row_top.h -- C ABI of the MI355X (gfx950) exact per-row top-K library.
 *
 * The operation is the exact top-K selection a sparse-attention (DSA) indexer
 * runs over one fp32 score row per query, as stated on the TensorRT-LLM pages:
 *
 *  - "Self-sampling GVR V2 prefill indexer top-K" (PR 18702), section
 *    "Kernel": per row r, the top-K of logits[r, ks:ke] with ks = row_starts[r]
 *    and ke = row_ends[r], written in the row's LOCAL frame (column - ks) with a
 *    trailing -1 pad, and the identity 0..nv-1 when nv = ke - ks <= K.
 *  - "Block-skip fast path for self-sampling GVR top-K decode" (PR 18122),
 *    first commit message ("Contract"): fp32 scores, K in {512, 1024, 2048},
 *    exact top-K in which indices may interchange only inside the K-th value's
 *    tie class; the short-row commit (identity then -1); the varlen commit
 *    (per-row valid lengths read on the device, no host reads).
 *
 * How it is computed (Guess-Verify-Refine, PR 20998 "GVR K=2048 reg_clus with
 * block64 sampling and parallel rescue", sections "Why the GLM row overflows"
 * and "What changes"): sample K scores as K/64 blocks of 64 spread over the
 * row, bracket the K-th value with the sample's min/max, histogram the row
 * against that bracket, find the bin where the count from the top crosses K,
 * keep the bins above it, compact the crossing bin's members as candidates and
 * refine them exactly; an invalid bracket or an oversized crossing bin takes an
 * exact radix-select rescue over the whole row inside the same launch.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All array arguments are DEVICE pointers owned by the caller; the library
 *    never frees or retains them.  Calls are stream-ordered on `stream`
 *    (NULL = the null stream): the host never waits, never reads device data
 *    and, when `workspace` is given, never allocates.
 *  - logits: fp32 [num_rows][row_stride], unit inner stride, base 16-byte
 *    aligned, row_stride a multiple of 4 floats (the float4 row-stride gate of
 *    PR 18702's format check).  Every row's full stride must be readable: the
 *    kernel loads whole aligned float4 groups, and masks lanes outside the
 *    window by position, so values outside [ks, ke) (poison) never reach the
 *    selection.
 *  - indices: int32 [num_rows][k], 4-byte aligned.  Long rows (nv > k) get k
 *    distinct positions in [0, nv) in unspecified order; short rows get
 *    0..nv-1 then -1.
 *  - NaN inside a window is outside the contract (PR 18122, the commit that
 *    documents run_varlen's inherited NaN-ordering limitation): the kernels
 *    stay memory-safe on such a row (every read and write stays inside the
 *    row's stride, its k output slots and the workspace), but the k indices
 *    written for it are unspecified: they need not be distinct, nor inside
 *    the window.  +-inf are ordinary values; -0 and +0 are equal.
 *  - workspace: optional caller-owned device buffer of at least
 *    topk_workspace_bytes(...) bytes, 16-byte aligned (TOPK_ELAYOUT
 *    otherwise: the split tier moves its counts as 16-byte words), zeroed
 *    ONCE by topk_workspace_init before
 *    its first use; every call returns it to that resting state (histograms,
 *    cursors and counters back to zero), so a captured graph can replay
 *    without a memset.  The
 *    split tier's row barriers need the workgroups of a launch to be resident
 *    together; the plan bounds each launch by the device's resident capacity,
 *    so kernels that pin the GPU's compute units for their whole lifetime must
 *    not run beside these calls; a row barrier that waits too long gives up,
 *    the call's results are then undefined, and topk_status reports it.
 *    Calls that run concurrently (different streams) must not share one
 *    workspace (PR 18122, "varlen engine and seam" commit: a caller
 *    workspace so that concurrent streams do not share the split tier's
 *    publish slab).  NULL selects a per-device slab (PR 18122, first commit:
 *    per-device workspace slab) the library allocates on first need, zeroes
 *    before the call returns, keeps until process exit, and grows only when a
 *    larger plan needs it (allocation is not capture-safe).  There is one slab
 *    per GPU: calls with a NULL workspace must all go to one stream, or be
 *    ordered across streams by the caller.
 *  - Return value: TOPK_OK or one of the TOPK_E* codes below; nothing else
 *    crosses the ABI (no exceptions).  Argument errors are detected on the
 *    host before anything is launched.
 */
#ifndef EXACT_ROW_TOP_H_
#define EXACT_ROW_TOP_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  TOPK_OK = 0,
  TOPK_EINVAL = 1,     /* null pointer with num_rows > 0, num_rows < 0, k not in
                          {512,1024,2048}, row_stride < 1 or >= 2^30, bad option
                          value, a row longer than the largest launch plan
                          (64 workgroups x 512 threads x 9 float4 groups:
                          1,179,648 scores from the 16-byte boundary below
                          the window's start) */
  TOPK_ELAYOUT = 2,    /* logits not 16-byte aligned, row_stride % 4 != 0,
                          indices / extents not 4-byte aligned, a caller
                          workspace the plan uses not 16-byte aligned */
  TOPK_EWORKSPACE = 3, /* caller workspace smaller than topk_workspace_bytes
                          (topk_decode_noalloc: a plan larger than its fixed
                          scratch) */
  TOPK_EDEVICE = 4,    /* current device is not gfx950, or no device */
  TOPK_ELAUNCH = 5,    /* a HIP launch or allocation failed */
};

/* Decode form (PR 18122 varlen contract with next_n = 1, compress ratio 1):
 * row r selects from logits[r, 0:nv) with nv = clamp(n_valid[r], 0,
 * row_stride).  n_valid: device int32[num_rows]. */
int topk_decode(const float* logits, int64_t row_stride, const int32_t* n_valid,
                int32_t num_rows, int32_t k, int32_t* indices, void* workspace,
                size_t workspace_bytes, hipStream_t stream);

/* Prefill form (PR 18702 "Kernel"): row r selects from logits[r, ks:ke) with
 * ks = clamp(row_starts[r], 0, row_stride), ke = clamp(row_ends[r], ks,
 * row_stride); indices are ks-relative.  row_starts / row_ends: device
 * int32[num_rows].  max_row_len: advisory host-side bound on ke - ks (0 =
 * none, < 0 rejected).  Launch shapes are always sized for row_stride, so any
 * window inside the stride is handled whatever the hint says. */
int topk_prefill(const float* logits, int64_t row_stride, const int32_t* row_starts,
                 const int32_t* row_ends, int32_t num_rows, int32_t k, int32_t* indices,
                 int64_t max_row_len, void* workspace, size_t workspace_bytes,
                 hipStream_t stream);

/* Decode form that allocates nothing, for callers that cannot call hipMalloc
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same selection as topk_decode with a NULL workspace, but
 * the multi-workgroup tier keeps its state in a fixed per-GPU scratch array
 * of the library (24 MiB, held from library load until process exit) instead
 * of a caller workspace or the library's slab.  Plans whose workspace would
 * exceed it give TOPK_EWORKSPACE (no decode plan on a 256-compute-unit GPU
 * does).  The first call on a GPU clears the array with a kernel on
 * `stream`; every call returns it to zero.  Every call on one GPU shares that
 * GPU's array: calls that overlap on one GPU (different streams, without
 * ordering between them) race and their results are undefined.  A row
 * barrier that gives up is counted by topk_status, whose reset also re-zeroes
 * the array. */
int topk_decode_noalloc(const float* logits, int64_t row_stride, const int32_t* n_valid,
                        int32_t num_rows, int32_t k, int32_t* indices, hipStream_t stream);

/* ---- Output options -------------------------------------------------------
 * Same selection as topk_decode / topk_prefill, with:
 *  values: optional device float[num_rows][k] (NULL = none), 4-byte aligned.
 *      values[r][i] is the score at indices[r][i] (logits[r, ks + idx]); short
 *      rows (nv <= k) keep their identity indices and pad values with
 *      -FLT_MAX (PR 18122, values-output commit).
 *  flags: TOPK_SORTED orders each long row's indices (and values) by value
 *      descending, then index ascending; TOPK_DETERMINISTIC resolves the K-th
 *      value's tie class by smallest index, so the selected set is the same on
 *      every call (PR 20998 "What changes" and "Walkthrough": smallest-index
 *      deterministic ties, optional output sorting).  With both flags a long
 *      row's output is its canonical top-k: positions ordered by value
 *      descending, equal values by position ascending.  Short rows are always
 *      identity + -1.  Unknown flag bits give TOPK_EINVAL.
 * Values and sorting run as a second kernel on the same stream. */
#define TOPK_SORTED 1u
#define TOPK_DETERMINISTIC 2u

int topk_decode_v(const float* logits, int64_t row_stride, const int32_t* n_valid,
                  int32_t num_rows, int32_t k, int32_t* indices, float* values, uint32_t flags,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

int topk_prefill_v(const float* logits, int64_t row_stride, const int32_t* row_starts,
                   const int32_t* row_ends, int32_t num_rows, int32_t k, int32_t* indices,
                   float* values, uint32_t flags, int64_t max_row_len, void* workspace,
                   size_t workspace_bytes, hipStream_t stream);

/* Varlen / MTP decode form (PR 18122, run_varlen commit: the production
 * decode contract): kv_lens is a device int32 array with one TOTAL cache length
 * per request, in uncompressed token space; row r belongs to request
 * r / next_n and selects from logits[r, 0:n) with
 *     n = (kv_lens[r / next_n] - next_n + r % next_n + 1) / compress_ratio
 * (integer division), no window when kv_lens[r / next_n] < next_n, and n
 * clamped to row_stride.  kv_lens needs ceil(num_rows / next_n) entries.
 * next_n >= 1 (MTP rows per request) and compress_ratio >= 1 (1 and 4 in the
 * pages' models), else TOPK_EINVAL.  values / flags as in topk_decode_v. */
int topk_decode_varlen(const float* logits, int64_t row_stride, const int32_t* kv_lens,
                       int32_t num_rows, int32_t next_n, int32_t compress_ratio, int32_t k,
                       int32_t* indices, float* values, uint32_t flags, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/* ---- Hint-guided guess ----------------------------------------------------
 * Decode forms that also take the previous decode step's top-K positions as
 * hints (PR 18122 run_varlen commit: request-level raw pre_idx shared by a
 * request's next_n rows; "hint-robustness" commit and PR 20998 "What
 * changes": hints only steer the guess, exactness never depends on them).
 *  pre_idx: device int32, one row of at least k entries per request (per row
 *      in the plain decode form), pre_idx_stride (>= k, else TOPK_EINVAL)
 *      entries apart, 4-byte aligned.  Entries are raw positions in the
 *      row's window; any value is allowed: -1, positions at or past the
 *      window end and duplicates are ignored or harmless.  The guess reads
 *      the first min(k, workgroup size) entries of a hint row (256 to 1024;
 *      keep the hints of a row in no particular order, e.g. as a selection
 *      returns them).  NULL = no hints (the calls then equal topk_decode_v /
 *      topk_decode_varlen).
 * The result is the same exact selection as without hints, whatever the
 * hints hold.  Hints steer the multi-workgroup tier (the bracket's top and
 * floor); hints whose scores give no usable bracket (all invalid, all one
 * position) change nothing.  One-workgroup rows do not read them: their
 * retry takes the row's own maximum. */
int topk_decode_hinted(const float* logits, int64_t row_stride, const int32_t* n_valid,
                       const int32_t* pre_idx, int64_t pre_idx_stride, int32_t num_rows, int32_t k,
                       int32_t* indices, float* values, uint32_t flags, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

int topk_decode_varlen_hinted(const float* logits, int64_t row_stride, const int32_t* kv_lens,
                              const int32_t* pre_idx, int64_t pre_idx_stride, int32_t num_rows,
                              int32_t next_n, int32_t compress_ratio, int32_t k, int32_t* indices,
                              float* values, uint32_t flags, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* ---- Block-skip pass --------------------------------------------------------
 * Decode form with per-32-score block maxima (PR 18122 "Description" and its
 * block-skip commit): the pass reads bmax and visits only the score blocks
 * whose maximum can reach the sampled threshold, then selects exactly as the
 * other forms do (same result, same output options).
 *  bmax: device float [num_rows][bmax_stride], bmax_stride >= ceil(row_stride
 *      / 32) (else TOPK_EINVAL), 4-byte aligned.  bmax[r][i] must be at least
 *      every score of logits[r, 32i : 32i + 32) inside the row's window (an
 *      upper bound suffices: NaN or +inf make a block always visited); with a
 *      smaller value the result is unspecified.  topk_block_max writes the
 *      exact maxima (the indexer GEMM's epilogue would in production).
 *  Gate (shape only): num_rows * row_stride * 4 >= 128 MiB and row_stride >=
 *  72 * k; other calls take the ordinary decode path, bmax unused.  The pass
 *  uses no workspace; hints are not used by it.
 *  Without bmax, decode calls of at least 128 rows whose row_stride exceeds
 *  what one resident workgroup holds (36864) and spans at least 4 * k blocks
 *  of 32 (up to 8192) take the pass in its streaming form, which makes the
 *  maxima itself (topk_options.blockskip = -1 keeps the resident tiers). */
int topk_decode_blockskip(const float* logits, int64_t row_stride, const int32_t* n_valid,
                          const float* bmax, int64_t bmax_stride, int32_t num_rows, int32_t k,
                          int32_t* indices, float* values, uint32_t flags, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* bmax[r][i] = max over logits[r, 32i : min(32i + 32, row_stride)) (NaN
 * ignored unless the whole block is NaN), for i < ceil(row_stride / 32). */
int topk_block_max(const float* logits, int64_t row_stride, int32_t num_rows, float* bmax,
                   int64_t bmax_stride, hipStream_t stream);

/* ---- Caller workspace and status ----------------------------------------
 * The pages' runner takes an optional caller workspace (PR 18122: run_ws
 * with a caller workspace, first commit; run_varlen(workspace=...) in the
 * "varlen engine and seam" commit, so that concurrent streams do not share
 * one publish slab).  These calls size, prepare and audit one. */

/* Bytes of workspace a call with num_rows rows of stride `max_row_len` needs
 * (pass the row_stride of the call; 0 when the plan uses one workgroup per
 * row and needs none).  The value does not depend on the device.  Returns 0
 * for invalid arguments as well.  Host only: no device access. */
size_t topk_workspace_bytes(int32_t num_rows, int64_t max_row_len, int32_t k);

/* Zero a workspace once before its first use: a stream-ordered memset of
 * workspace_bytes bytes of the caller's device buffer (the library keeps no
 * reference to it).  workspace NULL with workspace_bytes 0 is a no-op;
 * NULL with a size gives TOPK_EINVAL; a failed memset TOPK_ELAUNCH.  Not for
 * use inside a captured graph (it records a memset node); a zeroed workspace
 * stays zeroed between calls, so a graph needs none. */
int topk_workspace_init(void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Stream-ordered audit of the split tier's bounded waits on the current
 * device.  Writes to *timeouts (device int32, 4-byte aligned) the number of
 * row-barrier waits that gave up since the previous topk_status on this
 * device, then resets that count.  A non-zero count means some call since
 * then returned undefined indices (its workgroups were not all resident
 * together: another kernel held compute units).  When the count is non-zero
 * the same launch also re-zeroes the library-owned slab; any caller
 * workspace used since then must be re-zeroed with topk_workspace_init
 * before its next use.  Two kernels on `stream`, no allocation, no host
 * sync; timeouts NULL gives TOPK_EINVAL. */
int topk_status(int32_t* timeouts, hipStream_t stream);

/* Static text for a status code (the pages' calls raise contract errors
 * loudly instead of falling back: PR 18122, the run_varlen production commit
 * and its fp32-contract commit).  Never NULL; unknown codes give
 * "unknown status". */
const char* topk_strerror(int status);

/* ---- Test and diagnostic surface ------------------------------------------
 * Same operations with knobs for tests.  `opts` may be NULL (= defaults).
 *  force_wgs_per_row: 0 = automatic plan; 1 = one workgroup per row; G > 1 =
 *      G workgroups per row (G <= 64), subject to the plan still fitting.
 *  force_rescue: nonzero = treat every long row's bracket as invalid, so the
 *      exact radix rescue runs on every long row.
 *  row_stats: optional device int32[num_rows][TOPK_STATS_WORDS]; per row:
 *      [0] path (0 short, 1 bracket + refine, 2 rescue: invalid bracket,
 *          3 rescue: crossing bin over the candidate cap (after the
 *          recounts below, where they apply), 5 fast path after a recount:
 *          a split row whose counts above its floor fell short of k counted
 *          again with no floor; a one-workgroup row whose crossing bin was
 *          the crowded top bin counted that bin again up to the row's
 *          maximum),
 *      [1] m (crossing-bin population, -1 if not computed),
 *      [2] above (count in bins above the crossing bin, -1 if none),
 *      [3] crossing bin index (-1 if none),
 *      [4] bit pattern of the bracket's low end (the sample minimum, or the
 *          lowest hint score when hints steered it), [5] of its high end,
 *      [6] workgroups per row, [7] candidate cap,
 *      [8] split rows: the floor bin the row's histogram counts from (-1 for
 *          one-workgroup rows and rows without a valid bracket); block-skip
 *          rows: the score blocks the last walk visited.
 *  Block-skip rows report path 1 (survivors only), 5 (counts short of k: every
 *  block recounted without a floor), 3 (crossing bin over the member cap) or 2
 *  (invalid bracket or forced rescue: radix select over the whole row).
 */
#define TOPK_STATS_WORDS 9

typedef struct topk_options {
  int32_t force_wgs_per_row;
  int32_t force_rescue;
  int32_t* row_stats;
  float* values;   /* as in topk_decode_v */
  uint32_t flags;  /* as in topk_decode_v */
  const int32_t* pre_idx; /* as in topk_decode_hinted (decode forms only,
                             else TOPK_EINVAL) */
  int64_t pre_idx_stride;
  const float* bmax;      /* as in topk_decode_blockskip (decode forms only) */
  int64_t bmax_stride;
  int32_t blockskip;      /* with bmax: 0 = the gate decides, 1 = always the
                             block-skip pass, -1 = never; 2 = the pass with
                             maxima it makes itself in a first streaming pass
                             (decode forms, rows of at most 8192 blocks of
                             32; bmax unused) */
  int32_t barrier_spins;  /* polls a split-tier row-barrier wait makes before
                             it gives up: 0 = the default (2^24, about a
                             second), n > 0 = n; < 0 gives TOPK_EINVAL.
                             Small values make waits give up on purpose
                             (undefined results, counted by topk_status):
                             for tests of that path only. */
} topk_options;

int topk_decode_ex(const float* logits, int64_t row_stride, const int32_t* n_valid,
                   int32_t num_rows, int32_t k, int32_t* indices, void* workspace,
                   size_t workspace_bytes, hipStream_t stream, const topk_options* opts);

int topk_prefill_ex(const float* logits, int64_t row_stride, const int32_t* row_starts,
                    const int32_t* row_ends, int32_t num_rows, int32_t k, int32_t* indices,
                    int64_t max_row_len, void* workspace, size_t workspace_bytes,
                    hipStream_t stream, const topk_options* opts);

int topk_decode_varlen_ex(const float* logits, int64_t row_stride, const int32_t* kv_lens,
                          int32_t num_rows, int32_t next_n, int32_t compress_ratio, int32_t k,
                          int32_t* indices, void* workspace, size_t workspace_bytes,
                          hipStream_t stream, const topk_options* opts);

/* Host-only planning and validation, callable without a GPU.  Fills
 * out[0..6] = {workgroups per row, float4 groups per thread, rows per launch,
 * launches, workspace bytes, candidate cap, workgroup size} for the shapes
 * given (the same
 * plan topk_decode / topk_prefill would use; `force_wgs_per_row` as in
 * topk_options; `cu_count` and `wgs_per_cu` stand in for the device's resident
 * capacity).  Returns a status code. */
int topk_plan_query(int32_t num_rows, int64_t row_stride, int64_t max_row_len, int32_t k,
                    int32_t force_wgs_per_row, int32_t cu_count, int32_t wgs_per_cu,
                    int64_t* out);

/* Facts about the current device the planner uses (out holds 37 values):
 * out[0] = compute units; for k = {512, 1024, 2048}[ki] and the qi-th split
 * variant, out[1 + 3*ki + qi] = resident split-tier workgroups per compute
 * unit the planner uses, out[10 + ..] = the runtime occupancy figure,
 * out[19 + ..] = VGPRs per thread, out[28 + ..] = static LDS bytes.
 * Returns a status. */
int topk_device_query(int64_t* out);

/* Workspace layout (host-only): out[0] = error header bytes, out[1] = bytes
 * of each slot's fixed block (header, rescue digit counts, row histogram:
 * every word rests at zero between calls), out[2] = slots, out[3] = byte
 * offset of the per-slot data blocks; a plan with G workgroups per row has
 * data blocks of G * out[4] + out[5] bytes (out[4] = one workgroup's slice of
 * suffix counts, one 16-bit count per value bin; out[5] = the crossing-bin
 * member list).  Returns a status. */
int topk_workspace_layout(int64_t* out);

/* Measurement aid (not a selection): reads exactly the scores the selection
 * of the same call would read -- the windows of rows longer than k, as
 * aligned float4 groups -- in the launch shape the selection's plan uses
 * (one workgroup per row, or G per row with the same part split), and does
 * nothing else with them.  Its time is the floor the row reads alone set
 * under the selection's time.  mode 0: decode (extents = n_valid); mode 1:
 * prefill (extents = row_starts, extents2 = row_ends).  sink: device
 * uint32[1], written only on a data-dependent condition that keeps the loads.
 * Block-skip and streaming forms are not modelled.  Status as for
 * topk_decode. */
int topk_read_floor(int32_t mode, const float* logits, int64_t row_stride, const int32_t* extents,
                    const int32_t* extents2, int32_t num_rows, int32_t k, uint32_t* sink,
                    hipStream_t stream);

/* Host-side argument validation exactly as the entry points run it (no device
 * access).  mode: 0 decode (extents = n_valid, extents2 unused), 1 prefill. */
int topk_validate(int32_t mode, const void* logits, int64_t row_stride, const void* extents,
                  const void* extents2, int32_t num_rows, int32_t k, const void* indices,
                  const void* workspace, size_t workspace_bytes, int64_t max_row_len);

/* ---- Row operators beside the selection --------------------------------------
 * What a serving or training step chooses next to the top-K: the cache slots
 * behind the selected positions, the experts of a token, the token itself.
 * The conventions above hold (device pointers, stream order, status codes, no
 * host reads); none of these calls allocates, keeps state or uses the
 * library's slab, so calls on different streams are independent as long as
 * their outputs and workspaces are.  Outputs overlap neither each other nor an
 * input, but where a call says so.  Equal scores go to the lower index.
 * Scores come in float32, bfloat16 or float16 (a TOPK_DT_* value), rows
 * row_stride elements apart with unit inner stride, aligned to their element;
 * whole aligned 16-byte groups that hold a row's scores are read. */
#define TOPK_DT_F32 0
#define TOPK_DT_BF16 1
#define TOPK_DT_F16 2

/* One token per row of logits [num_rows][vocab].
 *
 * NaN and -inf logits are never drawn.  With m the row's largest logit and
 * w_i = exp((x_i - m) / temperature), the kept tokens are a prefix of the
 * order by logit descending, then index ascending, cut by each of
 *   top_k: its first top_k tokens (<= 0 or >= vocab: all);
 *   top_p: the shortest prefix of those that holds at least top_p of their
 *          weight, never fewer than one (>= 1 or NaN: all);
 *   min_p: the tokens of those with w_i >= min(min_p, 1) (<= 0 or NaN: all).
 * The token is the lowest index at which the kept weights' running sum in
 * index order exceeds uniforms[r] times their total; uniforms outside [0, 1)
 * are clamped into it, NaN counts as 0.  A temperature that is not > 0 gives
 * the first token of the order.  A row without a drawable token gives -1.
 * Weights are held as whole multiples of 2^-43 of the largest, so results do
 * not depend on the order of any sum; weights of 2^-44 and less count as zero
 * and their tokens are never drawn.  A sum of weights is thus off by at most
 * vocab * 2^-44 of the largest and 2^-44 of itself, and so are the borders
 * between tokens, the cuts' and the total in logprobs.  (The total of a row
 * without a cut, and the one that a top_p without a top_k takes its share of,
 * are sums of weights rounded more finely: within the same bound, but not to
 * the bit what the multiples add up to.)
 *  temperature, top_p, min_p: device float[num_rows], top_k: device
 *      int32[num_rows]; each may be NULL (temperature 1, no cut).
 *  logprobs: optional device float[num_rows]: ln(w_token / kept total) (0 for
 *      temperature <= 0, -inf beside token -1).
 *  vocab: 1 .. 2^20.  row_stride >= vocab.
 *  workspace: at least topk_sample_workspace_bytes(num_rows, vocab) bytes,
 *      16-byte aligned; it needs no initialisation and holds nothing between
 *      calls (TOPK_EWORKSPACE if NULL or too small).
 *  flags: TOPK_SAMPLE_WHOLE_ROW reads every row again instead of using the
 *      candidates and sums of its first reading (for tests; the same results
 *      but for borders and totals within that bound of each other). */
#define TOPK_SAMPLE_WHOLE_ROW 1u

size_t topk_sample_workspace_bytes(int32_t num_rows, int32_t vocab);

int topk_sample(const void* logits, int32_t dtype, int64_t row_stride, int32_t vocab,
                int32_t num_rows, const float* uniforms, const float* temperature,
                const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                float* logprobs, uint32_t flags, void* workspace, size_t workspace_bytes,
                hipStream_t stream);

/* The top_k experts of each token and their weights.
 *
 * logits [num_tokens][num_experts]; s = sigmoid(x) (TOPK_ROUTE_SIGMOID) or
 * softmax over the token's experts; c = s + bias (bias: device
 * float[num_experts] or NULL; it takes part in the choice only, and without
 * one the order is that of the logits).  With num_groups > 1 the experts lie
 * in that many equal groups; the topk_groups groups with the largest score
 * (largest c, or with TOPK_ROUTE_TOP2 the sum of the two largest, one where
 * the group has one) stay.  The top_k largest c among them are chosen, in
 * falling order.  Experts whose logit or c is -inf or NaN are never chosen.
 *  indices, weights: device int32 / float [num_tokens][top_k].  weights are s
 *      of the chosen, divided by their sum with TOPK_ROUTE_RENORMALIZE, times
 *      scale; slots without an expert hold -1 and 0, and a sum of zero gives
 *      weights of 0.  Scores are 64-bit numbers, good to 2^-45 of themselves:
 *      two c (or sums of two) of different logits that differ by less than
 *      that may come in either order.  A sigmoid below 2^-1022 counts as zero;
 *      softmax scores that are divided by their sum are taken relative to the
 *      largest of the chosen.
 *  num_experts 1 .. 1024, top_k 1 .. min(64, num_experts), num_groups 1 .. 16
 *  dividing num_experts, topk_groups 1 .. num_groups. */
#define TOPK_ROUTE_SIGMOID 1u
#define TOPK_ROUTE_TOP2 2u
#define TOPK_ROUTE_RENORMALIZE 4u

int topk_route(const void* logits, int32_t dtype, int64_t row_stride, int32_t num_tokens,
               int32_t num_experts, int32_t top_k, const float* bias, int32_t num_groups,
               int32_t topk_groups, uint32_t flags, float scale, int32_t* indices, float* weights,
               hipStream_t stream);

/* Gradient of topk_route's weights in the logits: grad_weights [num_tokens]
 * [top_k] -> grad_logits [num_tokens][num_experts] in the logits' type, every
 * element written.  flags and scale as in the forward call (TOPK_ROUTE_TOP2
 * has no effect); indices as it returned them (entries outside [0,
 * num_experts) have no gradient; an expert named twice counts twice).  The
 * choice itself, the bias and the groups have no gradient. */
int topk_route_backward(const void* logits, int32_t dtype, int64_t row_stride, int32_t num_tokens,
                        int32_t num_experts, int32_t top_k, uint32_t flags, float scale,
                        const int32_t* indices, const float* grad_weights, void* grad_logits,
                        int64_t grad_row_stride, hipStream_t stream);

/* Block tables and slot maps of one step of a paged cache, from request
 * lengths.  Request r holds kv_lens[r] tokens once the step is done, the last
 * new_tokens[r] of them new (clamped to 0 <= new <= kv).  Its table row gets
 * the blocks it lacks, entries [ceil((kv - new) / block_size), ceil(kv /
 * block_size)), from free_blocks, taken in request order from place
 * free_start[0] on; other entries are read or left as they are.  The step's
 * new tokens, request after request, get
 *  token_starts  int32[num_requests + 1]: first token of each request, total;
 *  token_requests, positions  int32[max_tokens]: request, position in it;
 *  slots  int32 or int64 (slots_64) [max_tokens]: table[pos / block_size] *
 *      block_size + pos % block_size;
 *  free_next  int32[1]: free_start plus the blocks taken.
 * Entries behind the last token hold -1; tokens past max_tokens are counted
 * but not written (their blocks are handed out all the same).  Blocks past
 * the table's max_blocks are not taken and their tokens' slots are -1, as are
 * slots of negative blocks, of blocks the free list (num_free entries) does
 * not hold (free_next then exceeds num_free) and, in int32, slots over
 * 2^31 - 1.  Sums saturate at 2^31 - 1.
 * num_requests 0 .. 4096; block_size 1 .. 2^30; free_next must not be
 * free_start. */
int topk_block_tables(int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                      int32_t num_requests, const int32_t* kv_lens, const int32_t* new_tokens,
                      const int32_t* free_blocks, int64_t num_free, const int32_t* free_start,
                      int32_t block_size, int64_t max_tokens, int32_t* token_starts,
                      int32_t* token_requests, int32_t* positions, void* slots, int32_t slots_64,
                      int32_t* free_next, hipStream_t stream);

/* Slots of selected positions (a selection's local indices): slots[r][j] =
 * table[i / block_size] * block_size + i % block_size for i = indices[r][j],
 * in the table row of request row_requests[r] (device int32[num_rows]) or,
 * without it, r / next_n.  -1 where i is negative or past the table, the
 * request is not in [0, num_requests), the block is negative, or an int32 slot
 * would exceed 2^31 - 1.  k >= 1: any row length.  int32 slots may be written
 * over indices. */
int topk_slots(const int32_t* indices, int64_t num_rows, int32_t k, const int32_t* block_tables,
               int64_t table_stride, int32_t max_blocks, int32_t num_requests,
               const int32_t* row_requests, int32_t next_n, int32_t block_size, void* slots,
               int32_t slots_64, hipStream_t stream);

/* ---- A beam search's step over a paged cache -----------------------------------
 * The choice across a request's rows, what it does to the rows' states and
 * cache, attention over a cache whose prefix sequences share, and which cached
 * positions stay.  The conventions of the row operators hold.  Block tables
 * are int32 rows of max_blocks entries, table_stride apart; position p of a
 * row lies in block table[p / block_size] at p % block_size. */

/* The k best continuations of each request's beams.
 *
 * logits [num_requests * beams][vocab]; scores, ended, lengths
 * [num_requests][beams].  Beam b offers each token i whose logit is neither
 * NaN nor -inf with the total scores[b] + x_i - ln sum_j exp(x_j) (+inf logits
 * share the whole weight); an ended beam offers end_token alone, with its
 * score as it is, and its logits are not read; a beam whose score is not
 * finite offers nothing.  A total's rank is total / n^length_penalty with n =
 * lengths[b] + 1 (ended: lengths[b]; at least 1) and the power kept within
 * 2^-500 and 2^500, or the total itself without lengths.  The k largest ranks are chosen in falling order, equal ones by
 * beam, then token.
 *  out_scores, parents, tokens: device float / int32 / int32
 *      [num_requests][k]: total, beam and token; places without a candidate
 *      hold -inf, -1, -1.
 *  ended: device uint8 or NULL, lengths: device int32 or NULL.
 * Sums are 64-bit, of exponentials good to 2^-39 of themselves, in one order:
 * only totals that near each other may come in either order, and beams with
 * equal scores and logits tie to the bit.  -inf and NaN logits add nothing.
 * vocab 1 .. 2^20, beams 1 .. 32, k 1 .. 64; workspace as for topk_sample, of
 * topk_beams_workspace_bytes(...) bytes. */
size_t topk_beams_workspace_bytes(int32_t num_requests, int32_t beams, int32_t k, int32_t vocab);

int topk_beams(const void* logits, int32_t dtype, int64_t row_stride, int32_t vocab, int32_t num_requests,
               int32_t beams, int32_t k, const float* scores, const uint8_t* ended, int32_t end_token,
               const int32_t* lengths, float length_penalty, float* out_scores, int32_t* parents,
               int32_t* tokens, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Rows by parent: for each array a, row r * k + j of targets[a] becomes row r *
 * beams + parents[r][j] of sources[a] (device pointers in host arrays;
 * strides and row_bytes in bytes, any alignment).  A target may be its source
 * (same stride, beams == k): rows are then moved in place, whatever the
 * parents; it overlaps nothing else, but arrays may lie side by side in rows of
 * one stride.  Rows whose parent is not in [0, beams)
 * are cleared (clear 1) or left (clear 0).  beams, k 1 .. 32. */
int topk_reorder_rows(int32_t num_arrays, const void* const* sources, void* const* targets,
                      const int64_t* source_strides, const int64_t* target_strides,
                      const int64_t* row_bytes, const int32_t* parents, int32_t num_requests,
                      int32_t beams, int32_t k, int32_t clear, hipStream_t stream);

/* Paged rows by parent.  All beams of request r hold kv_lens[r] tokens: full =
 * kv_lens[r] / block_size full blocks and, where kv_lens[r] % block_size > 0,
 * an open one.  Child j's table row gets its parent's entries [0, full), and
 * as entry `full` the child's own open block: tail_blocks[r][j] or, with
 * tail_blocks NULL (beams == k), the entry its own row holds there; the open
 * block's tokens are copied from the parent's to the child's own in every
 * cache.  Further entries are those of the child's own row (beams == k), else
 * -1.  So full blocks are shared and no block is ever taken or returned; the
 * open blocks of a request's rows are distinct, and blocks written for one
 * request are no other request's.  A child whose parent is not in [0, beams)
 * keeps its own row (-1 where beams != k); blocks outside [0, num_blocks) are
 * not copied.
 *  out_tables: [num_requests * k][max_blocks], may be block_tables (same
 *      stride, beams == k).
 *  caches: num_caches (at most 64) device arrays [num_blocks][block_size] of
 *      slot_bytes bytes each, contiguous and apart, in a host array.
 * beams, k 1 .. 32. */
int topk_reorder_blocks(const int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                        const int32_t* kv_lens, const int32_t* parents, int32_t num_requests,
                        int32_t beams, int32_t k, int32_t block_size, const int32_t* tail_blocks,
                        int32_t* out_tables, int64_t out_stride, int32_t num_caches, void* const* caches,
                        int64_t num_blocks, int64_t slot_bytes, hipStream_t stream);

/* Decode attention of sequences that share prefixes, bfloat16 or float16.
 *
 * q [num_seqs * next_n][num_heads][dim], next_n tokens a sequence, one after
 * the other; caches [num_blocks][block_size][num_kv_heads][dim] by their
 * strides (elements, multiples of 8); query head h reads key head h /
 * (num_heads / num_kv_heads).  Group g, the sequences group_starts[g] ..
 * group_starts[g + 1] - 1 (device int32[num_groups + 1], rising; NULL:
 * num_groups equal groups), sees the first shared_lens[g] positions of
 * shared_tables row g; then sequence s's token t sees the first own_lens[s] -
 * next_n + t + 1 positions of own_tables row s.  Sequences in no group have no
 * prefix, and starts that fall leave out all prefixes.
 *     out = sum_p softmax_p(scale q k_p) v_p,  lse = ln sum_p exp(scale q k_p)
 * over all of them; a token that sees nothing gives 0 and -inf.  Lengths are
 * cut to [0, what the table row holds] (and max_shared_len, max_own_len where
 * those are > 0: bounds that the work is planned for).  Positions whose block
 * is not in [0, num_blocks) are left out.  Slots behind the lengths may hold
 * anything; values that some token of a sequence sees must be finite for all
 * of its tokens.  scale >= 0.  Scores, sums and the weighted values are 32-bit;
 * weights are rounded to the caches' type for them (float16: weights below 2^-21
 * of the row's largest lose bits there, those below 2^-32 vanish).
 *  out: [num_seqs * next_n][num_heads][dim] in q's type, contiguous, 16-byte
 *      aligned; lse: float [num_seqs * next_n][num_heads] or NULL.
 *  workspace: topk_attend_workspace_bytes(...) bytes (ragged: group_starts is
 *      given; the longest lengths as planned for), 16-byte aligned.
 * dim 64 or 128, next_n 1 .. 1024, at most 2^30 positions a row, block_size
 * 1 .. 2^20, block and head strides below 2^31, slot strides below 2^27. */
size_t topk_attend_workspace_bytes(int32_t num_groups, int32_t num_seqs, int32_t ragged, int32_t next_n,
                                   int32_t num_heads, int32_t num_kv_heads, int32_t dim,
                                   int64_t max_shared_len, int64_t max_own_len);

int topk_attend(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride, int32_t num_seqs,
                int32_t next_n, int32_t num_heads, int32_t num_kv_heads, int32_t dim, const void* k_cache,
                int64_t k_block_stride, int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache,
                int64_t v_block_stride, int64_t v_slot_stride, int64_t v_head_stride, int64_t num_blocks,
                int32_t block_size, const int32_t* shared_tables, int64_t shared_stride,
                int32_t shared_width, const int32_t* shared_lens, const int32_t* group_starts,
                int32_t num_groups, const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                const int32_t* own_lens, float scale, int64_t max_shared_len, int64_t max_own_len,
                void* out, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Attention mass of cached positions, from topk_attend's lse:
 *     shared_out[g][h][p] = decay shared_mass[g][h][p] + sum of exp(scale q k_p
 *         - lse) over the group's tokens and the query heads of key head h,
 * and the same of own_out[s][h][p] over sequence s's tokens that see p.  Every
 * position of the rows ([..][num_kv_heads][shared_positions] and
 * [..][num_kv_heads][own_positions], contiguous float) is written; those that
 * no token sees get the decayed mass alone, as all of shared_out does where
 * group_starts fall.  A mass array may be NULL (zeros) or its output.  Tokens
 * whose lse is -inf or NaN add nothing.  A weight is as good as its score and its
 * 32-bit lse: 2^-23 of |lse|.  The rest as for topk_attend; sums have one order,
 * so results repeat bit for bit. */
int topk_attend_mass(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride, int32_t num_seqs,
                     int32_t next_n, int32_t num_heads, int32_t num_kv_heads, int32_t dim, const void* k_cache,
                     int64_t k_block_stride, int64_t k_slot_stride, int64_t k_head_stride, int64_t num_blocks,
                     int32_t block_size, const int32_t* shared_tables, int64_t shared_stride,
                     int32_t shared_width, const int32_t* shared_lens, const int32_t* group_starts,
                     int32_t num_groups, const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                     const int32_t* own_lens, float scale, const float* lse, float decay,
                     const float* shared_mass, float* shared_out, int32_t shared_positions,
                     const float* own_mass, float* own_out, int32_t own_positions, hipStream_t stream);

/* The same with the bounds that the topk_attend call was given: it cut lengths to
 * them (0: none), and its log-sums hold no position behind. */
int topk_attend_mass_bounded(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride,
                             int32_t num_seqs, int32_t next_n, int32_t num_heads, int32_t num_kv_heads,
                             int32_t dim, const void* k_cache, int64_t k_block_stride, int64_t k_slot_stride,
                             int64_t k_head_stride, int64_t num_blocks, int32_t block_size,
                             const int32_t* shared_tables, int64_t shared_stride, int32_t shared_width,
                             const int32_t* shared_lens, const int32_t* group_starts, int32_t num_groups,
                             const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                             const int32_t* own_lens, float scale, int64_t max_shared_len,
                             int64_t max_own_len, const float* lse, float decay, const float* shared_mass,
                             float* shared_out, int32_t shared_positions, const float* own_mass,
                             float* own_out, int32_t own_positions, hipStream_t stream);

/* The cached positions that stay: of request r's n = kv_lens[r] positions (cut
 * to [0, positions]) in each of num_heads rows of mass (strides in elements),
 * all where n <= budget, else the first `sinks`, the last `recent`, and the
 * budget - sinks - recent of the others with the largest mass (equal masses:
 * the lower position first; NaN below all).
 *  kept: int32 [num_requests][num_heads][budget], rising, then -1;
 *  mass_out: float [num_requests][num_heads][out_positions] or NULL: the kept
 *      positions' mass, then 0; out_positions >= budget;
 *  new_lens: int32 [num_requests]: min(n, budget).
 * budget >= 1, sinks + recent <= budget. */
int topk_evict_keep(const float* mass, int64_t request_stride, int64_t head_stride, int32_t positions,
                    int32_t num_requests, int32_t num_heads, const int32_t* kv_lens, int32_t budget,
                    int32_t sinks, int32_t recent, int32_t* kept, float* mass_out, int32_t out_positions,
                    int32_t* new_lens, hipStream_t stream);

/* Moves the kept positions' rows to the front: in every cache and of every head
 * group, position j of out_tables row r becomes position kept[r][h][j] of
 * block_tables row r (left as it is where kept is -1 or a block is not in [0,
 * num_blocks)).  kept rises and kept[r][h][j] >= j, as topk_evict_keep gives
 * it.  out_tables is block_tables (pointer and stride: in place) or names blocks
 * that block_tables does not; no block belongs to two requests.
 *  caches: num_caches (at most 64) device arrays [num_blocks][block_size] of
 *      slot_bytes bytes, contiguous, apart and 16-byte aligned, in a host array; head
 *      group h's share of a slot is the h-th of num_heads equal parts, a
 *      multiple of 16 bytes. */
int topk_evict_move(const int32_t* kept, int32_t num_requests, int32_t num_heads, int32_t budget,
                    const int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                    const int32_t* out_tables, int64_t out_stride, int32_t out_blocks, int32_t block_size,
                    int32_t num_caches, void* const* caches, int64_t num_blocks, int64_t slot_bytes,
                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ROW_TOP_H_ */
