/*
 * spax.h -- C ABI of libspax: three-tier activation-sparse decoding GEMV on gfx950.
 *
 * What the library computes (batch-one decoding, one activation vector per call):
 *
 *   SpAx, "Activation Sparsity with Weight Approximation for Faster LLM Decoding on
 *   Offloaded Weights" (arXiv:2610.02598), Abstract: each weight is read in its original
 *   form, read from a compressed approximation, or not read; activations closest to zero
 *   skip their weights, smaller-magnitude ones read the approximation, the largest read
 *   the original.  The eigenradar commentary on SpAx ("The route outside GPU memory",
 *   first and third paragraphs) makes the unit one weight column per input channel, the
 *   approximation two-bit, and stores jointly accessed columns together.
 *
 *   TopK-Guided (arXiv:2610.01763), section 2.1 "TopK-Guided Masking": the tier mask may
 *   be a TopK, a threshold, or a threshold estimate clipped to +-delta around the target
 *   followed by TopK.
 *
 *   y[r] = sum_{j in FULL} x[j] * W[r][j]  +  sum_{j in APPROX} x[j] * What[r][j]
 *
 * and what stands between two such products in a decoder layer: the append to a paged key-value
 * cache with its rotation, the attention of the new token, the residual add with its norms, and
 * the gated activation ("between the projections" below).  A prompt goes through the same layer
 * many tokens at a time: spax_packed_gemm, spax_kv_append, spax_chunk_attention.
 *
 * Conventions shared by every entry point:
 *   - Return SPAX_OK (0) or a negative spax_status.  All argument validation happens on
 *     the host before anything is enqueued; on error nothing runs and no output buffer
 *     is touched.  spax_last_error() then holds a thread-local message.
 *   - "device pointer" means memory the GPU can address (hipMalloc).  The caller owns
 *     every buffer; the library never allocates device memory in these calls.
 *   - Work is enqueued on the given HIP stream and is asynchronous unless stated.
 *   - fp16 values are passed as uint16_t bit patterns; y is fp32.
 *   - No exceptions cross this boundary.
 */
#ifndef SPAX_H
#define SPAX_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- status codes */
typedef enum spax_status {
  SPAX_OK = 0,
  SPAX_ERR_NULL = -1,        /* a required pointer is NULL                          */
  SPAX_ERR_SHAPE = -2,       /* layout sizes not supported (see spax_layout_init)    */
  SPAX_ERR_PARAM = -3,       /* tier parameters out of range                         */
  SPAX_ERR_ALIGN = -4,       /* a pointer is not aligned as required                 */
  SPAX_ERR_WORKSPACE = -5,   /* workspace too small                                  */
  SPAX_ERR_HIP = -6,         /* a HIP runtime call failed (message has the details)  */
  SPAX_ERR_UNSUPPORTED = -7, /* valid request the library does not implement         */
  SPAX_ERR_HOST = -8         /* host memory or a host thread could not be obtained   */
} spax_status;

/* ---------------------------------------------------------------- packed layout */
enum { SPAX_FMT_FP16 = 0, SPAX_FMT_INT4 = 1 };

#define SPAX_MAX_MATS 4
#define SPAX_MAX_DIN 32768     /* largest input vector one tier-mask workgroup holds */
#define SPAX_RECORD_ALIGN 128  /* column records are padded to one 128-byte line     */

/*
 * spax_layout: shape and byte layout of one packed weight blob.
 *
 * Pages: eigenradar commentary on SpAx, "The route outside GPU memory", third
 * paragraph (jointly accessed columns are placed together).  Matrices that multiply the
 * same activation vector (q|k|v, gate|up) are fused: the record of input channel j holds
 * column j of every matrix, concatenated along rows (matrix 0 rows first).
 *
 * Blob = region F (original tier) then region A (two-bit approximation); both are
 * column-major with one record per input channel, in channel order, each record
 * zero-padded to a multiple of 128 bytes:
 *   region F, record j at  j * stride_F:
 *     FP16: d_out_total fp16 values (little endian);
 *     INT4: d_out_total/2 bytes of codes (row 2k in bits [3:0], row 2k+1 in [7:4]) then
 *           d_out_total/base_group u32 words, fp16 scale in bits [15:0], fp16 zero in
 *           bits [31:16];
 *   region A, record j at  off_A + j * stride_A:
 *     d_out_total/4 bytes of two-bit codes (row 4k+i in bits [2i+1:2i]) then
 *     d_out_total/approx_group (scale, zero) u32 words as above.
 * A group of G rows reconstructs as w_hat = s*q + z (z = group minimum, s = (max-min)/L,
 * q = round-half-even((w - z)/s) clamped to [0, L], L = 3 for two-bit, 15 for int4;
 * every step in fp32 with round-to-nearest-even, s and z rounded to fp16).
 *
 * The caller fills the input fields; spax_layout_init fills the derived ones.
 */
typedef struct spax_layout {
  /* inputs */
  int32_t n_mats;                /* 1..SPAX_MAX_MATS matrices sharing one input       */
  int32_t d_in;                  /* input channels = columns, 1..SPAX_MAX_DIN          */
  int32_t d_out[SPAX_MAX_MATS];  /* rows of each matrix; each a multiple of every group */
  int32_t base_fmt;              /* SPAX_FMT_FP16 or SPAX_FMT_INT4                     */
  int32_t base_group;            /* INT4 group rows: 128                               */
  int32_t approx_group;          /* two-bit group rows: 64 or 128                      */
  int32_t reserved0;
  /* derived by spax_layout_init */
  int64_t d_out_total;           /* sum of d_out                                       */
  int64_t rec_F, rec_A;          /* unpadded record bytes                              */
  int64_t stride_F, stride_A;    /* padded record bytes (multiples of 128)             */
  int64_t off_A;                 /* byte offset of region A = d_in * stride_F          */
  int64_t total_bytes;           /* blob size                                          */
} spax_layout;

/* Validate the inputs of *L and fill its derived fields.  Host only; enqueues nothing.
 * Pages: eigenradar commentary on SpAx, "The route outside GPU memory", first paragraph (each
 * weight column has an original and a two-bit approximate form) and third paragraph (columns
 * used together are stored together); the SpAx Abstract's 16-bit and 4-bit weights give the
 * two base formats.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE if n_mats, d_in, a group size or the format is
 * out of range, or any d_out[m] is not a positive multiple of approx_group (and of
 * base_group for INT4). */
int spax_layout_init(spax_layout* L);

/*
 * Pack fp16 weights into the blob (offline, once per weight set).  Pages: eigenradar
 * commentary on SpAx, "The route outside GPU memory", first and third paragraphs (an original
 * and a two-bit form of every column, prepared ahead of decoding and stored together).
 *   W[m]   : host array of n_mats device pointers; W[m] is matrix m stored column-major
 *            as d_in records of d_out[m] fp16 values (the record of channel j is column j).
 *   packed : device pointer, total_bytes, 256-byte aligned; fully overwritten, padding
 *            included, so the result is a deterministic function of the weights.
 * Weights must be finite (non-finite input gives unspecified codes).
 * Errors: SPAX_ERR_NULL, SPAX_ERR_SHAPE (layout not initialised), SPAX_ERR_ALIGN
 * (packed not 256-byte aligned or a W[m] not 16-byte aligned), SPAX_ERR_HIP.
 */
int spax_pack_columns(const spax_layout* L, const uint16_t* const* W, void* packed,
                      hipStream_t stream);

/*
 * Offline placement of the column records (eigenradar commentary on SpAx, "The route outside
 * GPU memory", third paragraph: jointly accessed columns are placed together, so a token's
 * selection reads fewer, longer ranges).  Host only.
 *   tiers : host, n_tokens rows of d_in tier bytes (SPAX_TIER_*), the masks of calibration
 *           tokens (e.g. spax_build_tiers' tier output copied back).
 *   order : host, d_in entries: a permutation of [0, d_in) with channels in descending order of
 *           the bytes they made selected (stride_F per FULL, stride_A per APPROX), equal
 *           scores in channel order.  Position p of a placed blob holds channel order[p].
 * Errors: SPAX_ERR_NULL, SPAX_ERR_SHAPE (layout not initialised), SPAX_ERR_PARAM (n_tokens < 0,
 * a byte that is not a tier).
 */
int spax_placement_order(const spax_layout* L, const uint8_t* tiers, int32_t n_tokens,
                         int32_t* order);

/*
 * spax_pack_columns with a placement: record p of each region holds column perm[p] (perm:
 * device, d_in int32, a permutation such as spax_placement_order's order; entries are clamped
 * to [0, d_in) so a malformed one repeats a column but stays in bounds).  The activation vector
 * of a placed blob is permuted alike, x_placed[p] = x[perm[p]] (in a model, once, through the
 * rows of the layer that produces x); masks, lists and the product then work on positions, and
 * y is the product over the same columns.  Errors: as spax_pack_columns, plus SPAX_ERR_NULL
 * (perm) and SPAX_ERR_ALIGN (perm not 4-byte aligned).
 */
int spax_pack_columns_placed(const spax_layout* L, const uint16_t* const* W,
                             const int32_t* perm, void* packed, hipStream_t stream);

/* ---------------------------------------------------------------- tier masks */
enum { SPAX_TIER_SKIP = 0, SPAX_TIER_APPROX = 1, SPAX_TIER_FULL = 2 };
enum { SPAX_MODE_TOPK = 0, SPAX_MODE_THRESHOLD = 1, SPAX_MODE_TOPK_GUIDED = 2 };

/*
 * Tier-mask parameters.  Ranking: channel j outranks k iff key_j > key_k, or equal keys
 * and j < k, with key = (fp16 bits of x) & 0x7FFF (so NaN ranks above +Inf).
 *   TOPK         : ranks [0, n_full) FULL, the next n_approx APPROX, the rest SKIP.
 *   THRESHOLD    : FULL if |x| >= tau_full, else APPROX if |x| >= tau_skip, else SKIP.
 *   TOPK_GUIDED  : natural skip count c = #{|x| < tau}; n_skip = min(max(c, n_skip_lo),
 *                  n_skip_hi); kept = d - n_skip; n_approx = floor((approx_num*kept +
 *                  floor(approx_den/2)) / approx_den); then TOPK(kept - n_approx, n_approx).
 *                  (TopK-Guided section 2.1; spax_guided_bounds gives the +-delta band.)
 * Float thresholds are compared as fp16 keys: |x| >= tau  <=>  key >= K(tau), with K(tau)
 * from spax_key_threshold.
 */
typedef struct spax_tier_params {
  int32_t mode;
  int32_t n_full, n_approx;        /* TOPK                                   */
  int32_t n_skip_lo, n_skip_hi;    /* TOPK_GUIDED clip band on the skip count */
  int32_t approx_num, approx_den;  /* TOPK_GUIDED FULL/APPROX split of kept   */
  int32_t reserved0;
  double tau_skip, tau_full;       /* THRESHOLD                               */
  double tau;                      /* TOPK_GUIDED calibrated threshold        */
} spax_tier_params;

/*
 * Build one tier mask (one workgroup per vector).
 *   x          : device, d_in fp16 activations.
 *   tier       : device, d_in bytes of SPAX_TIER_* (may be NULL: not written).
 *   full_idx   : device, capacity d_in int32; ascending channel indices of the FULL tier.
 *   approx_idx : device, capacity d_in int32; ascending indices of the APPROX tier.
 *   counts     : device, 3 int32 = {n_full, n_approx, n_skip}.  Stays on the device.
 * List entries past their count are unspecified.  x, lists and counts 4-byte aligned.
 * Errors: SPAX_ERR_NULL, SPAX_ERR_SHAPE (d_in outside 1..SPAX_MAX_DIN), SPAX_ERR_PARAM
 * (unknown mode, counts out of range, n_skip_lo > n_skip_hi, approx_den outside
 * 1..65535, approx_num outside [0, approx_den], tau_skip > tau_full, NaN thresholds),
 * SPAX_ERR_ALIGN, SPAX_ERR_HIP.
 */
int spax_build_tiers(const uint16_t* x, int32_t d_in, const spax_tier_params* p,
                     uint8_t* tier, int32_t* full_idx, int32_t* approx_idx, int32_t* counts,
                     hipStream_t stream);

/* ---------------------------------------------------------------- tiered GEMV */

/* Workspace bytes spax_tiered_gemv needs for layout *L.  The current kernels need none and
 * return 0 (then ws may be NULL); callers should still size ws with this function.
 * Returns 0 also if *L is not initialised. */
size_t spax_gemv_workspace_bytes(const spax_layout* L);

/*
 * y = tiered product of one packed blob with one activation vector.  Pages: SpAx Abstract
 * (read the original weights of the largest activations, the compressed approximation for
 * smaller ones, nothing for those closest to zero); eigenradar commentary, "The route outside
 * GPU memory", third paragraph (the two-bit approximation is reconstructed on the GPU).
 *   packed      : device blob laid out by *L (spax_pack_columns), 256-byte aligned.
 *   x           : device, d_in fp16 activations (the same vector the mask was built from),
 *                 4-byte aligned; for odd d_in the kernels may read the two bytes that pad
 *                 x to a whole dword (never past that dword).
 *   full_idx, approx_idx, counts : device, as written by spax_build_tiers (or any
 *                 caller lists of distinct channels with counts[0], counts[1]).  Counts are
 *                 clamped to [0, d_in] and indices to [0, d_in) on the device, so malformed
 *                 lists give an unspecified y but never an out-of-bounds access.  Entries past
 *                 a list's count are not read: it need not be longer (one entry at least).
 *   y           : device, d_out_total fp32, 16-byte aligned; fully overwritten (all zeros
 *                 if both lists are empty).  Rows follow the fused order of *L.
 *   ws, ws_bytes: device workspace of at least spax_gemv_workspace_bytes(L) bytes,
 *                 256-byte aligned (may be NULL when that size is 0).
 * Accumulation is fp32.  Column chunks handled by different workgroups meet in y through
 * fp32 atomic adds, so y can differ in the last bits between runs; the tier masks and
 * lists are bit-exact.  Enqueues a zero fill of y before the product when the launch
 * splits the column lists.
 * Errors: SPAX_ERR_NULL, SPAX_ERR_SHAPE, SPAX_ERR_ALIGN, SPAX_ERR_WORKSPACE, SPAX_ERR_HIP.
 */
int spax_tiered_gemv(const spax_layout* L, const void* packed, const uint16_t* x,
                     const int32_t* full_idx, const int32_t* approx_idx,
                     const int32_t* counts, float* y, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/* ---------------------------------------------------------------- pinned-host path */

/*
 * Read ranges of one column list (host helper).  Pages: eigenradar commentary on SpAx, "The
 * route outside GPU memory", third paragraph (adjacent read ranges are merged; coarse
 * granularity can move more bytes than were selected).
 *   idx      : host array of n ascending, distinct, non-negative channel indices.
 *   gap      : runs of consecutive channels separated by at most `gap` unselected channels
 *              are merged into one range (the gap columns are moved too); 0 merges only
 *              adjacent channels.
 *   first, count : host arrays of capacity n receiving each range (may be NULL to count only).
 *   n_ranges : receives the number of ranges.
 * Errors: SPAX_ERR_NULL, SPAX_ERR_PARAM (n < 0, gap < 0, idx not ascending / distinct /
 * non-negative).
 */
int spax_column_ranges(const int32_t* idx, int32_t n, int32_t gap, int32_t* first,
                       int32_t* count, int32_t* n_ranges);

/* Byte ledger of one mask read from block storage (spax_storage_ledger). */
typedef struct spax_storage_stats {
  int64_t selected_bytes;  /* n_full * stride_F + n_approx * stride_A                         */
  int64_t moved_bytes;     /* bytes of the merged record ranges (selected + merged gaps)       */
  int64_t read_bytes;      /* bytes physically read: n_blocks * block_bytes                    */
  int64_t n_blocks;        /* blocks read, each range rounded out to block boundaries          */
  int32_t n_ranges;        /* merged ranges (FULL + APPROX) = read requests                    */
  int32_t reserved0;
} spax_storage_stats;

/*
 * Bytes selected against bytes physically read when the blob sits on block storage (host
 * helper).  Pages: eigenradar commentary on SpAx, "The route outside GPU memory", third
 * paragraph (coarse storage granularity can move more bytes than a selected column needs) and
 * last paragraph (for NVMe, selected bytes and bytes physically read are separate entries);
 * the SpAx Abstract reports the flash-offloaded case apart.
 * The blob (laid out by *L) starts on a block boundary; the selected columns of each region
 * are merged into ranges as by spax_column_ranges (gap); each range is one read request that
 * reads every block of block_bytes its bytes touch (a block touched by two requests is read
 * twice).
 *   full_idx, approx_idx : host, n_full / n_approx ascending distinct channels < d_in.
 *   out : host.
 * Errors: SPAX_ERR_NULL, SPAX_ERR_SHAPE (layout not initialised), SPAX_ERR_PARAM (lengths out
 * of range, gap < 0, block_bytes < 1, a list not ascending / distinct / inside [0, d_in)).
 */
int spax_storage_ledger(const spax_layout* L, const int32_t* full_idx, int32_t n_full,
                        const int32_t* approx_idx, int32_t n_approx, int32_t gap,
                        int64_t block_bytes, spax_storage_stats* out);

/* Byte account of one spax_tiered_gemv_pinned call. */
typedef struct spax_move_stats {
  int64_t selected_bytes;  /* n_full * stride_F + n_approx * stride_A                   */
  int64_t moved_bytes;     /* record bytes copied host -> device (selected + merged gaps) */
  int64_t list_bytes;      /* list bytes copied host -> device: 0 for SPAX_PINNED_GATHER
                              (the lists never leave the device); for SPAX_PINNED_MEMCPY and
                              SPAX_PINNED_HOSTGATHER one upload of the span of the two
                              compacted host lists (d_in entries each) that holds every used
                              entry                                                       */
  int32_t n_ranges;        /* merged ranges (FULL + APPROX)                               */
  int32_t n_full, n_approx;
  int32_t reserved0;
} spax_move_stats;

/* spax_tiered_gemv_pinned: how the ranges cross PCIe */
enum {
  /* the lists come back to the host (the call synchronizes `stream`), which merges the
   * ranges and issues one hipMemcpyAsync per range (host-driven DMA) */
  SPAX_PINNED_MEMCPY = 0,
  /* the ranges are merged on the device (one kernel, two workgroups) and one copy kernel
   * reads them from the mapped pinned blob (zero-copy) into the compacted staging area:
   * nothing waits for the host, so the call is asynchronous unless `stats` is requested */
  SPAX_PINNED_GATHER = 1,
  /* the lists come back to the host (the call synchronizes `stream`), which merges the
   * ranges; a pool of host threads (up to 16, started on first use) copies the records of
   * every range from the pinned blob into one library-owned pinned staging buffer (FULL
   * records, then APPROX records, back to back), which moves to the device in 8 MiB
   * hipMemcpyAsync chunks, each issued as soon as it is filled (CPU gather, one DMA stream
   * that overlaps the gathering) */
  SPAX_PINNED_HOSTGATHER = 2
};

/* Device workspace for spax_tiered_gemv_pinned: a compacted staging copy of the blob's
 * records (total_bytes, for the case that every column is selected), two compacted lists and
 * two slot -> column tables (4 * d_in bytes each) and 24 bytes of totals; 0 if *L is not
 * initialised. */
size_t spax_pinned_workspace_bytes(const spax_layout* L);

/*
 * Tiered GEMV with the packed blob in pinned host memory (allocated with hipHostMalloc).
 *   packed_host : the blob laid out by *L (e.g. a copy of spax_pack_columns' output).
 *   x, full_idx, approx_idx, counts, y : device, as for spax_tiered_gemv (the lists as
 *                 written by spax_build_tiers: ascending).
 *   gap   : range merging, as for spax_column_ranges.
 *   transfer : SPAX_PINNED_MEMCPY, SPAX_PINNED_GATHER or SPAX_PINNED_HOSTGATHER (same bytes
 *              moved, same result).
 *   ws    : device, >= spax_pinned_workspace_bytes(L) bytes, 256-byte aligned.
 *   stats : host, may be NULL (the byte account; requesting it synchronizes `stream`).
 * Merges the selected columns of each region into ranges (on the device for
 * SPAX_PINNED_GATHER; on the host, after reading counts and lists back, for
 * SPAX_PINNED_MEMCPY and SPAX_PINNED_HOSTGATHER), moves the ranges host -> device (see `transfer`) into a compacted
 * staging area of ws (a range's columns land in consecutive slots, ranges in order) with the
 * compacted lists (staging slot | channel << 16), then runs the tiered GEMV over the staged
 * records.  y equals spax_tiered_gemv's on a device copy of the blob up to the order of fp32
 * additions.  Returns with the work enqueued on `stream`; with `stats` it also waits for the
 * byte account.  SPAX_PINNED_MEMCPY and SPAX_PINNED_HOSTGATHER: library-owned pinned buffers
 * (allocated on first use and grown as needed) hold the lists and, for the host gather, the
 * staged records; a later call waits until the previous call's copies from them have completed
 * before reusing them.
 * SPAX_PINNED_GATHER on lists that are not strictly ascending gives an unspecified y (never
 * an access outside the blob or ws).
 * Errors: as spax_tiered_gemv, plus SPAX_ERR_PARAM (gap < 0, unknown transfer, packed_host
 * not pinned host memory mapped for the device, and for the host-merged transfers lists read
 * back not ascending) and SPAX_ERR_WORKSPACE.
 */
int spax_tiered_gemv_pinned(const spax_layout* L, const void* packed_host, const uint16_t* x,
                            const int32_t* full_idx, const int32_t* approx_idx,
                            const int32_t* counts, float* y, int32_t gap, int32_t transfer,
                            void* ws, size_t ws_bytes, spax_move_stats* stats,
                            hipStream_t stream);

/* ---------------------------------------------------------------- decode step */

/*
 * One group of projections that share an activation vector (q|k|v, o, gate|up, down).
 * All pointers are device pointers as in spax_build_tiers / spax_tiered_gemv.
 */
typedef struct spax_phase {
  const spax_layout* layout;   /* host pointer to an initialised layout */
  const void* packed;
  const uint16_t* x;
  spax_tier_params params;
  uint8_t* tier;               /* may be NULL */
  int32_t* full_idx;
  int32_t* approx_idx;
  int32_t* counts;
  float* y;
} spax_phase;

/* spax_step.flags */
enum {
  /* one fused mask+GEMV launch per phase whose d_in <= 16384 (and whose lists fit in LDS):
   * one 1024-thread workgroup per compute unit, each finding the boundaries itself; other
   * phases take the two launches of SPAX_STEP_SEPARATE.  Same outputs either way.  Kernel
   * launches only (no copy, no memset), so the step can be captured into a HIP graph. */
  SPAX_STEP_DEFAULT = 0,
  /* one stand-alone mask launch (spax_build_tiers' kernel, which also clears y) and one
   * GEMV launch (spax_tiered_gemv's kernel) per phase */
  SPAX_STEP_SEPARATE = 1,
  /* every phase's mask in one launch, then every phase's GEMV in one persistent launch per
   * base format present (fp16 phases, then int4 phases).
   * Only for phases that are independent: all x ready when the step is enqueued, and no
   * phase's outputs (tier, lists, counts, y) overlapping another phase's inputs or outputs
   * (checked; SPAX_ERR_PARAM).  Needs ws of spax_step_workspace_bytes bytes (per-phase
   * descriptor tables, copied from a library-owned pinned ring of host buffers, so not
   * capturable in a graph).  events: [0, 1] bracket the mask launch, [2, 3] the GEMV launches
   * (one phase: [0, 1] bracket both).  Cannot be combined with SPAX_STEP_SEPARATE. */
  SPAX_STEP_BATCHED = 2,
  /* (with SPAX_STEP_DEFAULT or SPAX_STEP_SEPARATE) y identical bit for bit from run to run: a
   * phase's column chunks store their partial sums in ws instead of adding them into y with
   * atomics, and one more launch per phase adds the chunks in a fixed order.  Needs ws of
   * spax_step_workspace_bytes bytes, disjoint from every phase's buffers; y need not be
   * cleared (it is overwritten).  Not with SPAX_STEP_BATCHED, nor through
   * spax_decode_step_projections_noalloc (SPAX_ERR_UNSUPPORTED). */
  SPAX_STEP_DETERMINISTIC = 4
};

typedef struct spax_step {
  int32_t n_phases;            /* e.g. 32 layers x 4 groups = 128               */
  int32_t flags;
  const spax_phase* phases;    /* host array of n_phases                        */
  void* ws;                    /* device workspace, see spax_step_workspace_bytes */
  size_t ws_bytes;
  /* Optional timing hook (NULL: none): 2 * n_phases caller-created events.  events[2i] and
   * events[2i+1] are recorded on the stream right before and right after phase i's fused
   * mask+GEMV launch (its GEMV launch when the phase takes two launches), so they bracket
   * exactly that kernel. */
  hipEvent_t* events;
} spax_step;

/* Workspace bytes for spax_decode_step_projections over these phases, enough for every
 * launch form: the largest of the per-phase GEMV workspaces (currently 0), the
 * SPAX_STEP_BATCHED descriptor tables (a few hundred bytes per phase) and the
 * SPAX_STEP_DETERMINISTIC partial sums of the widest phase (column chunks x d_out_total
 * floats, about 2 MB for a 7B decoder layer).  0 for invalid input. */
size_t spax_step_workspace_bytes(const spax_phase* phases, int32_t n_phases);

/*
 * One batch-one decode step over all projection groups, in order: for each phase, the
 * tier mask of its activation vector, then the tiered GEMV of its fused matrices.
 * Phase p+1 is enqueued after phase p (stream order), as in a decoder where each
 * group's input depends on the previous group's output.  Launch forms: see spax_step.flags.
 * (eigenradar commentary on SpAx, second and last paragraphs: selection applies per
 * generated token during batch-one decoding.)
 * Errors: the union of spax_build_tiers and spax_tiered_gemv errors, reported before
 * anything is enqueued.
 */
int spax_decode_step_projections(const spax_step* step, hipStream_t stream);

/*
 * spax_decode_step_projections without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation).  Same phases, flags, validation and results as spax_decode_step_projections;
 * step->ws and step->ws_bytes are ignored.  SPAX_STEP_BATCHED keeps its descriptor tables
 * in a static device array of the library (256 KiB per GPU, held until the process ends;
 * about 208 bytes per phase, so at most 1257 phases, else SPAX_ERR_WORKSPACE), filled from a
 * static host buffer by one copy on `stream`; SPAX_STEP_DETERMINISTIC, whose partial sums
 * need a workspace, is refused (SPAX_ERR_UNSUPPORTED).  The call makes no hipMalloc,
 * hipHostMalloc or hipFree call and no host heap allocation (its first call on a device looks
 * up the array's address and creates one event).  Every call on one GPU shares
 * that array: calls that overlap on one GPU (different streams, or host threads on one
 * device) race, so callers serialize them, e.g. on one stream.  A call waits on the host
 * until the previous call's table copy has left the host buffer.
 */
int spax_decode_step_projections_noalloc(const spax_step* step, hipStream_t stream);

/* ---------------------------------------------------------------- between the projections */

/*
 * Operators of a decoder layer that stand between two projection groups: the paged cache append
 * with rotation, with or without a norm of each head, the attention of one new token per sequence
 * or of a chunk of them, the residual add with its norms, and the gated activation; and the
 * projection of many rows at once.  They take rows of any number of tokens; spax_decode_layers
 * runs those of one token with the projections of a batch-one step.
 *
 * All of them: pointers inside the structs are device pointers, the structs themselves are host
 * memory read during the call; strides are in elements, positive, and every row's own values
 * are contiguous; sums, statistics and angles are kept in 32 bits or more and each result is
 * rounded once, to nearest even; no atomics, so the same inputs give the same bits; kernel
 * launches only, so a call can be captured into a graph; pointers and stream belong to the
 * current device.  No output may share bytes with another output or with an input, except
 * where stated.  Columns of the same rows (equal row strides) are told apart; any other strided
 * buffer counts as the whole span from its first to its last element.
 */
enum { SPAX_F32 = 0, SPAX_F16 = 1, SPAX_BF16 = 2, SPAX_E4M3 = 3 };

/*
 * A paged cache of keys and values.  Page p holds page_size rows of every key head: the row of
 * head h and position r in the page starts at k + p * k_page_stride + h * k_head_stride +
 * r * k_row_stride (elements), head_dim values; v likewise.  Any order of pages, heads and rows
 * in memory is a choice of strides.  Position i of sequence s is row i % page_size of page
 * page_table[s * table_stride + i / page_size].  An entry outside [0, n_pages) names no page:
 * nothing is read or written there.
 *   E4M3: a stored value q of head h stands for q * k_scale[h] (v_scale[h]); NULL means 1.
 * Limits: head_dim 64, 96, 128, 192 or 256; page_size a power of two, 4..65536; k and v 16-byte
 * aligned and their strides a multiple of 16 bytes.  Rows may not overlap, nor, where the cache is
 * written, k's with v's.  In one allocation k and v may be interleaved: page by page (equal page
 * strides, each page's rows in any order), or with equal strides throughout by heads, rows or
 * any other axis.
 */
typedef struct spax_kv_cache {
  void* k;
  void* v;
  const int32_t* page_table;
  const float* k_scale;        /* E4M3 only: n_kv_heads values, may be NULL */
  const float* v_scale;
  int64_t k_page_stride, k_head_stride, k_row_stride;
  int64_t v_page_stride, v_head_stride, v_row_stride;
  int64_t table_stride;        /* >= max_pages                              */
  int32_t type;                /* SPAX_F16, SPAX_BF16 or SPAX_E4M3          */
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  int32_t n_seqs, max_pages;   /* rows and used columns of page_table       */
  int32_t reserved0;
} spax_kv_cache;

/*
 * Append: for token t of sequence s = seq[t] (t itself if seq is NULL) at position p =
 * positions[t], k and v go to row p of s in the cache and q to q_out.  The leading rot_dim
 * values of every q and k head are rotated pair by pair on the way: with angle a = p *
 * inv_freq[i] (product and reduction by whole turns in 64 bits),
 *   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
 * pair i being (i, i + rot_dim/2), or (2i, 2i + 1) if interleaved; later values and v are
 * copied.  E4M3: x / scale (rounded to 32 bits), clamped to +-448 (NaN stays NaN).
 *   q, k, v : src_type; token t, head h starts at t * token_stride + h * head_stride (a fused
 *             q|k|v row is three pointers into it).  q and q_out may both be NULL (n_heads 0).
 *   q_out   : out_type (SPAX_F16 or SPAX_BF16).  May be q itself, if type and strides agree.
 *   cache   : type out_type or SPAX_E4M3.
 * p < 0 is padding: nothing is cached and the token's q_out is zeros.  A position past max_pages
 * or on an entry that names no page, or a sequence outside [0, n_seqs), caches nothing (q_out is
 * written).  Two tokens of one call on one row: the row then holds, value by value, either
 * token's.  n_tokens 0 does nothing.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE (head_dim, page_size, rot_dim odd or past head_dim, a
 * size < 1, n_tokens > n_seqs without seq or 2^24 and more); SPAX_ERR_UNSUPPORTED (types); SPAX_ERR_ALIGN
 * (a pointer not aligned to its element, the cache as above); SPAX_ERR_PARAM (strides that
 * overlap, outputs that overlap); SPAX_ERR_HIP.
 */
typedef struct spax_kv_append_args {
  const spax_kv_cache* cache;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const int32_t* positions;
  const int32_t* seq;          /* may be NULL */
  const float* inv_freq;       /* rot_dim / 2 values; NULL with rot_dim 0 */
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
  int64_t v_token_stride, v_head_stride, out_token_stride, out_head_stride;
  int32_t src_type, out_type, n_tokens, n_heads, rot_dim, interleaved;
} spax_kv_append_args;

int spax_kv_append(const spax_kv_append_args* a, hipStream_t stream);

/* spax_head_norm.kind (and spax_residual_norm_args.kind): x * w / sqrt(mean x^2 + eps), or
 * (x - mean x) * w / sqrt(mean (x - mean x)^2 + eps); plus the bias if there is one. */
enum { SPAX_NORM_RMS = 0, SPAX_NORM_LAYER = 1 };

/*
 * spax_kv_append with a norm of every query head and every key head (over its head_dim values)
 * before the rotation, in the same pass; values v are cached as they are.  All in 32 bits, one
 * rounding at the end.
 *   q_weight, k_weight : head_dim fp32 values, for all heads (stride 0) or a row per head (stride
 *             >= head_dim); NULL: those heads are not normed (not both NULL; q_weight needs q).
 *   q_bias, k_bias : likewise, with the strides of their weights; may be NULL.
 * Squares are summed in 32 bits, as by spax_residual_norm.
 * Errors: of spax_kv_append; SPAX_ERR_NULL (norm NULL, or without a weight); SPAX_ERR_UNSUPPORTED
 * (kind); SPAX_ERR_ALIGN; SPAX_ERR_PARAM (eps not finite or < 0, a bias without its weight, q_weight
 * without q, a stride neither 0 nor >= head_dim, an output that overlaps a weight or bias).
 */
typedef struct spax_head_norm {
  const float* q_weight;
  const float* q_bias;
  const float* k_weight;
  const float* k_bias;
  int64_t q_stride, k_stride;
  int32_t kind;
  float eps;
} spax_head_norm;

int spax_kv_append_normed(const spax_kv_append_args* a, const spax_head_norm* norm,
                          hipStream_t stream);

/*
 * Attention of one new token per sequence over the paged cache.  Sequence s (row s of the page
 * table) holds n = lens[s] keys, the new token's own among them; query head h reads key head
 * h / (n_heads / n_kv_heads).  Over the keys j in [max(0, n - window), n) (window 0: all):
 *   score_j = scale * k_scale * q . k_j,   out = v_scale * sum_j softmax(score)_j v_j,
 *   lse = ln sum_j exp(score_j).
 * lens[s] is taken as clamped to [0, min(max_len, max_pages * page_size)].  Keys on entries
 * that name no page are left out; bytes of rows outside the range never reach the result,
 * whatever they hold; a value in the range that is not finite leaves its dim of the result not
 * finite (NaN, as a rule).  A sequence with no keys, or whose scores are all -inf, gives zeros and
 * lse -inf.  q, out : `type` (SPAX_F16 or SPAX_BF16), the cache's type or the cache E4M3; 16-byte
 * aligned with strides a multiple of 8 elements.  Probabilities enter the product with v as the
 * sum of two `type` values: within 2^-17 of themselves in BF16, and in F16 within 2^-22 of
 * themselves or 2^-40 of the sequence's largest.
 *   max_len : host bound on lens; sets how the keys are shared out, and the workspace.
 *   ws      : spax_attention_workspace_bytes(a) bytes (0: none needed), 256-byte aligned, any
 *             contents; calls that may run at the same time need a workspace each.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE (as for the cache; n_heads not a multiple of
 * n_kv_heads or past 65535; max_len < 1, past max_pages * page_size or past 2^30; more than 2^30
 * tiles of 32 keys in n_seqs sequences of max_len, or of window, each counted as four tiles more;
 * window < 0); SPAX_ERR_UNSUPPORTED
 * (types); SPAX_ERR_ALIGN; SPAX_ERR_PARAM (scale not finite, overlapping buffers);
 * SPAX_ERR_WORKSPACE; SPAX_ERR_HIP.
 */
typedef struct spax_attention_args {
  const spax_kv_cache* cache;
  const void* q;
  void* out;
  float* lse;                  /* n_seqs * n_heads, may be NULL */
  const int32_t* lens;
  int64_t q_seq_stride, q_head_stride, out_seq_stride, out_head_stride;
  int32_t type, n_heads, max_len, window;
  float scale;
  int32_t reserved0;
} spax_attention_args;

size_t spax_attention_workspace_bytes(const spax_attention_args* a);
int spax_paged_attention(const spax_attention_args* a, void* ws, size_t ws_bytes,
                         hipStream_t stream);

/*
 * Attention of a chunk of new tokens per sequence over the paged cache: a prompt, a piece of a long
 * one, drafted tokens that are checked at once, or any mixture in one call.  The rows of all
 * sequences are packed: sequence s (row s of the page table) has n_new = starts[s + 1] - starts[s]
 * new tokens, rows starts[s].. of q and out, and lens[s] keys, the new tokens' own among them
 * (append first).  Its row i is the token at position p = lens[s] - n_new + i, and over the keys
 * j in [max(0, p + 1 - window), p] (window 0: all up to p), for query head h with key head
 * h / (n_heads / n_kv_heads):
 *   score_j = scale * k_scale * q . k_j,   out = v_scale * sum_j softmax(score)_j v_j,
 *   lse = ln sum_j exp(score_j).
 * lens[s] is taken as clamped to [0, min(max_len, max_pages * page_size)], starts[s] to
 * [0, n_tokens] and as no smaller than any start before it: a sequence whose starts do not ascend
 * has no tokens, and no row belongs to two.  Keys on entries that name no page are left out; bytes
 * of rows that a token does not see never reach its result, whatever they hold.  A value that it
 * sees and that is not finite decides its dim, however small its weight: infinite, or NaN if it is
 * NaN or meets an infinity of the other sign.  A token with no keys (or at a negative position),
 * or whose scores are all -inf, gives zeros and lse -inf.  Rows of no
 * sequence (before starts[0], behind starts[n_seqs]) are left as they were.
 *   q, out : `type` (SPAX_F16 or SPAX_BF16), the cache's type or the cache E4M3; 16-byte aligned
 *             with strides a multiple of 8 elements.
 *   lse    : n_tokens * n_heads, may be NULL.
 * Weighted values are summed in 32 bits before the division by the sum of the weights (each at
 * most 2^8 in BF16): BF16 values past 2^120 divided by the number of keys may come out infinite.
 * Probabilities enter the product with v as one `type` value (spax_paged_attention's as two): within
 * 2^-8 of themselves in BF16, and in F16 within 2^-11 of themselves or 2^-39 of the row's largest.
 *   max_len : host bound on lens; with n_tokens it sets how the keys are shared out, as if every
 *             sequence were that long, so one far above the lengths costs time and workspace (1 x 509
 *             tokens of 32 heads of 128: 15 us and none with 509, 31 us and 136 MB from 4096 on).
 *   ws      : spax_chunk_attention_workspace_bytes(a) bytes (0: none needed), 256-byte aligned,
 *             any contents; calls that may run at the same time need a workspace each.
 * n_tokens 0 does nothing.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE (as for the cache; n_heads not a multiple of n_kv_heads or
 * past 65535; n_tokens < 0, or so many that n_tokens * n_heads passes 2^30; max_len < 1, past
 * max_pages * page_size or past 2^30; window < 0; more work items than a grid holds);
 * SPAX_ERR_UNSUPPORTED (types); SPAX_ERR_ALIGN; SPAX_ERR_PARAM (scale not finite, overlapping
 * buffers); SPAX_ERR_WORKSPACE; SPAX_ERR_HIP.
 */
typedef struct spax_chunk_attention_args {
  const spax_kv_cache* cache;
  const void* q;
  void* out;
  float* lse;
  const int32_t* starts;       /* n_seqs + 1 */
  const int32_t* lens;         /* n_seqs     */
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int32_t type, n_heads, n_tokens, max_len, window;
  float scale;
} spax_chunk_attention_args;

size_t spax_chunk_attention_workspace_bytes(const spax_chunk_attention_args* a);
int spax_chunk_attention(const spax_chunk_attention_args* a, void* ws, size_t ws_bytes,
                         hipStream_t stream);

/*
 * A block's output joins the residual stream, and the next block's input leaves it.  Per row:
 *   t = block;  t = norm(t; post_weight, post_bias) if post_weight;  t = t * gate if gate;
 *   h = residual + scale * t;   x = norm(h; pre_weight, pre_bias)   (from h before rounding).
 * residual_out gets h, x the normed row; either may be NULL, not both.  residual or block may be
 * NULL (0 is taken), not both; residual_out may be residual itself (type and stride alike), x
 * may be block itself likewise.  gate: gate_type, one row (gate_stride 0) or one per row.
 * Weights and biases are fp32 rows of d (weight NULL: ones for pre, no norm for post).  Squares are
 * summed in 32 bits: values of 2^56 and more (with eps 0 also rows below 2^-56) are past a norm's range.
 *   residual, residual_out : residual_type; block : block_type (SPAX_F32, SPAX_F16, SPAX_BF16);
 *   x : x_type (the same three).  1 <= d <= 32768; n_rows 0 does nothing, and 2^32 threads of
 *   eight values (rows rounded up to 64 of them) are the most.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE; SPAX_ERR_UNSUPPORTED (types, kind); SPAX_ERR_ALIGN (a
 * pointer not aligned to its element); SPAX_ERR_PARAM (scale or eps not finite, eps < 0, a
 * stride below d, a bias without its weight, overlapping buffers); SPAX_ERR_HIP.
 */
typedef struct spax_residual_norm_args {
  const void* residual;
  const void* block;
  void* residual_out;
  void* x;
  const void* gate;
  const float* post_weight;
  const float* post_bias;
  const float* pre_weight;
  const float* pre_bias;
  int64_t residual_stride, block_stride, residual_out_stride, x_stride, gate_stride;
  int32_t residual_type, block_type, gate_type, x_type, kind, n_rows, d;
  float scale, eps;
  int32_t reserved0;
} spax_residual_norm_args;

int spax_residual_norm(const spax_residual_norm_args* a, hipStream_t stream);

/* spax_glu_args.act: g / (1 + exp(-g)), or the tanh form of gelu,
 * g/2 * (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
enum { SPAX_ACT_SILU = 0, SPAX_ACT_GELU_TANH = 1 };

/*
 * x = act(gate) * up, row by row (gate and up: src_type, usually the two halves of a gate|up
 * projection's row; x: x_type; types SPAX_F32, SPAX_F16, SPAX_BF16).  Any d from 1 to 2^30, fewer than
 * 2^24 pieces of 2048 values of a row; n_rows 0 does nothing.  x may be gate or up itself (type and stride alike).
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE; SPAX_ERR_UNSUPPORTED (types, act); SPAX_ERR_ALIGN;
 * SPAX_ERR_PARAM (a stride below d, overlapping buffers); SPAX_ERR_HIP.
 */
typedef struct spax_glu_args {
  const void* gate;
  const void* up;
  void* x;
  int64_t gate_stride, up_stride, x_stride;
  int32_t src_type, x_type, act, n_rows, d, reserved0;
} spax_glu_args;

int spax_glu(const spax_glu_args* a, hipStream_t stream);

/* spax_packed_gemm_args.form */
enum { SPAX_GEMM_PLAIN = 0, SPAX_GEMM_ACT = 1, SPAX_GEMM_GATED = 2 };

/*
 * The product of rows of many tokens with the original columns (region F) of one packed blob, the
 * projection of a prompt (selection applies per generated token during batch-one decoding:
 * eigenradar commentary on SpAx, second and last paragraphs).  With W the fused matrices and
 * t = x W^T + bias (bias NULL: 0), row by row:
 *   PLAIN: u = t;   ACT: u = act(t);   GATED (two matrices of equal d_out): u = act(t_0) * t_1;
 *   y = residual + scale * u   (residual NULL: scale * u).
 * y and residual have d_out_total columns, d_out[0] with GATED.  act: SPAX_ACT_SILU or
 * SPAX_ACT_GELU_TANH (not read with PLAIN).  A placed blob takes x permuted alike, as by
 * spax_pack_columns_placed.
 *   x        : n_rows rows of d_in fp16, 16-byte aligned, x_stride a multiple of 8 (what lies
 *              between a row's end and the next multiple of 8 may be read and never counts).
 *   residual : residual_type, y : y_type (SPAX_F32, SPAX_F16, SPAX_BF16); residual may be y itself
 *              (type and stride alike).
 * Sums are in 32 bits, in an order that depends on the sizes alone; the weights of an INT4 base
 * enter the product as w_hat rounded to fp16 (the tiered GEMV keeps them in 32 bits), so one of
 * 65520 and more is infinite.
 *   ws       : spax_packed_gemm_workspace_bytes(a) bytes (0: none needed), 256-byte aligned, any
 *              contents; calls that may run at the same time need a workspace each.
 * n_rows 0 does nothing.
 * Errors: SPAX_ERR_NULL; SPAX_ERR_SHAPE (layout not initialised; GATED without two equal
 * matrices; n_rows < 0 or 2^20 and more); SPAX_ERR_UNSUPPORTED (types, form, act); SPAX_ERR_ALIGN
 * (packed not 256-byte aligned, x as above, another pointer not aligned to its element);
 * SPAX_ERR_PARAM (scale not finite, a stride below its row, overlapping buffers);
 * SPAX_ERR_WORKSPACE; SPAX_ERR_HIP.
 */
typedef struct spax_packed_gemm_args {
  const spax_layout* layout;   /* host pointer to an initialised layout */
  const void* packed;
  const uint16_t* x;
  const float* bias;           /* d_out_total, may be NULL */
  const void* residual;        /* may be NULL              */
  void* y;
  int64_t x_stride, residual_stride, y_stride;
  int32_t n_rows, form, act, residual_type, y_type;
  float scale;
} spax_packed_gemm_args;

size_t spax_packed_gemm_workspace_bytes(const spax_packed_gemm_args* a);
int spax_packed_gemm(const spax_packed_gemm_args* a, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/*
 * One decoder layer of a batch-one step, in order: qkv, append, attention, o, attn_norm,
 * gate_up, glu, down, mlp_norm.  attn_norm's x is gate_up's input; mlp_norm's x is the next
 * layer's qkv input (the first layer's is the caller's, e.g. spax_residual_norm without a
 * block).  All pointers are host structs; layers may share buffers (stream order).
 */
typedef struct spax_decoder_layer {
  const spax_phase* qkv;
  const spax_kv_append_args* append;
  const spax_attention_args* attention;
  const spax_phase* o;
  const spax_residual_norm_args* attn_norm;
  const spax_phase* gate_up;
  const spax_glu_args* glu;
  const spax_phase* down;
  const spax_residual_norm_args* mlp_norm;
} spax_decoder_layer;

/* Workspace of spax_decode_layers in every launch form: the larger of the step's and the
 * attentions' (they use it one after another).  0 for invalid input. */
size_t spax_layers_workspace_bytes(const spax_decoder_layer* layers, int32_t n_layers);

/*
 * A whole batch-one decode step through n_layers decoder layers: the projections of
 * spax_decode_step_projections with the operators above between them, nothing else enqueued.
 *   flags : SPAX_STEP_DEFAULT, SPAX_STEP_SEPARATE and SPAX_STEP_DETERMINISTIC as for the step
 *           (SPAX_STEP_BATCHED needs independent phases: SPAX_ERR_UNSUPPORTED).
 *   ws    : spax_layers_workspace_bytes bytes, 256-byte aligned, disjoint from every buffer of
 *           the layers.
 * Everything is checked before anything is enqueued: each part as by its own call, that one row
 * (token, sequence) passes through, and that the parts are wired to each other: append reads
 * inside qkv's y and the attention reads append's q_out and its cache; o reads the attention's
 * out; attn_norm reads o's y and writes gate_up's x; glu reads inside gate_up's y and writes
 * down's x; mlp_norm reads down's y and writes the next layer's x.
 * Errors: of the parts; SPAX_ERR_PARAM for a part wired elsewhere (message names layer and part).
 */
int spax_decode_layers(const spax_decoder_layer* layers, int32_t n_layers, int32_t flags,
                       void* ws, size_t ws_bytes, hipStream_t stream);

/* spax_decode_layers of layers whose append norms the heads (spax_kv_append_normed): norms[i] is
 * layer i's, NULL for a layer without; host memory, read during the call.  Errors: also those of
 * spax_kv_append_normed; SPAX_ERR_NULL if norms is NULL. */
int spax_decode_layers_normed(const spax_decoder_layer* layers, const spax_head_norm* const* norms,
                              int32_t n_layers, int32_t flags, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* ---------------------------------------------------------------- diagnostics */

/* A plain streaming read, to measure what a launch that only reads gets from the memory
 * system (not a step of the method; the benchmark uses it for a read ceiling and for a
 * read floor at the byte counts of a decode step's launches).  The `bytes` bytes at p
 * (device memory) are read once with 16-byte non-temporal loads by 512-thread workgroups
 * (reads of 1 GiB or more: one contiguous chunk per workgroup, one workgroup per compute
 * unit; smaller reads: grid-stride over four workgroups per unit), and every wave stores
 * the XOR of the 32-bit words it read in its own word of `out` (device memory, out_words
 * uint32, at least 8; fewer words than waves means fewer workgroups).  The XOR of the first
 * *n_written words (host; nullable) is the XOR of all words read.  bytes = 0 launches
 * nothing and sets *n_written = 0.  Asynchronous on `stream`.  Errors: SPAX_ERR_NULL (p or
 * out NULL), SPAX_ERR_ALIGN (p or bytes not a multiple of 16, out not 4-byte aligned),
 * SPAX_ERR_PARAM (out_words < 8), SPAX_ERR_HIP. */
int spax_read_probe(const void* p, size_t bytes, uint32_t* out, int32_t out_words,
                    int32_t* n_written, hipStream_t stream);

/* ---------------------------------------------------------------- host helpers */

/* K(tau): smallest fp16 magnitude key k in [0, 0x7C00] with half(k) >= tau (compared in
 * double), else 0x7C01.  Returns -1 for NaN.  Pages: TopK-Guided section 2.1 (the natural
 * sparsity of a token counts activations below a calibrated threshold); the threshold is
 * compared on fp16 keys so the device compares integers only. */
int32_t spax_key_threshold(double tau);

/* Fixed keep fractions -> counts by cumulative round-half-up:
 * n_full = floor(p_full*d + 0.5), n_keep = floor((p_full + p_approx)*d + 0.5).  Pages:
 * TopK-Guided Abstract and section 1 (a TopK mask keeps a fixed count per token); the pages
 * give no rounding, cumulative round-half-up is this library's choice. */
int spax_counts_from_fractions(int32_t d, double p_full, double p_approx,
                               int32_t* n_full, int32_t* n_approx);

/* TopK-Guided +-delta band on the skip count (section 2.1): n_lo = max(0,
 * ceil(d*(s - delta) - 1e-9)), n_hi = min(d, floor(d*(s + delta) + 1e-9)). */
int spax_guided_bounds(int32_t d, double s, double delta, int32_t* n_lo, int32_t* n_hi);

/* ---------------------------------------------------------------- sparsity budgets (host) */

/*
 * Per-block sparsity targets from measured sensitivities (TopK-Guided, arXiv:2610.01763,
 * section 2.2 "Sensitivity-Aware Block Sparsity": blocks more sensitive than average get less
 * sparsity, the global budget moves to robust blocks, lambda sets how much moves, targets are
 * clamped; the pages clamp to [0.05, 0.95]).  Host only.
 *   sens    : n_blocks finite positive sensitivities (e.g. each block's output change at a
 *             probe sparsity, from a calibration pass).
 *   s_block : n_blocks outputs.  u_b = s + lambda * (mean(sens) - sens_b) / mean(sens);
 *             s_block[b] = min(max(u_b + c, s_min), s_max) with the shift c that makes the
 *             mean of s_block equal s (c = 0 when nothing is clamped).
 * Errors: SPAX_ERR_NULL; SPAX_ERR_PARAM (n_blocks < 1, lambda < 0, s outside [s_min, s_max],
 * a sensitivity not finite and positive).
 */
int spax_block_sparsity(const double* sens, int32_t n_blocks, double s, double lambda,
                        double s_min, double s_max, double* s_block);

/* Block output error of a trial allocation p[0..n_mats) (caller-defined, e.g. measured on
 * calibration tokens). */
typedef double (*spax_block_error_fn)(const double* p, int32_t n_mats, void* user);

/*
 * Greedy split of a block's sparsity over its matrices (TopK-Guided Appendix D "Block-wise
 * Greedy Sparsity Allocation", Table 4).  Host only.  From p = 0, each round tries one
 * increment alpha * mean(params) / params[m] on every matrix m that stays <= 1, keeps the one
 * whose trial allocation has the least block_error (ties: lower m), and records the row
 * (P, p[0..n_mats)), P = sum params[m] p[m] / sum params[m]; every increment moves P by
 * alpha / n_mats.  The first row is (0, zeros); the walk stops once P >= P_max or no matrix
 * can step.  Matrices that share one activation vector share one tier mask, so in a decoder
 * layer the units are the projection groups (q|k|v, o, gate|up, down).
 *   rows   : host, cap rows of (1 + n_mats) doubles; n_rows receives the rows recorded.
 * Errors: SPAX_ERR_NULL, SPAX_ERR_PARAM (n_mats outside 1..64, alpha <= 0, P_max > 1, a
 * parameter count not finite and positive, alpha so small that taking every matrix to 1
 * would need more than 1e7 increments, or a block_error value that is not finite: *n_rows
 * then holds the rows recorded before it), SPAX_ERR_WORKSPACE (more rows than cap; *n_rows
 * then holds the number needed).
 */
int spax_greedy_allocation(const double* params, int32_t n_mats, double alpha, double P_max,
                           spax_block_error_fn block_error, void* user, double* rows,
                           int32_t cap, int32_t* n_rows);

/* The allocation recorded for a block target (Appendix D: allocations are recorded against
 * the block's overall sparsity): p = the first row of `rows` whose P >= target (the last row
 * if none; zeros for target <= 0).  Host only.  Errors: SPAX_ERR_NULL, SPAX_ERR_PARAM. */
int spax_allocation_at(const double* rows, int32_t n_rows, int32_t n_mats, double target,
                       double* p);

const char* spax_status_string(int status);
const char* spax_last_error(void);   /* thread-local; "" if none */
const char* spax_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SPAX_H */
