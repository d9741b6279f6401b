/*
 * smla.h -- sparse multi-head latent attention (MLA) decode over packed
 * fp8_ds_mla KV records, for NVIDIA GB300 (sm_103a).  C ABI of libsmla.so.
 *
 * What is computed follows these pages:
 *   [P1] "vllm.models.kimi_k3.amd.ops.flydsl_sparse_mla_gfx950" (FlyDSL sparse
 *        MLA forward over fp8_ds_mla records, gfx950): module docstring
 *        (record layout, CSR tiles and masking, preconditions, writer rule)
 *        and the epilogue of build_sparse_mla_fp8ds_module (output and LSE).
 *   [P2] "vllm.models.deepseek_v41.amd.mono.attention.back" (K2 back):
 *        stage_split (per-chunk partial, max, sum) and stage_combine (chunk
 *        merge with the per-head sink).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the current CUDA device.  The
 *     library never allocates, frees, or synchronises; every call is
 *     asynchronous on `stream` (a cudaStream_t passed as void*, NULL = the
 *     legacy default stream).  The caller owns every buffer.
 *   - Return value: SMLA_OK (0) or a negative smla_status.  Argument errors are
 *     detected on the host before anything is enqueued.  A non-zero status
 *     from a launch is SMLA_ERR_LAUNCH.  smla_strerror() names each code.
 *   - Integers are little-endian; strides are in elements of the tensor's type.
 */
#ifndef SMLA_H
#define SMLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Record layout, [P1] module docstring "Record (656 B)": bytes [0, 512) hold
 * 512 E4M3 latent values, [512, 528) four little-endian f32 power-of-two
 * scales (scale b covers latent dims [128 b, 128 b + 128)), [528, 656) the
 * 64 bf16 RoPE dims.  656 = 41 * 16, so every record is 16-byte aligned when
 * the cache base is. */
#define SMLA_RECORD_BYTES 656
#define SMLA_LATENT_DIM 512
#define SMLA_ROPE_DIM 64
#define SMLA_QK_DIM 576
#define SMLA_SCALE_BLOCK 128
#define SMLA_MAX_HEADS 64

typedef enum smla_status {
  SMLA_OK = 0,
  SMLA_ERR_NULL = -1,       /* a required pointer is NULL */
  SMLA_ERR_SHAPE = -2,      /* a size is out of range (n_q < 0, heads not in [1, 64], ...) */
  SMLA_ERR_STRIDE = -3,     /* a stride overlaps rows/heads or is negative */
  SMLA_ERR_ALIGN = -4,      /* a pointer or stride breaks the alignment rules below */
  SMLA_ERR_WORKSPACE = -5,  /* workspace missing or smaller than smla_decode_workspace_size */
  SMLA_ERR_SPLITS = -6,     /* num_splits outside [0, SMLA_MAX_SPLITS] */
  SMLA_ERR_DEVICE = -7,     /* no CUDA device, or the current device is not sm_103 */
  SMLA_ERR_LAUNCH = -8      /* a kernel launch failed (an error that was there before is none of its own) */
} smla_status;

/* Bits a decode call ORs into *status (when status != NULL). */
#define SMLA_STATUS_INDEX_OOB 0x1   /* an index >= n_kv_rows was met and masked */
#define SMLA_STATUS_TIMEOUT 0x2     /* an in-kernel pipeline wait gave up: results invalid */
#define SMLA_STATUS_SMEM_LAYOUT 0x4 /* the kernel could not align its shared memory and
                                       computed nothing: results invalid */
#define SMLA_STATUS_FOREIGN_SCALE 0x8 /* native-fp8 kernel: a gathered record holds a block
                                         scale that is neither zero nor a positive normal
                                         power of two (smla_pack_records never writes one);
                                         the rows holding it are not computed exactly: run
                                         SMLA_KERNEL_TENSOR_CORE_BF16 on such caches */

#define SMLA_MAX_SPLITS 64

/* Arguments of one decode call.
 *
 * Row r's keys are the CSR slice indices[indptr[r] : indptr[r + 1]] ([P1]
 * module docstring, "Tiles").  Its length is max(indptr[r+1] - indptr[r], 0),
 * further capped at max(lens[r], 0) when lens != NULL.  Position p of the
 * slice contributes iff its offset indptr[r] + p lies in [0, n_indices) and
 * 0 <= indices[offset] < n_kv_rows.  Entries < 0 are masked with or without
 * has_invalid ([P1] "Tiles": masked positions contribute nothing); an entry
 * >= n_kv_rows, which [P1] lists as a precondition the host cannot check, is
 * masked the same way here, never dereferenced, and flagged in *status.
 * Duplicate entries count once per position.
 *
 * For each row r and head h, over the contributing keys t:
 *   k_t[d] = e4m3(rec_t[d]) * scale_t[d / 128]   (d < 512), bf16 rope (512 <= d < 576)
 *   s_t    = sm_scale * sum_{d < 576} q[r, h, d] * k_t[d]
 *   m = max_t s_t,  l = sum_t exp(s_t - m)
 *   lse[r, h] = m + ln(l)                          ([P1] epilogue; the sink is
 *                                                  not part of the LSE)
 *   out[r, h, d] = sum_t exp(s_t - m) k_t[d] / (l + exp(sink[h] - m))   (d < 512)
 * with the sink term absent when sink == NULL (it enters the denominator once,
 * as [P2] stage_combine folds it).  A row with no contributing key gives
 * out = 0 and lse = -inf, sink or not ([P1] epilogue).
 *
 * Layouts and alignment:
 *   q        bf16, element [r][h][d] at q + r*q_stride_row + h*q_stride_head + d;
 *            16-byte aligned base, strides multiples of 8 elements.
 *   kv_cache uint8 [n_kv_rows][656], 16-byte aligned.  Row ids are 64-bit
 *            byte offsets, so caches beyond 4 GiB work; n_kv_rows <= 2^31.
 *   indices  int32 [n_indices]; indptr int32 [n_q + 1]; lens int32 [n_q] or NULL.
 *   sink     f32 [num_heads] or NULL, in the natural-log units of s_t.
 *   out      bf16, element [r][h][d] at out + r*out_stride_row + h*out_stride_head + d;
 *            16-byte aligned base, strides multiples of 8 elements.
 *   lse      f32 [n_q][num_heads] contiguous, or NULL.
 *   n_valid  int32 [n_q] or NULL: number of contributing keys of each row.
 *   status   int32 [1] or NULL: SMLA_STATUS_* bits are ORed in (never cleared).
 */
typedef struct smla_decode_params {
  int32_t n_q;
  int32_t num_heads;
  const void* q;
  int64_t q_stride_row;
  int64_t q_stride_head;
  const void* kv_cache;
  int64_t n_kv_rows;
  const int32_t* indices;
  int64_t n_indices;
  const int32_t* indptr;
  const int32_t* lens;
  /* Planning hints; results never depend on them.  max_row_len: an upper
   * bound of the rows' slice lengths known on the host (e.g. top-k); <= 0 means
   * unknown (n_indices / n_q is used).  has_invalid: rows may end in -1
   * padding ([P1] "Tiles", has_invalid).  Masked entries contribute nothing
   * either way; with has_invalid the tensor-core plan first trims each row to
   * its last entry >= 0 (a pass with a warp per row, plan.trim_kernel = 1) so
   * that the decode skips tiles of padding. */
  int32_t max_row_len;
  int32_t has_invalid;
  float sm_scale;
  const float* sink;
  void* out;
  int64_t out_stride_row;
  int64_t out_stride_head;
  float* lse;
  int32_t* n_valid;
  int32_t* status;
  /* Split-KV control ([P2] stage_split / stage_combine).  0 lets the planner
   * choose from the row length, the batch and the SM count.  k >= 1: the
   * CUDA-core kernel cuts every row into k chunks; the tensor-core kernel
   * spreads the tiles over n_q * k CTAs (about k parts per row). */
  int32_t num_splits;
  /* Which kernel runs the call (all compute the same definition):
   *   SMLA_KERNEL_TENSOR_CORE (0, default): the native-fp8 kernel for the head
   *     counts it supports (1..16), else the bf16 tensor-core kernel;
   *   SMLA_KERNEL_CUDA_CORE (1): an fp32 CUDA-core kernel kept as a cross-check;
   *   SMLA_KERNEL_TENSOR_CORE_BF16 (2): tcgen05 kind::f16 on latents dequantised
   *     to bf16 (exact for power-of-two scales up to 2^7, any scale accepted);
   *   SMLA_KERNEL_TENSOR_CORE_FP8 (3): tcgen05 kind::mxf8f6f4 on the E4M3 bytes as
   *     they are, the block scales as E8M0 scale factors (heads 1..16; a call
   *     with more heads returns SMLA_ERR_SHAPE).  Needs writer-format scales:
   *     zero or positive normal powers of two; others set
   *     SMLA_STATUS_FOREIGN_SCALE. */
  int32_t kernel;
} smla_decode_params;

#define SMLA_KERNEL_TENSOR_CORE 0
#define SMLA_KERNEL_CUDA_CORE 1
#define SMLA_KERNEL_TENSOR_CORE_BF16 2
#define SMLA_KERNEL_TENSOR_CORE_FP8 3

/* How a decode call with given params is laid out on the GPU.
 *
 * Tensor-core kernels (bf16: tile_len 64; native fp8: tile_len 128): a
 * persistent, balanced schedule.  Each row r is cut into
 * T_r = max(1, ceil(len_r / tile_len)) tiles of tile_len slice positions
 * and takes s + k T_r slots of a schedule space, rows in order (s slots stand
 * for the cost of starting a row: its epilogue and q staging; bf16 kernel:
 * k = 1 slot per tile and s = 2; native-fp8 kernel: k = 2, s = 1, i.e. half
 * a tile), so that tile t of row r starts at slot R_r + k t with
 * R_r = s + sum_{r' < r} (s + k T_r').  CTA c of G = grid takes the slots
 * [b_c, e_c) with b_c = floor(c W / G), W the slot total, and the tiles whose
 * first slot lies there, and streams through them across row boundaries.
 * A row lying wholly inside one CTA's range is finished there; a row shared
 * by CTAs c_a..c_b (the CTAs holding its first and last tile) gets
 * one partial per CTA, stored in workspace slot 2 c + (R_r < b_c ? 0 : 1), and
 * is merged from those slots ([P2] stage_combine).  bf16 kernel: by a second,
 * small kernel launched right after (merge_kernel = 1 whenever grid > 1; a
 * warp merges one head of a row).  Native-fp8 kernel (with more than 32
 * heads two CTAs, head groups of 32, share each slot range): a row of up to 4
 * parts is merged inside the decode launch by the CTA whose part arrives last
 * (per-row ticket); when the other parts had all arrived before that CTA's
 * final part ended, it merges from its own O without writing that part's
 * partial.  Rows of more parts, possible only when ceil(grid / n_q) + 1 > 4,
 * are left to the merge kernel (merge_kernel = 1 then).
 * CUDA-core kernel: one CTA per (row, chunk); chunk c of a row covers slice
 * positions [c chunk_len, (c + 1) chunk_len), the last chunk everything after;
 * partial slot r * num_splits + c; the last chunk to finish merges.
 *
 * Tensor-core kernel with has_invalid: a pass before the decode (warp per
 * row, 512 slice positions per step from the end) writes each row's length
 * trimmed to its last entry >= 0 into the workspace, and the decode schedules
 * those lengths (trim_kernel = 1).
 *
 * Fields: kernel (the SMLA_KERNEL_* that runs: 1, 2 or 3), grid (CTAs of the decode launch), tile_len
 * (keys per tile), num_splits and chunk_len (CUDA-core kernel only),
 * partial_slots, merge_kernel, trim_kernel, workspace_bytes.  num_sms > 0 makes the plan
 * pure host arithmetic (no CUDA call); num_sms = 0 asks the current device. */
typedef struct smla_plan_info {
  int32_t kernel;
  int32_t grid;
  int32_t tile_len;
  int32_t num_splits;
  int32_t chunk_len;
  int32_t partial_slots;
  int32_t merge_kernel;
  int32_t trim_kernel;
  int32_t head_groups;
  int64_t workspace_bytes;
} smla_plan_info;

int smla_plan(const smla_decode_params* params, int32_t num_sms, smla_plan_info* plan);

/* Workspace bytes smla_decode needs for these params on the current device
 * (0 when none; also 0 for invalid params).
 *
 * Layout (each part 256-byte aligned), S = plan.partial_slots:
 *   ticket   int32 [2 n_q]       per-row (and head group) arrival counters (CUDA-core and
 *                                native-fp8 kernels)
 *   row_tile int64 [n_q + 1]     tensor-core kernel: first slot of every row, then W
 *   o_part   f32 [S][H][512]     unnormalised partial sum_t 2^(x_t - m) v_t of a row part
 *   ml_part f32 [S][H][2]        (m, l) of x_t = s_t * log2(e): m is the part's reference
 *                                maximum (its max, or at most 24 (bf16 kernel) or 16 (native
 *                                fp8) below it), l = sum_t 2^(x_t - m);
 *                                m = -inf, l = 0 for a part without keys
 *   nv_part int32 [S]            contributing keys of the part
 *   lens    int32 [n_q]          trimmed row lengths (only when plan.trim_kernel)
 * The ticket counters must be zero when a call starts (e.g. allocate the
 * workspace zeroed); every completed call returns them to zero.  A call with
 * other sizes may have written partials over that region, so re-zero bytes
 * [0, 8 n_q) before reusing a workspace across calls of different n_q,
 * num_heads, kernel or plan.  Calls that share a workspace must be ordered
 * (same stream); a call that reports SMLA_STATUS_TIMEOUT leaves it undefined. */
size_t smla_decode_workspace_size(const smla_decode_params* params);

/* Sparse MLA decode (the definition above): one decode launch, preceded by
 * the row-trim pass when plan.trim_kernel = 1 and followed by the merge kernel
 * when plan.merge_kernel = 1.  Each CTA gathers its tiles' records,
 * dequantises them to bf16 (exact), runs QK over 576 dims and PV over 512 dims
 * on the tcgen05 tensor cores with an online softmax in between, and writes
 * out / lse of its whole rows and partials of shared rows (see smla_plan).
 * `workspace` may be NULL only when smla_decode_workspace_size() returns 0.
 * Accuracy: q, k and v enter the products exactly when every block scale is a
 * positive normal power of two up to 2^7 (all scales smla_pack_records
 * writes); a block with any other f32 scale (zero, negative, not a power of
 * two, above 2^7) has each latent value e4m3 * scale formed in f32 and
 * rounded once to bf16 (exact where that product is a bf16), on a slower
 * path.  p is rounded to bf16, sums are f32, out is rounded to bf16 (round to
 * nearest even). */
int smla_decode(const smla_decode_params* params, void* workspace, size_t workspace_bytes,
                void* stream);

/* Bytes of the fixed device array behind smla_decode_noalloc: 64 MiB per
 * device.  A default tensor-core plan on a 152-SM GPU needs about 40 MiB at 64
 * heads (304 partial slots x 64 heads x 2 KiB) plus 12 bytes per query row. */
#define SMLA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* smla_decode without a caller-supplied workspace, for callers that cannot
 * allocate device memory at call time: code running inside another runtime's
 * memory pool or allocation-free serving loop, where a cudaMalloc (or a
 * framework allocation) on the call path is not allowed or would stall other
 * work.  The pages describe no such entry point; it is an addition of this
 * library.
 *
 * Same params, outputs, accuracy and launches as smla_decode; the split-KV
 * workspace (the layout of smla_decode_workspace_size) lives instead in a
 * file-scope device array of SMLA_NOALLOC_SCRATCH_BYTES bytes inside
 * libsmla.so.  The call allocates nothing.
 *   - Set-up: the first call on a device (the current device) looks up the
 *     device address of that array once (cudaGetSymbolAddress, which may load
 *     the library's module on that device).  Make that first call before any
 *     stream capture.
 *   - Limit: a call whose workspace would exceed SMLA_NOALLOC_SCRATCH_BYTES
 *     returns SMLA_ERR_WORKSPACE and launches nothing (use smla_decode with a
 *     workspace of smla_decode_workspace_size bytes instead).
 *   - Sharing: every call on a device uses the same array and leaves its last
 *     contents there.  Calls whose work may overlap on the GPU (different
 *     streams without an ordering event) race on it and give wrong results;
 *     order them.  With the CUDA-core and native-fp8 kernels the call first
 *     clears the ticket counters (bytes [0, 8 n_q)) on `stream`; the bf16
 *     tensor-core kernel writes every part of the array it reads and needs
 *     nothing cleared.
 * Errors as smla_decode, plus SMLA_ERR_DEVICE when the set-up fails. */
int smla_decode_noalloc(const smla_decode_params* params, void* stream);

/* The record writer ([P1] module docstring, "Preconditions": vLLM's
 * concat_and_cache_ds_mla rule).  For each of n records:
 *   scale_b = pow2ceil(max(amax_b, 1e-4) / 448), amax_b = max |latent[128 b .. 128 b + 127]|
 *   bytes [0, 512)   = E4M3(latent_d / scale_{d/128}), round to nearest even, saturating
 *   bytes [512, 528) = the four scales as f32
 *   bytes [528, 656) = the 64 rope bf16 values, bit for bit
 * latent: bf16 [n][latent_stride] (first 512 used), rope: bf16 [n][rope_stride]
 * (first 64 used), kv_out: uint8 [n][656].  Pointers 16-byte aligned, strides
 * multiples of 8 elements.  scale <= 2^7 holds iff |latent| <= 57344. */
int smla_pack_records(const void* latent, int64_t latent_stride, const void* rope,
                      int64_t rope_stride, int64_t n, void* kv_out, void* stream);

/* ---- The paged cache: write, read back, attend ------------------------------
 *
 * A paged cache holds records in n_pages pages of page_size records each (the
 * record layout above); sequences own pages through a block table.  With
 * page_stride == page_size * SMLA_RECORD_BYTES the cache is also the flat
 * cache of smla_decode, a record's row id being page * page_size + offset.
 *
 * Batch: sequence b owns the token rows cu_rows[b] .. cu_rows[b + 1] - 1 of the
 * token tensors (latent, rope, q, out, lse), which are its positions up to
 * seq_lens[b] - 1:
 *   position of row r of sequence b = seq_lens[b] - (cu_rows[b + 1] - r).
 * Position p lives in page block_table[b][p / page_size] at offset
 * p % page_size.  A position < 0, past the table's max_pages pages, or in a
 * page whose id is < 0 or >= n_pages is masked: its record is neither read
 * nor written.  Ids >= n_pages and positions past the table set
 * SMLA_STATUS_INDEX_OOB; negative ids are padding and set nothing.  Token rows
 * of no sequence are left as they are.  cu_rows must not decrease; values
 * outside [0, n_rows] are clamped.
 *
 * Layouts and alignment: kv_cache uint8, 16-byte aligned; page_stride (bytes)
 * a multiple of 16, at least page_size * SMLA_RECORD_BYTES; block_table int32
 * [n_seqs][block_table_stride], max_pages entries used; cu_rows int32
 * [n_seqs + 1]; seq_lens int32 [n_seqs]; n_rows the rows of the token tensors;
 * status int32 [1] or NULL.  max_pages * page_size <= 2^30, n_rows <= 2^30,
 * n_seqs <= 2^24.
 * All of it is device memory and read on the device: a captured graph may be
 * replayed with other tables, lengths and row splits in the same buffers. */
#define SMLA_DTYPE_BF16 0
#define SMLA_DTYPE_F16 1
#define SMLA_DTYPE_F32 2

typedef struct smla_paged_batch {
  void* kv_cache;
  int64_t n_pages;
  int64_t page_stride;
  int32_t page_size;
  int32_t max_pages;
  const int32_t* block_table;
  int64_t block_table_stride;
  const int32_t* cu_rows;
  const int32_t* seq_lens;
  int64_t n_rows;
  int32_t n_seqs;
  int32_t* status;
} smla_paged_batch;

/* Writes every token row's record at its position: the rule of
 * smla_pack_records (bit for bit for finite bf16 inputs) for latent and rope of
 * type dtype, values in f32 and rope rounded to bf16 (nearest even).  A NaN
 * latent is stored as the NaN code and does not enter its block's scale.  An
 * infinity counts as the largest f32 there: the block's scale becomes 2^120,
 * the infinity is stored as +-448 times that (and read back as +-inf), and the
 * block's values up to 2^110 become zeros of their sign.
 * latent [n_rows][latent_stride] (512 used), rope [n_rows][rope_stride] (64
 * used), 16-byte aligned, strides multiples of 16 bytes.  The rows' positions
 * have to lie in different slots: of two rows that a block table sends to one
 * slot, either's bytes may remain there. */
int smla_paged_write(const smla_paged_batch* batch, const void* latent, int64_t latent_stride, const void* rope,
                     int64_t rope_stride, int32_t dtype, void* stream);

/* Reads every token row's record back: latent[r][d] = e4m3 * scale (the f32
 * product, rounded once to dtype), rope[r] converted to dtype.  A row whose
 * position is masked gets zeros.  A whole history is read with
 * cu_rows[b + 1] - cu_rows[b] = seq_lens[b]; a part of it that ends at position
 * e with seq_lens[b] = e.  Layouts as smla_paged_write. */
int smla_paged_read(const smla_paged_batch* batch, void* latent, int64_t latent_stride, void* rope,
                    int64_t rope_stride, int32_t dtype, void* stream);

#define SMLA_PAGED_MAX_HEADS 128

/* Attention of the token rows over their sequences' records.  For row r of
 * sequence b at position p, the visible keys are the unmasked positions
 * t <= p (causal = 1) or t < seq_lens[b] (causal = 0); with k_t, s_t, the sink,
 * out and lse as in smla_decode.  A row without a visible key gives out = 0 and
 * lse = -inf.  A visible score of -inf (q or a key's rope infinite) weighs
 * nothing: a row that has no other ends like a row without a visible key.  A
 * score of +inf or NaN makes the row's out and lse NaN.  A sink of +inf gives
 * out = 0 (unless the row is NaN), one of -inf changes nothing.  A visible
 * record whose latent holds a value that is not finite (a NaN code, a scale that
 * is not finite) makes the row's out and lse NaN; what a row may not see never
 * reaches it.
 *
 * q bf16 [n_rows][num_heads][576] and out bf16 [n_rows][num_heads][512] with
 * strides as in smla_decode (16-byte aligned, strides multiples of 8); sink f32
 * [num_heads] or NULL; lse f32 [n_rows][num_heads] contiguous or NULL;
 * num_heads in [1, SMLA_PAGED_MAX_HEADS]; sm_scale * log2(e) finite in f32
 * (SMLA_ERR_SHAPE otherwise).  The records of the token rows
 * themselves are read from the cache like all others: write them first.
 * Accuracy as the bf16 tensor-core kernel of smla_decode (k and v enter the
 * products as bf16(e4m3 * scale), exact for scales 2^-116 .. 2^7; p is rounded
 * to bf16; sums, maxima and the softmax statistics are f32).
 * One kernel serves a call, chosen by the mean rows (n_rows * num_heads /
 * n_seqs) of its sequences: up to 16, up to 64, or more.  Results do not depend
 * on it beyond rounding, times do.  Empty and padding sequences count in n_seqs:
 * pass as many as there are where a chunk matters.  A batch of many single tokens
 * and a long chunk may be faster as two calls.  Time also grows by up to 2.6 us
 * for every 1000 sequences, empty or not. */
typedef struct smla_paged_attend_params {
  smla_paged_batch batch;
  int32_t num_heads;
  int32_t causal;
  const void* q;
  int64_t q_stride_row;
  int64_t q_stride_head;
  float sm_scale;
  const float* sink;
  void* out;
  int64_t out_stride_row;
  int64_t out_stride_head;
  float* lse;
} smla_paged_attend_params;

/* Workspace bytes of smla_paged_attend for these params on the current device
 * (0 for invalid params and empty batches).  It depends on the sizes alone
 * (num_heads, n_rows, n_seqs, page_size, max_pages) and never grows when n_rows,
 * n_seqs, page_size or max_pages shrinks: a workspace for a server's largest batch
 * serves all of its calls of as many heads.  It needs no initial contents and is
 * 256-byte aligned.  Calls that may overlap on the GPU need workspaces
 * of their own. */
size_t smla_paged_attend_workspace_size(const smla_paged_attend_params* params);

int smla_paged_attend(const smla_paged_attend_params* params, void* workspace, size_t workspace_bytes, void* stream);

/* ---- New rows with their rotation, trees of drafted tokens -------------------
 *
 * Serving calls around smla_paged_attend.  A step over plain tokens is
 * smla_paged_append, smla_paged_attend; one that verifies drafted trees is
 * smla_paged_tree, smla_paged_append, smla_paged_attend_tree, smla_paged_accept.
 * All lengths, boundaries and trees are read on the device. */

/* Turns of the 32 rope pairs per position, as fractions of 2^64 modulo a whole turn
 * (two's complement), from the angles inv_freq in radians: host arithmetic on host
 * arrays of 32 entries, within 2^-64 turns plus 2^-100 of the angle.  |inv_freq| <= 2^32
 * (SMLA_ERR_SHAPE otherwise, also for a NaN). */
int smla_rotation_turns(const double* inv_freq, uint64_t* turns);

/* smla_paged_write with the rope of keys and queries rotated on the way.  With t the
 * turn of pair k at a row's rotation position, p * inv_freq[k] radians,
 *   (x, y) -> rope_scale * (x cos t - y sin t, x sin t + y cos t),
 * the pair being dims 2k and 2k + 1 (interleaved) or k and k + 32.  Whole turns drop out
 * exactly at every int32 position (but for the table's 2^-64 of a turn, times the position);
 * what is left of the angle is cut after 2^-32 of a turn and rounded to f32, by 2^-26 of a
 * turn at most.  Cosine, sine and the products are f32, and each result is rounded once to bf16.
 *   latent, rope, dtype  as in smla_paged_write (rope before the rotation)
 *   turns       device, smla_rotation_turns
 *   rope_scale  finite; it enters cosine and sine
 *   positions   int32 [n_rows] on the device, rotation positions of the rows (of a tree's
 *               nodes: smla_paged_tree), or NULL: the rows' positions in the cache.  Where
 *               a record is stored does not depend on it.
 *   q_rope      [n_rows][num_heads][64] of type dtype -> q_out, bf16, e.g. the last 64 dims
 *               of smla_paged_attend's q; 16-byte aligned, strides multiples of 16 bytes.
 *               They may be the same bf16 memory, with the same strides; another overlap
 *               is undefined.  num_heads = 0: no queries.
 * Rows of no sequence are left alone, in q_out too.  A row whose record is masked has
 * its queries rotated all the same. */
typedef struct smla_paged_append_params {
  smla_paged_batch batch;
  const void* latent;
  int64_t latent_stride;
  const void* rope;
  int64_t rope_stride;
  int32_t dtype;
  int32_t interleaved;
  const uint64_t* turns;
  float rope_scale;
  int32_t num_heads;
  const int32_t* positions;
  const void* q_rope;
  int64_t q_rope_stride_row;
  int64_t q_rope_stride_head;
  void* q_out;
  int64_t q_out_stride_row;
  int64_t q_out_stride_head;
} smla_paged_append_params;

int smla_paged_append(const smla_paged_append_params* params, void* stream);

/* Masks and positions of drafted trees.  The token rows of sequence b are the nodes
 * 0, 1, ... of its tree, a parent before its children; parents[r] is the node that row r
 * hangs on, or negative for a root (there may be several).  For node i
 *   mask[r], bit j % 32 of word j / 32 = node j is i or an ancestor of i
 *   positions[r] = (position of node 0) + (number of ancestors of i)
 * A parent that is not a lower node makes its row a root and sets
 * SMLA_STATUS_INDEX_OOB; so does a node that its masks' words cannot hold, whose bit is
 * left out.  All words of the rows of a sequence are written; rows of no sequence
 * are left alone.  mask uint32 [n_rows][mask_stride], mask_words used, or NULL with
 * mask_words = 0; positions int32 [n_rows] or NULL.  The time grows with the depth. */
int smla_paged_tree(const int32_t* parents, const int32_t* cu_rows, const int32_t* seq_lens, int64_t n_rows,
                    int32_t n_seqs, uint32_t* mask, int64_t mask_stride, int32_t mask_words, int32_t* positions,
                    int32_t* status, void* stream);

/* smla_paged_attend where the token rows of a sequence see each other by masks: of the
 * sequence's row j, a row sees the key if bit j % 32 of word j / 32 of its mask is set,
 * and of earlier positions all.  Rows behind the masks' words are not seen; bits behind the
 * sequence's rows mean nothing.  With causal = 1 a row in addition sees no position
 * behind its own (in the cache), which for smla_paged_tree's masks changes no result and
 * passes over the keys of later nodes.  A row that sees
 * nothing gives out = 0 and lse = -inf; what a row may not see never reaches it.  mask
 * uint32 [n_rows][mask_stride], mask_words used (NULL with mask_words = 0: the history
 * alone).  Workspace, accuracy and the choice of the kernel as smla_paged_attend. */
int smla_paged_attend_tree(const smla_paged_attend_params* params, const uint32_t* mask, int64_t mask_stride,
                           int32_t mask_words, void* workspace, size_t workspace_bytes, void* stream);

/* Keeps the accepted path of each tree: path[b] names nodes of sequence b, rising, and the
 * record of its i-th node moves to the position of node 0 plus i (byte for byte, so that
 * the rotation, made for that depth, holds); new_lens[b] = position of node 0 + number of
 * nodes accepted.  The path ends at its first negative entry (padding), or at one
 * that is no node of the tree or does not rise, which sets SMLA_STATUS_INDEX_OOB.
 * A record whose old or new place is masked stays where it is.  Records of the tree behind
 * the accepted ones are left as they are.  path int32 [n_seqs][path_stride],
 * path_len used; new_lens int32 [n_seqs], which may be the batch's seq_lens; the batch's
 * n_rows clamps the boundaries as in the other calls, and with none of it every new length
 * is the old one.  As in smla_paged_write, the rows' positions have to lie in different
 * slots. */
int smla_paged_accept(const smla_paged_batch* batch, const int32_t* path, int64_t path_stride, int32_t path_len,
                      int32_t* new_lens, void* stream);

/* Name of a status code. */
const char* smla_strerror(int status);

/* SMLA_OK when the current CUDA device can run the kernels (sm_103). */
int smla_device_check(void);

/* Limit, in ns, of every in-kernel pipeline wait of the tensor-core kernels
 * launched after this call on the current device (process-wide); 0 restores
 * the default of 2 s.  (In smla_paged_attend's kernel for more than 64 rows a sequence
 * it is the time within which a pair of CTAs has to get on to its next tile of keys,
 * whichever wait that is; a pair that then still stands ends after 2 s more.)
 * A wait that runs out sets SMLA_STATUS_TIMEOUT: the CTA
 * then skips its remaining waits, still issues its pending copies and MMAs,
 * waits (2 s at most each) until they have completed, frees its tensor memory
 * and exits, so that the CUDA context stays usable.  out, lse, n_valid and the
 * workspace are then undefined (re-zero the ticket region before the next
 * call).  stall_first_wait = 1 makes the first softmax wait of every CTA wait
 * on a barrier that nothing signals, so that it runs out after the limit: a
 * test of that path, with no fault and no hang; 0 for normal operation.
 * Returns SMLA_ERR_DEVICE off sm_103, SMLA_ERR_LAUNCH when the values cannot
 * be set. */
int smla_set_wait_limit(uint64_t limit_ns, int stall_first_wait);

#ifdef __cplusplus
}
#endif

#endif /* SMLA_H */
