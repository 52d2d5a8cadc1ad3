/*
 * gqa.h -- C ABI of libgqa: grouped-query attention kernels for NVIDIA GB300
 * (sm_103a), head_dim 128, 32 query heads over 8 KV heads (4 query heads per
 * KV head); for paged caches of other layouts the append, the attention of one
 * token and what a step with drafted tokens needs (their masks, their attention
 * and the compaction of the accepted ones), whose descriptors give the sizes.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers.  Every tensor argument is a plain pointer to a dense, row-major
 * (C-contiguous) array with the shape stated below; the entry points of other
 * cache layouts (gqa_paged_append_t, gqa_paged_norm_append_t,
 * nvfp4_paged_append_t, nvfp4_paged_norm_append_t, gqa_paged_attn_t,
 * gqa_paged_window_attn_t, gqa_paged_tree_attn_t, gqa_paged_keep_t) also take
 * strided ones, and they and gqa_tree_mask_t device memory only.  All tensor
 * pointers of one call must be either
 *   - device memory of one and the same CUDA device (cudaMalloc'd, managed,
 *     or a PyTorch CUDA tensor's data pointer): the call enqueues its kernels
 *     on `stream` and returns without synchronising; or
 *   - host memory (pageable or pinned): the call stages the inputs into a
 *     library-owned device buffer on the calling thread's current device,
 *     runs the same kernels on `stream`, copies the output back, and
 *     synchronises `stream` before returning.
 * Mixing host and device pointers, or device pointers of two devices, is
 * rejected with GQA_ERR_DEVICE_MISMATCH.  Device pointers must be 16-byte
 * aligned (GQA_ERR_INVALID_ARG otherwise).
 *
 * Device selection.  For device pointers the call switches to the pointers'
 * device for its duration and restores the caller's current device on
 * return; the caller's current device need not match.  (The launcher
 * conventions of "FlashInfer NVFP4 QKV GEMM 최적화: SM103a Epilogue 통합 및 CUDA
 * 런처 개선", section 2: all tensors on one device, scoped device switch, no
 * current-device check, positive launch grid.)
 *
 * Ownership.  The caller owns every tensor.  The library owns a grow-only
 * scratch workspace per (device, stream), released by
 * gqa_release_workspace().  Two calls on the same stream are ordered by the
 * stream; calls on different streams use different workspaces.
 * cudaStreamPerThread counts as one stream of each host thread;
 * the workspaces of gqa_paged_attn_t, gqa_paged_window_attn_t and
 * gqa_paged_tree_attn_t for it are released when the thread ends.  Of these two
 * attentions' own workspaces, which never move, one takes 5.7 MB and the other 45 MB
 * on each stream that they are called on without one (what the largest head layout
 * needs); a workspace that is given may be smaller.
 *
 * Errors.  Every entry point returns a gqa_status; GQA_OK means the work was
 * validated and enqueued (device pointers) or completed (host pointers).  On
 * any other status nothing was launched, and gqa_last_error() returns a
 * thread-local message.  No C++ exception crosses this boundary.
 */
#ifndef GQA_H_
#define GQA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA runtime headers; 0 is the legacy
 * default stream. */
typedef struct CUstream_st* gqa_stream_t;

typedef enum gqa_status {
  GQA_OK = 0,
  GQA_ERR_INVALID_ARG = 1,        /* null pointer, bad size, dtype or strides, misalignment */
  GQA_ERR_UNSUPPORTED = 2,        /* shape outside what the kernels handle */
  GQA_ERR_UNSUPPORTED_SHAPE = 2,  /* (the same code, by the name the descriptor entry points use) */
  GQA_ERR_DEVICE_MISMATCH = 3,    /* pointers on different devices / host+device mix */
  GQA_ERR_CUDA = 4,               /* a CUDA runtime call failed */
  GQA_ERR_OOM = 5,                /* workspace allocation failed */
  GQA_ERR_TIMEOUT = 6,            /* a kernel's bounded wait expired (see gqa_check_device_errors) */
  GQA_ERR_WORKSPACE = 7           /* a captured call without a workspace (see gqa_paged_attn_t, gqa_paged_tree_attn_t) */
} gqa_status;

/*
 * Tensor descriptor of the *_t entry points below: the pointer entry points'
 * arguments plus what a C caller would otherwise have to get right unaided --
 * element type, placement, shape and strides -- so that the library can
 * check them (a DLPack-like record of our own).
 *
 *   data     first element (device or host memory)
 *   dtype    a gqa_dtype
 *   device   CUDA device ordinal of `data`, or -1 for host memory; checked
 *            against where the memory really is
 *   ndim     number of dimensions (<= 6)
 *   shape    extents; strides in elements, dense row-major required (a
 *            dimension of extent 1 may carry any stride)
 */
typedef enum gqa_dtype {
  GQA_F16 = 1,   /* IEEE binary16 */
  GQA_E4M3 = 2,  /* OCP FP8 E4M3 ("fn") bytes */
  GQA_U8 = 3,    /* bytes: packed E2M1 pairs, or E4M3 codes given as raw bytes */
  GQA_I32 = 4,
  GQA_F32 = 5,
  GQA_BF16 = 6   /* bfloat16 */
} gqa_dtype;

typedef struct gqa_tensor {
  void* data;
  int32_t dtype;
  int32_t device;
  int32_t ndim;
  int64_t shape[6];
  int64_t strides[6];
} gqa_tensor;

/* Message for the last non-OK status returned on this thread. */
const char* gqa_last_error(void);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int gqa_version(void);

/*
 * gqa_decode -- FP16 grouped-query attention for one new token per sequence.
 *
 * Defined by "NVIDIA SM110 GPU를 위한 실험적인 FP16 GQA 디코드 커널 추가",
 * section 1 (the sm110_gqa_decode API and its docstring) and section 3 (the
 * scaled_dot_product_attention comparator with enable_gqa=True):
 *
 *   out[b,h,:] = sum_t softmax_t(s) * V[b,g,t,:],   g = h / 4,
 *   s_t = (q[b,h,:] . K[b,g,t,:]) * q_scale / sqrt(128),   0 <= t < len_b,
 *   K = kv[b,0,...], V = kv[b,1,...],  len_b = clamp(seq_lens[b], 0, capacity).
 *
 *   q         [batch, 32, 128]                 float16
 *   kv        [batch, 2, 8, capacity, 128]     float16 (K stacked over V)
 *   seq_lens  [batch]                          int32 (read by the kernels)
 *   out       [batch, 32, 128]                 float16, written; caller-owned
 *   batch     1 .. 65535
 *   capacity  1 .. 2^31 - 1 tokens per sequence
 *   q_scale   finite; multiplies the standard 1/sqrt(128) scale
 *
 * A sequence of length 0 produces a zero row.  Element offsets are computed
 * in 64-bit, so kv may hold 2^31 or more elements.
 */
gqa_status gqa_decode(const void* q, const void* kv, const int32_t* seq_lens, void* out, int64_t batch,
                      int64_t capacity, float q_scale, gqa_stream_t stream);

/*
 * gqa_decode_noalloc -- gqa_decode that allocates no memory.  (An addition
 * of this library; the pages have no counterpart.)
 *
 * Same operation, arguments, layouts and results as gqa_decode, for callers
 * that cannot allocate device memory at call time: engines that reserve
 * nearly all of HBM up front for their KV cache and own every byte through
 * their own allocator (a late cudaMalloc would fail or fragment it), and
 * latency-critical loops that must not block in cudaMalloc/cudaFree, which
 * can synchronise the device.  The split partials go to a file-scope device
 * array of 16 MiB instead of the library workspace; every GPU that loads
 * libgqa holds that array until the process exits.
 *
 *   - Device pointers only (host buffers would need staging memory):
 *     GQA_ERR_UNSUPPORTED otherwise.
 *   - Rejects, with GQA_ERR_UNSUPPORTED and a message naming the sizes, a
 *     (batch, capacity) whose partials exceed 16 MiB: batch * 32 * splits *
 *     520 bytes, splits as reported by gqa_decode_plan.  The benchmark shapes
 *     (64 x 8192, 8 x 131072) need 8.5 MB.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) and caches it with the device's current CUDA
 *     context; a call that finds another context current (after
 *     cudaDeviceReset, which reloads the library's device code) looks it up
 *     again.  Make the first call on a device, and the first after a reset,
 *     before any stream capture.
 *   - Every call on a device shares the one array and leaves its contents
 *     behind (nothing in it needs to start at zero).  Calls whose kernels
 *     overlap on the GPU -- on different streams, without ordering -- race on
 *     it; order them on one stream or with events.
 *   - Calls no cudaMalloc, cudaFree or allocating library routine.
 */
gqa_status gqa_decode_noalloc(const void* q, const void* kv, const int32_t* seq_lens, void* out, int64_t batch,
                              int64_t capacity, float q_scale, gqa_stream_t stream);

/*
 * gqa_decode_paged -- the operation of gqa_decode over a paged K/V cache:
 * the same split-KV kernels, each 16-token K/V tile gathered through the
 * block table ("NVIDIA SM110 GPU를 위한 실험적인 FP16 GQA 디코드 커널 추가",
 * section 1, for the operation; the page layout is the one the context
 * attention uses, "GB300 NVFP4 Context Attention: scale slot 조기 반납과 8단
 * packed K/V ring", introduction, with fp16 values).
 *
 *   q            [batch, 32, 128]                 fp16
 *   k_pages      [num_pages, 8, 64, 128]          fp16, HND: page p, KV head g,
 *   v_pages      [num_pages, 8, 64, 128]          slot s holds token 64*p' + s
 *                of the sequence whose block_table row maps logical page p'
 *                to p
 *   block_table  [batch, max_pages_per_seq]       int32; entries for logical
 *                pages < ceil(len_b / 64) must be in [0, num_pages)
 *   seq_lens     [batch]                          int32, read on the device,
 *                clamped to [0, 64 * max_pages_per_seq]
 *   out          [batch, 32, 128]                 fp16, written
 *
 * Splits as gqa_decode_plan(batch, 64 * max_pages_per_seq) reports.  Same
 * placement rules as gqa_decode (one device, or all host buffers: staged,
 * synchronous, table entries checked on the host).  A page index outside
 * [0, num_pages) met on the device is not read: page 0 is used instead and
 * bit 1 of the error word (gqa_check_device_errors) is set.  Errors:
 * GQA_ERR_UNSUPPORTED for batch outside [1, 65535], GQA_ERR_INVALID_ARG for
 * bad sizes, NULL or misaligned pointers, a non-finite q_scale.
 */
gqa_status gqa_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                            const int32_t* seq_lens, void* out, int64_t batch, int64_t num_pages,
                            int64_t max_pages_per_seq, float q_scale, gqa_stream_t stream);

/*
 * Descriptor forms of gqa_decode, gqa_decode_paged and nvfp4_paged_ctx_attn:
 * the same operations, with every tensor given as a gqa_tensor.  Before any
 * CUDA work they check each descriptor's dtype, rank, shape (including the
 * extents the tensors share: batch, pages, total_q), dense row-major strides
 * and non-null data -- GQA_ERR_INVALID_ARG, or GQA_ERR_UNSUPPORTED_SHAPE for
 * an extent the kernels do not handle (32 query heads, 8 KV heads, head dim
 * 128, 64-token pages) -- then that all tensors share one `device` field and
 * that the memory really is there (GQA_ERR_DEVICE_MISMATCH); then they call
 * the pointer form with the sizes read from the shapes.  Accepted dtypes:
 * q/kv/out/pages of the decodes GQA_F16; q_fp8, k_sf, v_sf, out_fp8 GQA_E4M3
 * or GQA_U8; k_fp4, v_fp4 GQA_U8; seq_lens, block_table, qo_indptr, kv_lens
 * GQA_I32.  Shapes as in the pointer forms' comments.
 */
gqa_status gqa_decode_t(const gqa_tensor* q, const gqa_tensor* kv, const gqa_tensor* seq_lens, gqa_tensor* out,
                        float q_scale, gqa_stream_t stream);
gqa_status gqa_decode_paged_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                              const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out,
                              float q_scale, gqa_stream_t stream);
gqa_status nvfp4_paged_ctx_attn_t(const gqa_tensor* q_fp8, float q_scale, const gqa_tensor* k_fp4,
                                  const gqa_tensor* k_sf, const gqa_tensor* v_fp4, const gqa_tensor* v_sf,
                                  const gqa_tensor* block_table, const gqa_tensor* qo_indptr,
                                  const gqa_tensor* kv_lens, gqa_tensor* out_fp8, float out_scale,
                                  gqa_stream_t stream);

/*
 * gqa_decode_plan -- how gqa_decode splits the KV sequence for a given batch
 * and capacity (chosen from these two only; the lengths stay on the device):
 * *tokens_per_split tokens per split CTA, *num_splits splits per sequence,
 * *num_launches kernels per call (1 when one split covers the capacity: the
 * split kernel then writes the output itself; 2 otherwise: split + merge).
 * Any output pointer may be NULL.
 */
gqa_status gqa_decode_plan(int64_t batch, int64_t capacity, int32_t* tokens_per_split, int32_t* num_splits,
                           int32_t* num_launches);

/*
 * nvfp4_paged_ctx_attn -- paged context (prefill) attention with FP8-E4M3
 * query and output and NVFP4 K/V pages, bottom-right causal.
 *
 * Defined by "GB300 NVFP4 Context Attention: scale slot 조기 반납과 8단 packed
 * K/V ring", introduction: FP8 (E4M3) query/output, NVFP4 K/V pages with
 * E4M3 block scales, dequantised to E4M3 in shared memory, head dim 128,
 * bottom-right causal mask, HND page layout.  For sequence b with
 * q_len_b = qo_indptr[b+1] - qo_indptr[b] and kv_len_b = kv_lens[b], query i
 * (row qo_indptr[b] + i) sees key j iff j <= kv_len_b - q_len_b + i, and
 *
 *   Kq[b,g,j,d] = E4M3_rne_sat( e2m1(code) * e4m3(scale) )   (same for Vq)
 *   s_j  = (q[row,h,:] . Kq[b,g,j,:]) * q_scale / sqrt(128),  g = h / 4
 *   out[row,h,:] = E4M3_rne_sat( (sum_j softmax_j(s) Vq[b,g,j,:]) / out_scale )
 *
 *   q_fp8        [total_q, 32, 128]                E4M3 bytes
 *   k_fp4, v_fp4 [num_pages, 8, 64, 64]            uint8, two E2M1 codes per
 *                byte, head-dim element 2i in the low nibble of byte i;
 *                page p, KV head g, slot s holds token 64*p' + s of the
 *                sequence whose block_table row maps logical page p' to p
 *   k_sf, v_sf   [num_pages, 8, 64, 8]             E4M3 scale per 16 head-dim
 *                elements (element d uses scale d / 16)
 *   block_table  [batch, max_pages_per_seq]        int32 physical page ids;
 *                entries for logical pages < ceil(kv_len_b / 64) must be in
 *                [0, num_pages)
 *   qo_indptr    [batch + 1]                       int32, qo_indptr[0] = 0,
 *                non-decreasing, qo_indptr[batch] = total_q
 *   kv_lens      [batch]                           int32, 0 <= kv_len_b <=
 *                64 * max_pages_per_seq
 *   out_fp8      [total_q, 32, 128]                E4M3 bytes, written
 *   q_scale, out_scale  finite, out_scale > 0
 *
 * qo_indptr and kv_lens are read on the device only.  A query row that sees
 * no key (q_len_b > kv_len_b) is written as zeros.  The kernels check
 * qo_indptr on the device: when it does not run non-decreasing from 0 to
 * total_q they set bit 2 of the error word (gqa_check_device_errors), write
 * rows past qo_indptr[batch] as zeros, and never read or write a row outside
 * [0, total_q); the other rows are then unspecified.  (With host buffers the
 * library checks qo_indptr, kv_lens and the used block-table entries before
 * staging and returns GQA_ERR_INVALID_ARG.)  The softmax numerators P
 * enter the P*V product as f16 (V's dequantised E4M3 values widened to f16
 * exactly), so the result matches the exact value to within the output's
 * E4M3 rounding.
 *
 * Work is split by (sequence, block of 64 queries, KV head).  When those
 * units cannot fill the GPU (short query lengths: decode-like calls, few
 * sequences), each unit's KV range is also split, as gqa_ctx_plan reports,
 * and a second kernel merges the ranges; the partials live in the library's
 * workspace for (device, stream) (n_splits * total_q * 32 * 520 bytes).
 */
gqa_status nvfp4_paged_ctx_attn(const void* q_fp8, float q_scale, const void* k_fp4, const void* k_sf,
                                const void* v_fp4, const void* v_sf, const int32_t* block_table,
                                const int32_t* qo_indptr, const int32_t* kv_lens, void* out_fp8,
                                float out_scale, int64_t batch, int64_t total_q, int64_t num_pages,
                                int64_t max_pages_per_seq, gqa_stream_t stream);

/*
 * gqa_ctx_plan -- how nvfp4_paged_ctx_attn divides the KV range of each work
 * unit, chosen from batch, total_q and max_pages_per_seq only (qo_indptr and
 * kv_lens stay on the device): *tiles_per_split 64-key tiles per split CTA
 * (0 when unsplit), *num_splits ranges per unit, *num_launches kernels per
 * call (0 when total_q = 0; 1 unsplit; 2 with the merge).  The split is used
 * when at most 76 units (8 KV heads x floor((total_q + 63 * batch) / 64), a
 * bound on the (sequence, 64-query block) pairs) can be launched and every
 * range keeps at least 8 tiles.  *persistent = 1 when an unsplit call runs
 * the persistent grid (one CTA per SM walks a share of the units; same
 * result, bit for bit): at least 304 units and max_pages_per_seq <= 48, i.e.
 * short units, whose per-CTA start and end it saves.  *decode_shaped = 1 when
 * the call runs the decode-shaped kernel instead (total_q <= batch, i.e. at
 * most one query per sequence on average, and max_pages_per_seq >= 16): S and
 * P V computed transposed (keys on the MMA's M dimension, 4 queries x 4 heads
 * on N), always as KV ranges (*num_splits of *tiles_per_split 128-key tiles)
 * that the merge combines (*num_launches = 2); its outputs meet the same
 * parity bar but are not bit-identical to the other kernels'.  Any output
 * pointer may be NULL.
 */
gqa_status gqa_ctx_plan(int64_t batch, int64_t total_q, int64_t max_pages_per_seq, int32_t* tiles_per_split,
                        int32_t* num_splits, int32_t* num_launches, int32_t* persistent, int32_t* decode_shaped);

/*
 * gqa_set_ctx_grid -- test switch: the grid of later unsplit
 * nvfp4_paged_ctx_attn calls (all devices, all threads; process-wide).
 * GQA_CTX_GRID_PLANNED (0) = as gqa_ctx_plan reports; GQA_CTX_GRID_PER_UNIT
 * (1) = one CTA per work unit; GQA_CTX_GRID_PERSISTENT (2) = the persistent
 * grid; GQA_CTX_GRID_DECODE_SHAPED (3) = the decode-shaped kernel for every
 * call.  The first two compute the same result, bit for bit; split-KV calls
 * and the ring-depth study instances (gqa_set_schedule) always run one CTA
 * per unit.  Modes 1 and 2 keep calls off the decode-shaped kernel.
 * GQA_ERR_INVALID_ARG for another mode (nothing changes).
 */
enum { GQA_CTX_GRID_PLANNED = 0, GQA_CTX_GRID_PER_UNIT = 1, GQA_CTX_GRID_PERSISTENT = 2, GQA_CTX_GRID_DECODE_SHAPED = 3 };
gqa_status gqa_set_ctx_grid(int mode);

/*
 * gqa_debug_dequant_pages -- test export of the context kernel's NVFP4 ->
 * E4M3 dequantisation (same device routine), gathered through the block
 * table into a dense array.
 *
 *   fp4          [num_pages, 8, 64, 64]   uint8 (as k_fp4 above)
 *   sf           [num_pages, 8, 64, 8]    E4M3 (as k_sf above)
 *   block_table  [batch, max_pages_per_seq] int32
 *   kv_lens      [batch] int32 (device-read)
 *   out_e4m3     [batch, max_kv, 8, 128]  E4M3 bytes: token t of sequence b
 *                for t < min(kv_lens[b], max_kv); zero bytes beyond
 */
gqa_status gqa_debug_dequant_pages(const void* fp4, const void* sf, const int32_t* block_table,
                                   const int32_t* kv_lens, void* out_e4m3, int64_t batch, int64_t num_pages,
                                   int64_t max_pages_per_seq, int64_t max_kv, gqa_stream_t stream);

/*
 * gqa_paged_append_t -- rotary position embedding of new query and key rows,
 * and the append of the new keys and values to a paged K/V cache.  (An
 * addition of this library, like the two entry points after it: they fill and
 * read caches of other head counts, head dims, page sizes, element types and
 * memory orders than the entry points above take.)
 *
 * The new tokens of a batch lie one sequence after the other.  Token t of
 * sequence b (qo_indptr[b] <= t < qo_indptr[b+1]) has the position
 *   pos = kv_lens[b] - (qo_indptr[b+1] - t)
 * (kv_lens counts the new tokens: the lengths that the attention of the same
 * step is given) and goes to page block_table[b, pos / page_size], slot
 * pos % page_size.  The first `rot` elements of each q and k head are rotated
 * with the cosines c = rope[pos, 0 .. rot/2) and sines s = rope[pos, rot/2 ..
 * rot):  (x, y) -> (x c - y s, y c + x s) over the pairs (i, i + rot/2), or
 * (2i, 2i + 1) if `interleaved`.  Everything is computed in f32 and rounded
 * once.  E4M3 pages store round-to-nearest-even, saturating values of
 * k * (1 / k_scale) and v * (1 / v_scale), the reciprocals in f32.
 *
 *   q            [total, q_heads, d]  f16 or bf16, or NULL (then q_out is NULL
 *                too: keys and values only)
 *   k, v         [total, kv_heads, d]  the same type
 *   k_pages, v_pages  [num_pages, kv_heads, page_size, d]  the same type, or
 *                E4M3 (GQA_E4M3 or GQA_U8), written
 *   block_table  [batch, max_pages_per_seq]  int32
 *   kv_lens      [batch]  int32
 *   qo_indptr    [batch + 1]  int32, or NULL: one token per sequence (total =
 *                batch)
 *   rope         [positions, rot]  f32, or NULL: nothing is rotated
 *   q_out        [total, q_heads, d]  q's type, written; may be q itself
 *   batch 1 .. 2^20; d 64, 128 or 256; 1 .. 1024 heads; page_size 1 .. 2^20; rot
 *   a multiple of 16, at most d
 *   k_scale, v_scale  finite, > 0; 1 for pages of the inputs' type
 *
 * Strides.  q, k, v, q_out and the pages may have any strides that are
 * multiples of 16 bytes as long as the last dimension is dense (slices of a
 * fused projection; token-major pages given as a permuted view); what is
 * written must not overlap itself (checked) nor any other argument (not
 * checked), but that q_out may be q.  Every other tensor is dense.
 *
 * Rows left alone.  Tokens at and behind qo_indptr[batch] (a padded batch) and
 * tokens of negative position (a sequence with kv_lens[b] = 0) are skipped:
 * nothing of them is written, in q_out neither.  A token whose position lies
 * outside the block table or the rope table, or whose page lies outside [0,
 * num_pages), is skipped too and bit 1 of the error word
 * (gqa_check_device_errors) is set; offsets that are not non-decreasing from 0
 * to at most `total` set bit 2, and nothing out of range is read or written.
 * Two tokens that share a slot leave pieces of either's row.  No workspace;
 * nothing is synchronised.  Host tensors are refused (GQA_ERR_UNSUPPORTED): a cache that
 * lives on the host has nothing to be appended to on the device.
 */
gqa_status gqa_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                              gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                              const gqa_tensor* qo_indptr, const gqa_tensor* rope, gqa_tensor* q_out, int interleaved,
                              float k_scale, float v_scale, gqa_stream_t stream);

/*
 * nvfp4_paged_append_t -- gqa_paged_append_t into the NVFP4 pages that
 * nvfp4_paged_ctx_attn reads; the rotated queries leave as the E4M3 values it
 * takes:
 *   sf    = E4M3_rne_sat(amax / 6) of each 16 elements of a k or v head,
 *   codes = E2M1_rne_sat(x / sf), all 0 where sf is 0 or NaN,
 *   q_out = E4M3_rne_sat(q * (1 / q_scale)), the reciprocal in f32.
 * The codes are those of f32 divisions.  A block that holds a NaN gets a NaN
 * scale; an infinity gets the largest scale and code.  There is no scale for k
 * and v beside the blocks': a block of magnitudes up to 6 * 2^-10 is stored as
 * zeros, and sf has its 4 bits from amax = 6 * 2^-6 on.  q_scale is then the
 * attention's q_scale.
 *
 *   q      [total, 32, 128], k, v [total, 8, 128]  f16 or bf16, strided as above
 *   k_fp4, v_fp4  [num_pages, 8, 64, 64]  uint8, k_sf, v_sf [num_pages, 8, 64,
 *          8]  E4M3 (or uint8), dense, written
 *   q_out  [total, 32, 128]  E4M3 (or uint8), written; strides multiples of 16
 *          bytes
 *   rot    a multiple of 32
 * The other arguments, and what is skipped, as above (qo_indptr may be NULL).
 */
gqa_status nvfp4_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                                gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                                const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                                gqa_tensor* q_out, int interleaved, float q_scale, gqa_stream_t stream);

/*
 * gqa_paged_norm_append_t, nvfp4_paged_norm_append_t -- the two appends with a
 * norm of each query and key head before the rotation, and with angles of given
 * positions:
 *   x <- x * w / sqrt(sum_i x_i^2 / d + norm_eps)   (w = q_norm for q's heads,
 *        k_norm for k's; values are not normed), then rotated, everything in f32
 *        and rounded once, to what is stored
 *   token t is rotated with row positions[t] of the rope table instead of row pos
 *
 *   q_norm, k_norm  [d]  the inputs' type or f32, both of one type; either or
 *                both may be NULL: those heads are not normed
 *   positions    [total]  int32, or NULL.  For tokens whose place in the cache is
 *                not their position: drafted tokens of a tree (gqa_tree_mask_t).
 *                They choose the angles alone; page and slot are as above.  A
 *                token whose position lies outside the rope table is skipped and
 *                bit 1 of the error word is set.  Needs rope
 *   norm_eps     finite, >= 0 (read where there is a norm); a head of zeros stays
 *                zeros, with a norm_eps of 0 too
 * Everything else as gqa_paged_append_t and nvfp4_paged_append_t.  q_norm and
 * k_norm overlap nothing that is written.
 */
gqa_status gqa_paged_norm_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                                   gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                                   const gqa_tensor* qo_indptr, const gqa_tensor* rope, const gqa_tensor* positions,
                                   const gqa_tensor* q_norm, const gqa_tensor* k_norm, gqa_tensor* q_out, int interleaved,
                                   float norm_eps, float k_scale, float v_scale, gqa_stream_t stream);
gqa_status nvfp4_paged_norm_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                                     gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                                     const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                                     const gqa_tensor* positions, const gqa_tensor* q_norm, const gqa_tensor* k_norm,
                                     gqa_tensor* q_out, int interleaved, float norm_eps, float q_scale, gqa_stream_t stream);

/*
 * gqa_paged_attn_t -- attention of one new token per sequence over a paged K/V
 * cache, split over the cache's length and joined:
 *
 *   s_t = (q[b,h,:] . K_t) * q_scale * k_scale / sqrt(d),   K_t of KV head
 *         h / (q_heads / kv_heads), token t of sequence b
 *   s_t = softcap * tanh(s_t / softcap)  if softcap > 0
 *   out[b,h,:] = v_scale * sum_t softmax_t(s) V_t,  lse[b,h] = ln sum_t exp(s_t)
 *   over max(0, len_b - window) <= t < len_b (window = 0: from 0),
 *   len_b = clamp(seq_lens[b], 0, page_size * max_pages_per_seq)
 *
 *   q            [batch, q_heads, d]  f16 or bf16; strides multiples of 16 bytes,
 *                last dimension dense
 *   k_pages, v_pages  [num_pages, kv_heads, page_size, d]  q's type, or E4M3
 *                (GQA_E4M3 or GQA_U8); strides as gqa_paged_append_t's
 *   block_table  [batch, max_pages_per_seq]  int32; only the entries of pages
 *                that hold a visible token are read
 *   seq_lens     [batch]  int32, read on the device
 *   out          [batch, q_heads, d]  q's type, dense, written
 *   lse          [batch, q_heads]  f32, dense, written; or NULL
 *   workspace    NULL: the library's own for (device, stream), like the other
 *                entry points'.  Or device memory of at least
 *                gqa_paged_attn_workspace(q_heads, kv_heads, d) bytes, 16-byte
 *                aligned, whose contents mean nothing before or after a call: one
 *                each for calls that can run at the same time.  A call that is
 *                being captured has to be given one (GQA_ERR_WORKSPACE without:
 *                two graphs captured on one stream may be replayed at once), which
 *                belongs to the graph as long as it is replayed
 *   batch 1 .. 65535; d 64, 128 or 256; 1 .. 1024 query heads, a multiple of the
 *   kv_heads; page_size 16, 32, 64, 128 or 256; page_size * max_pages_per_seq at
 *   most 2^30, and times batch * kv_heads (more for groups of over 8) at most
 *   about 2^43; q_scale finite, the other scales > 0 too
 *
 * Scores, maxima, sums and the output's accumulators are f32; a cap is exact to
 * 2^-19 of the capped score, whatever its size.  A softmax weight
 * meets V as two 16-bit terms of the pages' type (f16 for E4M3 ones), 22 bits in
 * f16 and 16 in bf16; f16 terms are exact to 2^-39 of the largest weight at best.
 * A bf16 query over E4M3 pages is exact to 2^-40 of its row's largest element.
 * The accumulators of the product with V cut sums off; they take 65536 tokens at
 * most (32768 at d = 256; about 5e-5 of sum w |V| by then) before they are added up
 * with rounding, so that the error does not grow with the length.
 *
 * A sequence of length 0 produces a zero row and lse = -infinity.  Slots outside
 * the visible tokens may hold anything, NaN too; an infinity among the visible
 * values makes its element of the output infinite or NaN.  out and lse overlap
 * no other argument.  A page outside [0, num_pages)
 * is not read: page 0 is used instead and bit 1 of the error word is set.  The
 * split is chosen on the device from the lengths, so a captured call stays
 * balanced when they change.  One kernel, or two; host tensors are refused
 * (GQA_ERR_UNSUPPORTED).
 */
gqa_status gqa_paged_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                            const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out, gqa_tensor* lse,
                            float q_scale, float k_scale, float v_scale, int window, float softcap, void* workspace,
                            int64_t workspace_bytes, gqa_stream_t stream);

/* Bytes of workspace that gqa_paged_attn_t needs for a head layout, whatever the
 * batch and the lengths (0 for one that it does not take). */
int64_t gqa_paged_attn_workspace(int64_t q_heads, int64_t kv_heads, int64_t d);

/*
 * gqa_paged_window_attn_t -- gqa_paged_attn_t whose sliding window leaves the
 * first `sinks` tokens of a sequence visible: the sum runs over
 *   t < min(sinks, len_b)  and  max(0, len_b - window) <= t < len_b,
 * each token once.  sinks >= 0; without a window (0) every token is visible and
 * sinks means nothing.  Only the block table's entries of pages that hold a
 * visible token are read: those between the sinks and the window may be given
 * back.  Workspace, errors and everything else as gqa_paged_attn_t, which is
 * this with sinks = 0.
 */
gqa_status gqa_paged_window_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                                   const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out,
                                   gqa_tensor* lse, float q_scale, float k_scale, float v_scale, int window, int sinks,
                                   float softcap, void* workspace, int64_t workspace_bytes, gqa_stream_t stream);

/*
 * gqa_tree_mask_t -- positions and visibility of trees of drafted tokens, once for
 * all layers of a step.  The drafted tokens of a batch lie one sequence after the
 * other; token i of sequence b is row t = qo_indptr[b] + i and, in the cache,
 * behind base_b = kv_lens[b] - (qo_indptr[b+1] - qo_indptr[b]) tokens.
 *   depth_i        = 0 if parents[t] is -1 (it follows the last cached token), else
 *                    depth of token parents[t] of its sequence, plus 1
 *   positions[t]   = base_b + depth_i
 *   mask[t], bit j = token j of the sequence is i or above it, and, under a window
 *                    (> 0), depth_i - depth_j < window or base_b + depth_j < sinks
 *
 *   parents    [total]  int32, each -1 or less than its token's own number
 *   qo_indptr  [batch + 1], kv_lens [batch]  int32; the drafted tokens included
 *   mask       [total, words]  int32, bit j % 32 of word j / 32; written
 *   positions  [total]  int32, written
 *   (mask and positions overlap nothing else, which is checked; positions may be
 *   parents itself)
 *   words      1 .. 32: trees of up to 32 * words tokens; batch 1 .. 2^20
 *   window, sinks  >= 0, those of the attention
 *
 * A parent out of range counts as -1 and sets bit 1 of the error word; tokens from
 * the 32 * words-th of a tree on are left alone and set it too.  A sequence whose
 * offsets do not lie in order within [0, total] is left alone and sets bit 2, as
 * does qo_indptr[0] != 0.  Rows behind qo_indptr[batch] are left as they are.
 * Device tensors only; no workspace; one kernel.
 */
gqa_status gqa_tree_mask_t(const gqa_tensor* parents, const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, gqa_tensor* mask,
                           gqa_tensor* positions, int window, int sinks, gqa_stream_t stream);

/*
 * gqa_paged_tree_attn_t -- attention of several new tokens per sequence over a paged
 * K/V cache: the drafted tokens of a tree, or of a chain, whose keys and values have
 * been appended.  Token i of sequence b (row t = qo_indptr[b] + i of q and out) lies at
 * place base_b + i of the cache, base_b as above, and sees
 *   with a mask (a tree): the cached tokens j < base_b that its window leaves, j >
 *     positions[t] - window or j < sinks (all of them without a window), and the
 *     drafted tokens at places base_b + j >= 0 whose bit j mask[t] has
 *   without: the tokens j <= base_b + i with j > base_b + i - window or j < sinks
 *   s_j = (q[t,h,:] . K_j) * q_scale * k_scale / sqrt(d), capped as gqa_paged_attn_t's
 *   out[t,h,:] = v_scale * sum_j softmax_j(s) V_j,  lse[t,h] = ln sum_j exp(s_j)
 *
 *   q            [total, q_heads, d]  f16 or bf16; strides multiples of 16 bytes,
 *                last dimension dense
 *   k_pages, v_pages, block_table  as gqa_paged_attn_t's
 *   qo_indptr    [batch + 1], kv_lens [batch]  int32, read on the device; kv_lens
 *                counts the new tokens and is clamped to the block table's capacity
 *   mask         [total, words]  int32, words 1 .. 32, as gqa_tree_mask_t writes it
 *                (its own bit is a token's sight of itself); a drafted token behind
 *                the 32 * words-th is seen by none.  Or NULL: chains
 *   positions    [total]  int32; read with a mask and a window only (then needed),
 *                values below base_b count as base_b; or NULL
 *   out          [total, q_heads, d]  q's type, dense, written
 *   lse          [total, q_heads]  f32, dense, written; or NULL
 *   workspace    as gqa_paged_attn_t's, of gqa_paged_tree_attn_workspace(q_heads,
 *                kv_heads, d) bytes
 *   batch 1 .. 65535; total >= 0; window, sinks >= 0; head layouts, page sizes, the
 *   other numbers and the limit on their product as gqa_paged_attn_t's
 *
 * Scores, maxima, sums and accumulators are f32.  A softmax weight meets V as two
 * 16-bit terms of the pages' type (f16 for E4M3 ones), 22 bits in f16 and 16 in bf16;
 * f16 terms are exact to 2^-31 of the largest weight at best.  A bf16 query over E4M3
 * pages is exact to 2^-40 of its row's largest element.  The accumulators of the product
 * with V cut sums off; they take 16384 tokens at most (about 2e-5 of sum w |V| by
 * then) before they are added up with rounding, so that the error does not grow with the
 * length.
 *
 * A row that sees nothing (a sequence of length 0, an empty mask) becomes zeros, with
 * lse = -infinity; rows behind qo_indptr[batch] are left as they are.  Slots that no
 * row of their sequence can see -- behind its length, or between the sinks and the
 * window of its first new token -- may hold anything, NaN too; an infinity or NaN in a
 * row of V that some row of the sequence sees may make its element NaN in the others,
 * whether they see it or not.  A page outside [0, num_pages) is not read: page 0 is
 * used instead and bit 1 of the error word is set.  A sequence whose offsets do not lie
 * in order within [0, total] is left out (its rows are not written) and sets bit 2, as
 * does qo_indptr[0] != 0; where offsets fall so often that the sequences between pass
 * the limit on the product, all are left out (but rows without a token become zeros).
 * out and lse overlap no other argument.  The split is chosen on the device from the
 * lengths.  One kernel, or two; host tensors are refused.
 */
gqa_status gqa_paged_tree_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                                 const gqa_tensor* block_table, const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens,
                                 const gqa_tensor* mask, const gqa_tensor* positions, gqa_tensor* out, gqa_tensor* lse,
                                 float q_scale, float k_scale, float v_scale, int window, int sinks, float softcap,
                                 void* workspace, int64_t workspace_bytes, gqa_stream_t stream);

/* Bytes of workspace that gqa_paged_tree_attn_t needs for a head layout, whatever the
 * batch, the tokens and the lengths (0 for one that it does not take). */
int64_t gqa_paged_tree_attn_workspace(int64_t q_heads, int64_t kv_heads, int64_t d);

/*
 * gqa_paged_keep_t -- compaction of a paged cache after verification: of each
 * sequence's drafted tokens the accepted ones move together, behind its cached
 * tokens, and the others are given up.  Drafted token kept[b, i] of sequence b
 * (place base_b + kept[b, i] in the cache, base_b as above) goes to place
 * base_b + i for 0 <= i < num_kept[b], and new_lens[b] = base_b + num_kept[b].
 * Rows behind the new length are not cleared.
 *
 *   pages        1 to 4 tensors [num_pages, heads, page_size, w] or, for the pages
 *                of several layers at once, [layers, num_pages, heads, page_size,
 *                w] of any type; rows of a multiple of 8 bytes, strides multiples
 *                of 8 bytes with a dense last dimension; num_pages and page_size
 *                are common to all.  K and V pages, or the codes and scales of
 *                NVFP4 ones.  Written; they overlap neither themselves (checked)
 *                nor one another
 *   block_table  [batch, max_pages_per_seq], qo_indptr [batch + 1], kv_lens
 *                [batch]  int32, as for the step's append
 *   kept         [batch, max_kept]  int32, rising; entries from num_kept[b] on are
 *                not read
 *   num_kept     [batch]  int32
 *   new_lens     [batch]  int32, written; overlaps none of the other small tensors
 *                (checked), nor pages
 *   batch        1 .. 65535
 *
 * A sequence whose kept tokens do not rise, or do not lie in its draft, or which is
 * shorter than its draft, is left as it is (new_lens[b] = kv_lens[b]; bit 1 of the
 * error word unless it keeps nothing, or bit 2 where its offsets fall).  A row whose old or new place lies
 * outside the block table or the pages stays where it is and sets bit 1.  Sequences
 * that share a page must not both move rows in it.  Device tensors only; no
 * workspace; one kernel; the same bits whatever the order.
 */
gqa_status gqa_paged_keep_t(const gqa_tensor* const* pages, int num_tensors, const gqa_tensor* block_table,
                            const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* kept,
                            const gqa_tensor* num_kept, gqa_tensor* new_lens, gqa_stream_t stream);

/*
 * gqa_check_device_errors -- synchronise `device` and return (then clear)
 * the kernels' device error word in *word: bit 0 = a bounded wait expired,
 * bit 1 = an out-of-range page index, position of a token, parent of a tree or list of
 * kept tokens was skipped, bit 2 = qo_indptr was not non-decreasing from 0 to total_q
 * (to at most total where rows behind it are allowed), bit 3 = the dequantisation export's
 * self-check failed.  Returns GQA_ERR_TIMEOUT when bit 0 is set,
 * GQA_ERR_INVALID_ARG when another bit is set, GQA_OK when the word is 0.
 * After a timeout the outputs of the affected call are unspecified; every
 * kernel waits for the tensor-core operations and copies it started before
 * it releases its resources, so later calls are unaffected.
 */
gqa_status gqa_check_device_errors(int device, uint32_t* word);

/*
 * gqa_debug_wait_expiry -- test export of the kernels' failure detection: on
 * `device`, one CTA waits on an mbarrier that nothing completes, through the
 * bounded wait every kernel of the library uses.  After about 2 s the wait
 * gives up, sets bit 0 of the error word and the kernel returns; a following
 * gqa_check_device_errors reports GQA_ERR_TIMEOUT.  No trap and no fault: the
 * context stays usable.  Asynchronous on `stream`.
 */
gqa_status gqa_debug_wait_expiry(int device, gqa_stream_t stream);

/*
 * gqa_set_schedule -- study switch: ring depths of later launches (all
 * devices, all threads; process-wide).  Every depth computes the same
 * result, bit for bit -- the invariant "GB300 NVFP4 Context Attention: scale
 * slot 조기 반납과 8단 packed K/V ring" checks for its ring changes (section 2
 * and its results section) -- so a schedule changes only speed.
 *
 *   ctx_packed_stages, ctx_kv_slots  packed NVFP4 page stages and dequantised
 *       K/V tile slots of the one-CTA-per-unit context attention kernel of
 *       unsplit calls; 0 = its production depth (4 stages, 4 slots).
 *       Instantiated (stages, slots): (4,4) (6,4) (8,4) (10,4) (6,3) (12,3)
 *       (6,5) (6,2).  A non-production depth runs every unsplit call on the
 *       one-CTA-per-unit grid; split-KV calls and the persistent grid always
 *       run their production depths (6 stages, 4 slots).
 *   decode_stages  16-token K/V stages of the decode ring (stacked cache);
 *       0 = the production depth 8; also 4, 12, 16.  The paged decode always
 *       runs depth 8.
 *
 * GQA_ERR_UNSUPPORTED for a depth that is not instantiated (nothing changes).
 */
gqa_status gqa_set_schedule(int ctx_packed_stages, int ctx_kv_slots, int decode_stages);

/*
 * gqa_debug_starve_producers -- test switch of the failure detection.  With
 * enable != 0, every later launch (all devices, all threads) runs its
 * kernels with producers that issue no copies: each consumer's bounded wait
 * expires after about 2 s, every role leaves its loop, the CTA drains what it
 * started, frees its tensor memory and exits, and gqa_check_device_errors
 * reports GQA_ERR_TIMEOUT.  enable = 0 restores normal operation.  Not for
 * concurrent use with real work: the setting is process-wide.
 */
gqa_status gqa_debug_starve_producers(int enable);

/* Free every workspace the library holds (all devices and streams).  The
 * caller must ensure no libgqa work is still running. */
gqa_status gqa_release_workspace(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_H_ */
