/*
 * vsa.h -- C ABI of the GB300 (sm_103a) block-sparse attention forward library
 * (libvsa_gb300.so).
 *
 * The operation (both entry points compute the same thing; they differ in how the
 * block selection is encoded):
 *
 *   For batch b, head h and query row i, let qb = i / block be its query block.
 *   Key j (key block kb = j / block) is attended iff kb is selected for (b, h, qb)
 *   and (j mod block) < variable_block_sizes[kb].  Over the attended keys A_i:
 *
 *     out[b,h,i,:] = sum_{j in A_i} softmax_j(scale * q_i . k_j) * v[b,h,j,:]
 *     lse[b,h,i]   = log2( sum_{j in A_i} exp(scale * q_i . k_j) )
 *                  = max_j(q_i.k_j * scale * log2 e) + log2(l)      (base 2)
 *
 *   A row with no attended key gets out = +0.0 in every element and
 *   lse = VSA_LSE_EMPTY.
 *
 *   Sources: "FastVideo block_sparse_attn_sm100a.py" -- module docstring (forward
 *   returns (out, lse), lse = max(qk*qk_scale) + log2(l), [B,H,S] fp32; 64- and
 *   128-token blocks) and is_supported docstring (BHSD bf16, head_dim 128, even
 *   number of blocks, per-row counts in [0, max_kv], padding past a row's count never
 *   read, count 0 -> zero output and a finite LSE sentinel, keys at or past a block's
 *   valid count masked); "TheRock rocke sparse_attention.py" -- module docstring (the
 *   Jenga i8 MaskBitmap[q_block, k_block], 1 = attend; the VSA per-q-block LUT of
 *   BlockCount entries) and _lds_bitmap_predicate (a nonzero byte means attend).
 *
 * Conventions shared by every entry point:
 *   - Tensors are dense and contiguous.  q, k, v, out are bf16 bit patterns laid out
 *     [B, H, S, D] (BHSD), D = VSA_HEAD_DIM = 128, 16-byte aligned.  The library
 *     never takes ownership of and never retains a pointer; it allocates nothing.
 *   - Device pointers unless the name says host.  All work is enqueued on `stream`
 *     (a cudaStream_t; NULL = the legacy default stream) and is asynchronous: the
 *     call returns once the work is enqueued.  No host-device synchronisation, no
 *     reads of tensor contents on the host.
 *   - Argument checks happen on the host before anything is enqueued; a failed check
 *     returns an error and enqueues nothing.
 *   - Metadata is int32.  LUT entries below a row's count must lie in [0, nb);
 *     entries outside that range are skipped, counts are clamped to [0, max_kv], and
 *     a block named twice in one row is attended once (set semantics).
 *   - Each kernel bounds every internal wait (about one second).  A wait that runs
 *     out records a code in a device status word and the kernel returns early; read
 *     it with vsa_device_status().
 */
#ifndef VSA_GB300_H
#define VSA_GB300_H

#include <float.h>
#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vsa_status {
  VSA_OK = 0,
  VSA_ERR_INVALID_ARG = 1,    /* null pointer, bad shape, misaligned tensor, bad scale */
  VSA_ERR_UNSUPPORTED = 2,    /* valid but not built for: D != 128, block not 64/128,
                                 too many key blocks, device not sm_103 */
  VSA_ERR_CUDA = 3,           /* a CUDA runtime call failed (launch, copy, attribute) */
  VSA_ERR_DEVICE_TIMEOUT = 4  /* a kernel gave up on an internal wait (vsa_device_status) */
} vsa_status;

/* Finite stand-in for log2(0) written to lse for rows with no attended key:
 * -FLT_MAX, the most negative finite binary32. */
#define VSA_LSE_EMPTY (-FLT_MAX)
#define VSA_HEAD_DIM 128
/* Largest number of key blocks per sequence (Sk / block) the kernels accept. */
#define VSA_MAX_BLOCKS 2048
/* Largest num_splits vsa_fwd_split accepts. */
#define VSA_MAX_SPLITS 64

/* every entry point is exported from the shared library */
#if defined(__GNUC__)
#define VSA_API __attribute__((visibility("default")))
#else
#define VSA_API
#endif

typedef uint16_t vsa_bf16;            /* bf16 bit pattern */
typedef struct CUstream_st *vsa_stream_t; /* == cudaStream_t */

/* VSA forward.
 *   q, k, v      [B, H, S, D] bf16.
 *   q2k_idx      [B, H, nb, max_kv] int32, nb = S / block: the key blocks each query
 *                block attends; row (b, h, qb) holds its q2k_num[b, h, qb] valid entries
 *                first, anything after them (e.g. -1 padding) is never read.
 *   q2k_num      [B, H, nb] int32 valid-entry counts (0 allowed).
 *   variable_block_sizes  [nb] int32, each in [0, block]: valid keys of each key block;
 *                keys at positions >= it are masked (values are clamped to [0, block]).
 *   block        64 or 128 tokens per block; S must be a multiple.  (The FastVideo
 *                contract asks for an even nb; an odd nb is accepted as well: with block
 *                64 the last query block of each head is then computed on its own.)
 *   scale        natural-exp softmax scale (finite, > 0), typically 1/sqrt(D).
 *   out          [B, H, S, D] bf16 output; must not overlap any input.
 *   lse          [B, H, S] fp32 output (base 2), or NULL to skip it (need_lse = false).
 *   workspace    NULL, or device memory of at least vsa_workspace_bytes() bytes that
 *                is all zero before the first call; each call leaves it zero again.
 *                With a workspace, work items are handed out dynamically (better
 *                balance for uneven counts); calls sharing one workspace must not
 *                overlap on the GPU.  NULL selects a static round-robin schedule.
 * Source: "FastVideo block_sparse_attn_sm100a.py", block_sparse_attn_sm100a and
 * is_supported; "TheRock rocke sparse_attention.py", build_vsa_sparse_attention. */
VSA_API vsa_status vsa_fwd(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                   const int32_t *q2k_idx, const int32_t *q2k_num,
                   const int32_t *variable_block_sizes, int B, int H, int S, int D,
                   int max_kv, int block, float scale, vsa_bf16 *out, float *lse,
                   void *workspace, vsa_stream_t stream);

/* Jenga forward: the selection is one i8 bitmap mask_bitmap[S/block_q, S/block_k],
 * shared by every batch and head; a nonzero byte means attend.  Every key of a selected
 * block is valid (no tail mask).  block_q == block_k, 64 or 128; S a multiple of it.
 * Other arguments as vsa_fwd.
 * Source: "TheRock rocke sparse_attention.py", module docstring (Jenga bullet),
 * _stage_jenga_mask_to_lds, _lds_bitmap_predicate, build_jenga_sparse_attention. */
VSA_API vsa_status jenga_fwd(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                     const int8_t *mask_bitmap, int B, int H, int S, int D, int block_q,
                     int block_k, float scale, vsa_bf16 *out, float *lse, void *workspace,
                     vsa_stream_t stream);

/* Grouped-query and cross-length VSA forward: vsa_fwd with separate query / key-value
 * head counts and sequence lengths.
 *   q, out       [B, Hq, Sq, D] bf16;  k, v  [B, Hkv, Sk, D] bf16;  Hq a multiple of Hkv.
 *                Query head hq reads key/value head hq / (Hq / Hkv).
 *   q2k_idx      [B, Hq, Sq/block, max_kv] int32, entries in [0, Sk/block).
 *   q2k_num      [B, Hq, Sq/block] int32.
 *   variable_block_sizes  [Sk/block] int32, or NULL for full key blocks.
 *   lse          [B, Hq, Sq] fp32 or NULL.
 *   Sq and Sk are multiples of block; Sk / block <= VSA_MAX_BLOCKS.  Sk = 0 is allowed:
 *   every row is then empty (out 0, lse VSA_LSE_EMPTY).  Hq % Hkv != 0 is
 *   VSA_ERR_INVALID_ARG.  Other arguments and errors as vsa_fwd; with Hq = Hkv = H and
 *   Sq = Sk = S this is vsa_fwd.
 * Source: "TheRock rocke sparse_attention.py", JengaSparseSpec / VsaSparseSpec (separate
 * seqlen_q, seqlen_k and query / key-value head counts; the key-value head of a query
 * head, kv_head_idx). */
VSA_API vsa_status vsa_fwd_gqa(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                               const int32_t *q2k_idx, const int32_t *q2k_num,
                               const int32_t *variable_block_sizes, int B, int Hq, int Hkv,
                               int Sq, int Sk, int D, int max_kv, int block, float scale,
                               vsa_bf16 *out, float *lse, void *workspace, vsa_stream_t stream);

/* Forward straight from a block map, compacted inside the kernel (no LUT is built in
 * memory).
 *   block_map    int8, nonzero = attend.  map_shared == 0: [B, Hq, Sq/block, Sk/block],
 *                one map per (batch, query head); map_shared != 0: [Sq/block, Sk/block],
 *                one map for every batch and head (the Jenga layout).
 *   variable_block_sizes  [Sk/block] int32 valid keys per key block, or NULL = full.
 *   Shapes, lse, workspace and errors as vsa_fwd_gqa.  The result equals vsa_fwd_gqa on
 *   the LUT that vsa_bitmap_to_lut makes from the same map with max_kv = Sk/block.
 * Source: "FastVideo block_sparse_attn_sm100a.py", _block_sparse_attn_sm100a_from_mask_
 * inference and block_sparse_attn_sm100a_from_mask (a bool block_map [B, H, nb, nb] turned
 * into the forward's selection); "TheRock rocke sparse_attention.py", Jenga bullet of the
 * module docstring (an i8 map, nonzero = attend). */
VSA_API vsa_status vsa_fwd_from_mask(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                                     const int8_t *block_map, int map_shared,
                                     const int32_t *variable_block_sizes, int B, int Hq,
                                     int Hkv, int Sq, int Sk, int D, int block, float scale,
                                     vsa_bf16 *out, float *lse, void *workspace,
                                     vsa_stream_t stream);

/* Split-KV forward: vsa_fwd_gqa with each work item's key tiles divided into num_splits
 * contiguous ranges processed by different CTAs, then combined by a second kernel.  For
 * shapes with few work items (a short query, few heads) and long key lists, where one
 * CTA per item would leave most SMs idle.
 *   A work item is 128 query rows (one block-128 query block, or an adjacent pair of
 *   block-64 query blocks); its selected key blocks form key tiles of 128 keys, and range
 *   s of n tiles is tiles [n*s/num_splits, n*(s+1)/num_splits) (possibly empty).
 *   Each range leaves in the workspace an fp32 partial: O [128][128] relative to the
 *   row's running maximum m, then m, the sum of the bf16-rounded weights and the sum of
 *   the fp32 weights per row; the merge takes M = max m_s and c_s = 2^(m_s - M) and
 *   writes out = sum c_s O_s / sum c_s l_round_s and lse = M + log2(sum c_s l_exact_s),
 *   the same arithmetic the single-pass kernel uses to join its two key halves, so the
 *   result matches vsa_fwd_gqa within rounding (not bit for bit).
 *   num_splits   1..VSA_MAX_SPLITS; 1 is vsa_fwd_gqa (workspace then optional, as there).
 *   workspace    device memory of at least vsa_split_workspace_bytes(B, Hq, Sq, block,
 *                num_splits) bytes, 16-byte aligned, whose first vsa_workspace_bytes()
 *                bytes are zero before the call (they are left zero); the rest needs no
 *                initialisation.  Must not overlap q, out or lse.  Calls sharing a
 *                workspace must not overlap on the GPU.
 *   workspace_bytes  its size; a smaller one is VSA_ERR_INVALID_ARG.
 *   Other arguments and errors as vsa_fwd_gqa.  Enqueues two kernels.
 * Source: the split-K decode pattern of "vLLM FlyDSL tq_decode" (partial (m, l, O) per
 * key partition plus a reduction); the arithmetic of each part is that of vsa_fwd. */
VSA_API vsa_status vsa_fwd_split(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                                 const int32_t *q2k_idx, const int32_t *q2k_num,
                                 const int32_t *variable_block_sizes, int B, int Hq, int Hkv,
                                 int Sq, int Sk, int D, int max_kv, int block, float scale,
                                 int num_splits, vsa_bf16 *out, float *lse, void *workspace,
                                 size_t workspace_bytes, vsa_stream_t stream);

/* Workspace bytes vsa_fwd_split needs for this shape (0 for an invalid one). */
VSA_API size_t vsa_split_workspace_bytes(int B, int Hq, int Sq, int block, int num_splits);

/* Backward: dq, dk, dv of the vsa_fwd_gqa forward for an upstream gradient dout.
 *   With p_ij = 2^(scale * log2(e) * q_i . k_j - lse_i) over the attended keys (0 for the
 *   rest), D_i = dout_i . out_i and ds_ij = p_ij (dout_i . v_j - D_i):
 *     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
 *   dk and dv summed over every query head of a key/value group.  Rows with no attended
 *   key contribute nothing (their dq is 0); keys no row attends get dk = dv = 0.
 *   q, k, v, q2k_idx, q2k_num, variable_block_sizes, shapes, max_kv, block, scale: as given
 *     to the forward.
 *   out          the forward's output [B, Hq, Sq, D] bf16.
 *   lse          the forward's lse [B, Hq, Sq] fp32 (required, 16-byte aligned).
 *   dout         [B, Hq, Sq, D] bf16.
 *   dq           [B, Hq, Sq, D] bf16 output;  dk, dv  [B, Hkv, Sk, D] bf16 outputs.
 *   workspace    at least vsa_bwd_workspace_bytes(B, Hq, Sq, Sk, block) bytes, 256-byte
 *                aligned, no initialisation needed (the block map, -D and -lse per
 *                query row and an fp32 dq accumulator live there).
 *   No output may overlap an input or another output.  Enqueues up to four kernels and
 *   one memset; errors as vsa_fwd_gqa, and VSA_ERR_UNSUPPORTED for more than 65536 query
 *   blocks per head or more than 4096 query heads per key/value head.
 * Source: "FastVideo block_sparse_attn_sm100a.py", module docstring (the backward
 * consumes the forward's base-2 lse); the gradient is that of softmax attention. */
VSA_API vsa_status vsa_bwd(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                           const vsa_bf16 *out, const vsa_bf16 *dout, const float *lse,
                           const int32_t *q2k_idx, const int32_t *q2k_num,
                           const int32_t *variable_block_sizes, int B, int Hq, int Hkv, int Sq,
                           int Sk, int D, int max_kv, int block, float scale, vsa_bf16 *dq,
                           vsa_bf16 *dk, vsa_bf16 *dv, void *workspace, size_t workspace_bytes,
                           vsa_stream_t stream);

/* Workspace bytes vsa_bwd needs for this shape (0 for an invalid one). */
VSA_API size_t vsa_bwd_workspace_bytes(int B, int Hq, int Sq, int Sk, int block);

/* Bytes of device workspace the forward entry points use when given one. */
VSA_API size_t vsa_workspace_bytes(void);

/* Size of the library's own scheduling scratch used by vsa_fwd_noalloc. */
#define VSA_NOALLOC_SCRATCH_BYTES 256

/* vsa_fwd for callers that cannot allocate device memory.  (The pages describe no such
 * entry point; it exists for this library's users.)  Some callers have no way to obtain
 * a workspace buffer: a plug-in whose host framework owns every device allocation and
 * offers no hook for extra buffers, or a serving loop that must not call cudaMalloc once
 * it is running because cudaMalloc can synchronise the device and stall other streams.
 * This entry point takes the same arguments as vsa_fwd minus `workspace`, allocates
 * nothing and calls no allocating routine: its dynamic-schedule scratch is a static
 * device array of VSA_NOALLOC_SCRATCH_BYTES bytes inside the library, which every GPU
 * that loads the library keeps until the process exits.
 *   - The first call on a device (with that device current) looks up the array's
 *     device address and caches it for the device's current context; a later call in
 *     a new context (after cudaDeviceReset, say) looks it up again.  Make the first
 *     call on a device before any stream capture begins.
 *   - Every call on a device shares the array, which keeps what the last call left.
 *     Each call clears the scheduling counters in stream order before its kernel, so
 *     calls on one stream are safe; calls that overlap on the GPU (different streams
 *     without ordering between them) race on the counters and must not be issued.
 *   - A call whose scratch need exceeds VSA_NOALLOC_SCRATCH_BYTES returns
 *     VSA_ERR_UNSUPPORTED.  Argument errors and unsupported configurations are those
 *     of vsa_fwd and are reported before anything is enqueued; a VSA_ERR_CUDA from a
 *     failed launch can come after the scratch reset was enqueued (harmless: the
 *     scratch is left zero). */
VSA_API vsa_status vsa_fwd_noalloc(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                                   const int32_t *q2k_idx, const int32_t *q2k_num,
                                   const int32_t *variable_block_sizes, int B, int H, int S,
                                   int D, int max_kv, int block, float scale, vsa_bf16 *out,
                                   float *lse, vsa_stream_t stream);

/* LUT -> bitmap, bit-exact: bitmap[r, kb] = 1 iff kb is one of the first
 * clamp(q2k_num[r], 0, max_kv) entries of q2k_idx row r (entries outside [0, nb)
 * skipped), else 0.  q2k_idx [rows, max_kv], q2k_num [rows], bitmap [rows, nb] int8.
 * Source: "TheRock rocke sparse_attention.py", _stage_vsa_bitmap_to_lds (zero the
 * row, then scatter 1 at every listed block; idempotent). */
VSA_API vsa_status vsa_lut_to_bitmap(const int32_t *q2k_idx, const int32_t *q2k_num, int rows,
                             int max_kv, int nb, int8_t *bitmap, vsa_stream_t stream);

/* bitmap -> LUT, bit-exact: row r lists the indices of its nonzero bytes in
 * ascending order, the first min(count, max_kv) of them, then -1 up to max_kv;
 * q2k_num[r] = min(count, max_kv).  bitmap [rows, nb] int8 -> q2k_idx [rows, max_kv],
 * q2k_num [rows] int32.
 * Source: "FastVideo block_sparse_attn_sm100a.py", _block_sparse_attn_sm100a_from_
 * mask_inference (a bool block map compacted into (q2k_idx, q2k_num), -1 fill). */
VSA_API vsa_status vsa_bitmap_to_lut(const int8_t *bitmap, int rows, int nb, int max_kv,
                             int32_t *q2k_idx, int32_t *q2k_num, vsa_stream_t stream);

/* vsa_fwd with HOST buffers: copies q, k, v, q2k_idx, q2k_num, variable_block_sizes
 * from host memory into the caller's device buffers (the d_* arguments, same shapes as
 * vsa_fwd), runs the forward, and copies out (and lse, if h_lse is not NULL) back to host
 * memory.  The work is split into chunks of consecutive (b, h) heads (about 20 MB of q,
 * k, v each, at most 32, at most one per head): a chunk's inputs go over on an input
 * stream, its forward runs on `stream` as soon as they have landed, and its outputs come
 * back on an output stream, so copies of one chunk overlap the forward of another.  The two internal streams (and their events) are created once
 * per device on first use -- no device memory -- and fork from `stream` at the start of
 * the call and join it at the end: everything is ordered after earlier work on `stream`,
 * and later work on `stream` (or a synchronisation of it) sees the whole call complete.
 * The caller synchronises `stream` before reading h_out / h_lse.  Host buffers should
 * be pinned (page-locked) for the copies to be asynchronous.  d_lse may be NULL only if
 * h_lse is NULL.  Calls from several host threads are serialised on an internal lock.
 * Argument errors are reported before anything is enqueued. */
VSA_API vsa_status vsa_fwd_from_host(const vsa_bf16 *h_q, const vsa_bf16 *h_k, const vsa_bf16 *h_v,
                             const int32_t *h_q2k_idx, const int32_t *h_q2k_num,
                             const int32_t *h_variable_block_sizes, int B, int H, int S,
                             int D, int max_kv, int block, float scale, vsa_bf16 *h_out,
                             float *h_lse, vsa_bf16 *d_q, vsa_bf16 *d_k, vsa_bf16 *d_v,
                             int32_t *d_q2k_idx, int32_t *d_q2k_num,
                             int32_t *d_variable_block_sizes, vsa_bf16 *d_out, float *d_lse,
                             void *workspace, vsa_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Choosing the blocks, and serving single tokens from an 8-bit cache.
 *
 * vsa_block_mean and vsa_select_blocks make the (q2k_idx, q2k_num) that vsa_fwd,
 * vsa_fwd_gqa, vsa_fwd_split and vsa_bwd take: one mean per block of q and of k, and for
 * every query block the key blocks of the highest q_mean . k_mean.  (The choice has no
 * gradient; that of the attention over the chosen blocks is vsa_bwd's.)
 *
 * The 8-bit cache holds a server's keys and values.  Its pool has `pages` pages; a page
 * holds `block` (64 or 128) consecutive tokens of one sequence and key/value head:
 *   k_cache, v_cache  [pages, block, D] e4m3 codes (uint8), 16-byte aligned
 *   k_scale, v_scale  [pages] fp32: value = code * scale
 *   k_mean            [pages, D] bf16: the mean of the page's keys as the cache holds them
 * table[b, h, j] (int32 [B, Hkv, max_blocks]) is the page of tokens j*block .. of sequence
 * b and key/value head h, lens[b] (int32 [B]) the tokens that sequence b holds, at most
 * max_blocks * block.  A table entry outside [0, pages) names no page: nothing is written
 * there, and its tokens are not attended or chosen.  Entries past a sequence's last block
 * are ignored.  A cache whose pages hold all heads together, [n, Hkv, block, D], is this
 * one with pages = n * Hkv and table entries page * Hkv + h.
 * A step of a server: vsa_cache_write the new tokens, add their number to lens,
 * vsa_cache_select (or none: all blocks), vsa_fwd_cache, and now and then
 * vsa_cache_evict.  max_blocks <= VSA_MAX_BLOCKS.
 * ------------------------------------------------------------------------------------- */

/* Block means: mean[b, h, j] = the mean of the first n_j tokens of block j of x, in fp32,
 * rounded to bf16 once; 0 where n_j = 0.
 *   x      [B, H, S, D] bf16, 16-byte aligned; S need not be a multiple of block.
 *   sizes  [nb] int32, nb = ceil(S / block): n_j = sizes[j] clamped to [0, block] and to
 *          the tokens there are; NULL = all of them.  Tokens past n_j are not read.
 *   mean   [B, H, nb, D] bf16 output; must not overlap x or sizes. */
VSA_API vsa_status vsa_block_mean(const vsa_bf16 *x, const int32_t *sizes, int B, int H, int S,
                                  int D, int block, vsa_bf16 *mean, vsa_stream_t stream);

/* The key blocks each query block attends.  For query head hq (key/value head
 * hq / (Hq / Hkv)) and query block i, with d = i + nk - nq the key block on its diagonal:
 * of the eligible blocks j, the min(topk, their number) of the highest
 * q_mean[b, hq, i] . k_mean[b, hkv, j], ascending in q2k_idx with -1 behind, and their
 * number in q2k_num.
 *   eligible   sizes[j] > 0 (sizes [nk] int32, or NULL), with causal != 0 j <= d, and the
 *              score is not NaN
 *   forced     blocks j < n_first or |j - d| < n_near that are eligible but for the score
 *              come before all others whatever their score (a NaN too)
 * Scores are compared by their fp64 sums, and equal ones go to the lower index; fp32 sums
 * serve where their error bound leaves no doubt.  Products of bf16 values are exact in fp64,
 * and so is their sum while the products of a score differ by less than 2^30 in size: the
 * order is then that of the real numbers.  Beyond that the sum, always taken in the same
 * order, is off by at most 2^-48 of sum |q||k|.  A row with nothing eligible gets a count
 * of 0.
 *   q_mean [B, Hq, nq, D], k_mean [B, Hkv, nk, D] bf16, 16-byte aligned; nk <=
 *   VSA_MAX_BLOCKS; q2k_idx [B, Hq, nq, topk], q2k_num [B, Hq, nq] int32 outputs, which
 *   must not overlap anything else.  topk >= 1 (it may exceed nk).
 * Rows with more than 32 blocks inside the fp32 error band -- blocks with equal means, or
 * means whose common part is large against what tells them apart -- take a far slower path,
 * on which every score of the row is an fp64 sum: with every row on it 43 ms instead of 0.15
 * for 24 heads of 1,536 x 1,536 blocks, 0.94 ms instead of 0.013 for 12 heads of 256 x 256.
 * A part that all key means share changes no order: with it taken off them beforehand the
 * rows stay on the fast path. */
VSA_API vsa_status vsa_select_blocks(const vsa_bf16 *q_mean, const vsa_bf16 *k_mean,
                                     const int32_t *sizes, int B, int Hq, int Hkv, int nq, int nk,
                                     int D, int topk, int causal, int n_first, int n_near,
                                     int32_t *q2k_idx, int32_t *q2k_num, vsa_stream_t stream);

/* vsa_select_blocks for one token per sequence over the cache: for each sequence and
 * key/value head, the blocks of the highest score, a block's score being the largest of
 * q[b, hq] . k_mean[page] over the query heads of the group.  The diagonal is the
 * sequence's last block (n_near = 1 forces it), n_first forces the first ones; ties,
 * forced blocks and NaN as in vsa_select_blocks.
 *   q [B, Hq, 1, D] bf16; idx [B, Hkv, topk], num [B, Hkv] int32 outputs, the listing that
 *   vsa_fwd_cache takes. */
VSA_API vsa_status vsa_cache_select(const vsa_bf16 *q, const vsa_bf16 *k_mean,
                                    const int32_t *table, const int32_t *lens, int B, int Hq,
                                    int Hkv, int D, int pages, int max_blocks, int block,
                                    int topk, int n_first, int n_near, int32_t *idx, int32_t *num,
                                    vsa_stream_t stream);

/* Tokens lens[b] .. lens[b] + n_new[b] - 1 of every sequence into the cache.
 *   k, v   [B, Hkv, T, D] bf16: row t is token lens[b] + t; rows from n_new[b] on (a padded
 *          batch) are not read.  n_new int32 [B], clamped to [0, T], or NULL = T each.
 *   lens   the tokens held before the call; it is not changed (add n_new to it after).
 * A page's scale is the least power of two s >= 2^-100 with max |x| <= 448 s over its
 * finite values so far, and a code the nearest e4m3 value of x / s (ties to even;
 * infinities become +-448 s, NaN stays NaN).  When a new token raises a page's scale, the
 * codes it holds move to the new one: exactly while they stay normal (2^-6 or more); a code
 * that becomes subnormal is rounded to a multiple of 2^-9 at each move.  So a page written
 * token by token ends as one written at once, but for codes up to 2^-6, which may be one
 * step of 2^-9 apart (and the mean, which is that of the codes held), and for infinities,
 * which count as 448 times the scale of their time.  k_mean (or NULL) gets the mean of the
 * page's keys as now held.  Page bytes of tokens not yet held stay as
 * they are, tokens past max_blocks * block are dropped, and what a page held before its
 * first token is ignored.  No two written pages may be the same.  Scales that were not
 * made here must be powers of two. */
VSA_API vsa_status vsa_cache_write(const vsa_bf16 *k, const vsa_bf16 *v, const int32_t *table,
                                   const int32_t *lens, const int32_t *n_new, int B, int Hkv,
                                   int T, int D, int pages, int max_blocks, int block,
                                   uint8_t *k_cache, uint8_t *v_cache, float *k_scale,
                                   float *v_scale, vsa_bf16 *k_mean, vsa_stream_t stream);

/* Attention of one token per sequence over its cache (lens counts the token itself if it
 * has been written): out and lse as vsa_fwd's, over the tokens of the listed blocks.
 *   q, out  [B, Hq, 1, D] bf16; lse [B, Hq, 1] fp32 (base 2) or NULL.
 *   idx     [B, Hkv, max_sel] int32, num [B, Hkv]: the blocks the whole group of a
 *           key/value head attends (counts clamped to [0, max_sel], entries outside the
 *           sequence skipped, a block named twice attended once), or both NULL: every
 *           block.  k_scale, v_scale may be any numbers of up to 2^80 in magnitude (and
 *           scale * |q| up to 2^40): products and sums are taken in fp32, whose range
 *           larger ones can leave although the result would not.
 *   weight  [B, Hkv, max_blocks] fp32 or NULL: becomes keep * weight + w, w the sum of the
 *           attention weights that the group's heads give the block's tokens (0 for a
 *           block not attended).  keep = 1 accumulates, 0 records this step alone (what
 *           was there is not read), between them the past fades.
 *   workspace  at least vsa_cache_workspace_bytes(B, Hq, Hkv, max_blocks, weight != NULL)
 *           bytes, 16-byte aligned, whose first 256 KB are zero before the first call;
 *           each call leaves them zero.  It may serve calls of other shapes in turn, but
 *           calls sharing it must not overlap on the GPU (give graphs that may run at the
 *           same time one each).
 * A sequence that attends nothing gets out = +0 and lse = VSA_LSE_EMPTY; a head that attends
 * tokens whose weights are no numbers (a NaN among the scores, or all of them -infinity) gets
 * NaN in out, lse and the weights.  Results do not
 * depend on timing: splits of a row are joined in their order.  One kernel.
 * B * Hkv * (ceil(Hq / Hkv / 8) + 1) <= 65536. */
VSA_API vsa_status vsa_fwd_cache(const vsa_bf16 *q, const uint8_t *k_cache,
                                 const uint8_t *v_cache, const float *k_scale,
                                 const float *v_scale, const int32_t *table, const int32_t *lens,
                                 const int32_t *idx, const int32_t *num, int max_sel, int B,
                                 int Hq, int Hkv, int D, int pages, int max_blocks, int block,
                                 float scale, float keep, vsa_bf16 *out, float *lse,
                                 float *weight, void *workspace, size_t workspace_bytes,
                                 vsa_stream_t stream);

/* Workspace bytes vsa_fwd_cache needs for this shape (0 for an invalid one). */
VSA_API size_t vsa_cache_workspace_bytes(int B, int Hq, int Hkv, int max_blocks, int weight);

/* Eviction: every sequence with n = ceil(len / block) > budget blocks is cut to budget, in
 * each key/value head on its own: its first n_first and last n_last blocks stay, and of the
 * others those of the highest weight (equal ones: the lower index; NaN counts as the
 * lowest).  n_last >= 1 (the last block may be part full), n_first + n_last <= budget.
 *   table_out, weight_out  [B, Hkv, max_blocks]: the entries that stay, in their order,
 *           then -1 and 0.
 *   lens_out, n_freed      [B]: the tokens still held, and the pages that went, per head.
 *   freed   [B, Hkv, max_blocks]: the pages that went, -1 behind.
 * Pages mapped ahead of a sequence's last block (table entries from n on) are in neither
 * table_out nor freed: the caller still has them, in `table`, and has to map them, or freed
 * ones, behind the new last block before vsa_cache_write opens one there -- where no page is
 * mapped it drops the token.  This holds for sequences that lost nothing too.
 * The outputs overlap nothing: a server keeps two tables and swaps them.  Codes do not
 * move. */
VSA_API vsa_status vsa_cache_evict(const float *weight, const int32_t *table,
                                   const int32_t *lens, int B, int Hkv, int max_blocks, int block,
                                   int budget, int n_first, int n_last, int32_t *table_out,
                                   float *weight_out, int32_t *lens_out, int32_t *freed,
                                   int32_t *n_freed, vsa_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * The pages of the 8-bit cache: which are free, and who shares them.
 *
 * A pool's state is refs [pages] int32, the number of table entries that name a page, and
 * free_bits [ceil(pages / 32)] uint32, bit p % 32 of word p / 32 set where refs[p] is 0 (bits
 * past the pool are ignored).  An empty pool has refs 0 and all bits set.  Pages are taken
 * lowest first, in the order of the entries (b, h, j) that ask for them, so every outcome is
 * unique.  Calls on one pool must not overlap on the GPU.  B * Hkv, B * Hkv * max_blocks (and
 * those of N) < 2^31.
 *
 * Shared pages.  A page that several entries name is not to be written.  vsa_cache_fork shares
 * full blocks only, and a write goes behind those, so none is as long as lens only grows.  Where
 * lens is set back, what lies behind it is let go first (vsa_pages_free with lens).  It may then
 * still end inside a block that others share (drafts rejected that were there when the sequence
 * was forked): vsa_pages_reserve counts that block as lacking.  Fork the sequence, whose
 * part-full block is copied then, and go on with the fork in its place.
 * ------------------------------------------------------------------------------------- */

/* Lets pages go: every entry of table [B, Hkv, max_blocks] from block ceil(lens[b] / block) on
 * (lens NULL: every entry) becomes -1, and the page that it named loses a reference; without
 * any left it is free.  With lens, that takes back what was mapped ahead (after rejected
 * tokens, say, lens having been set back); without, it ends sequences, or takes what
 * vsa_cache_evict put in `freed`.  Entries that name no page become -1; references below 0 do
 * not arise.  One kernel. */
VSA_API vsa_status vsa_pages_free(int32_t *table, const int32_t *lens, int B, int Hkv,
                                  int max_blocks, int block, int pages, int32_t *refs,
                                  uint32_t *free_bits, vsa_stream_t stream);

/* Maps pages ahead of a write: blocks lens[b] / block .. ceil((lens[b] + n_new[b]) / block) - 1
 * (n_new NULL: one token each; at most max_blocks) that have no page in the table get one.
 *   lacking [B] output: what sequence b lacks for its tokens to come, all its heads together:
 *           pages that the pool could not give (their entries are -1, and a write drops those
 *           tokens), and the next token's block where other entries name its page too (it
 *           stays as it is; a write would change it for the others).
 * One kernel. */
VSA_API vsa_status vsa_pages_reserve(int32_t *table, const int32_t *lens, const int32_t *n_new,
                                     int B, int Hkv, int max_blocks, int block, int pages,
                                     int32_t *refs, uint32_t *free_bits, int32_t *lacking,
                                     vsa_stream_t stream);

/* N children of sequences that the cache holds (samples of one prompt, beams): child i goes on
 * from sequence parent[i] (int32 [N]; one that is not in [0, B) leaves the child empty).
 *   table_out [N, Hkv, max_blocks]: full blocks name the parent's pages, each with a reference
 *           more; a part-full last block gets a page of its own, with what the parent's holds
 *           (its tokens' codes, scales and mean); -1 behind.
 *   lens_out [N]: the parent's length.  lacking [N]: pages that the pool could not give; their
 *           entries are -1, and such a child is to be let go or forked anew.
 *   Outputs overlap nothing else.  The parents stay: vsa_pages_free(table) ends them.
 * Two kernels. */
VSA_API vsa_status vsa_cache_fork(const int32_t *table, const int32_t *lens, const int32_t *parent,
                                  int B, int N, int Hkv, int D, int max_blocks, int block,
                                  int pages, uint8_t *k_cache, uint8_t *v_cache, float *k_scale,
                                  float *v_scale, vsa_bf16 *k_mean, int32_t *refs,
                                  uint32_t *free_bits, int32_t *table_out, int32_t *lens_out,
                                  int32_t *lacking, vsa_stream_t stream);

/* Closes a pool up: with U pages in use, those from U on move to the free ones below U, in
 * order, whole (codes, scales, mean, count), and the table's entries follow.
 *   to     [pages] output: where each page in use is now, -1 for free ones; entries of other
 *          tables on the pool are to be replaced by to[entry] where they name a page (>= 0).
 *   n_used [1] output: U.  Pages from U on are free: the pool can be cut, or saved, there.
 * k_mean may be NULL.  Two kernels. */
VSA_API vsa_status vsa_cache_compact(int32_t *table, int B, int Hkv, int D, int max_blocks,
                                     int block, int pages, uint8_t *k_cache, uint8_t *v_cache,
                                     float *k_scale, float *v_scale, vsa_bf16 *k_mean,
                                     int32_t *refs, uint32_t *free_bits, int32_t *to,
                                     int32_t *n_used, vsa_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Attention over whole prompts: every query of a sequence against that sequence's keys, for
 * the prompt that fills a cache and for layers without a choice of blocks.
 *
 * Sequences.  The host does not know their lengths; int32 device arrays do.
 *   packed != 0  the sequences lie one behind the other along the token axis (the tensors have
 *                no batch axis): q_seq [B + 1] holds the first row of each and, last, the end;
 *                k_seq the same for keys and values.  Starts ascend from 0 or more; rows of no
 *                sequence are neither read into a result nor written.
 *   packed == 0  a padded batch: sequence b is rows 0 .. q_seq[b] - 1 of batch b (k_seq for
 *                keys); q_seq [B], k_seq [B], or NULL = all Sq (Sk) rows.  Rows behind a length
 *                are written: 0, and VSA_LSE_EMPTY in lse.
 *   Starts and lengths outside the tensor are clamped to it.
 * Masks.  Sequence b has nq queries and nk keys.  Query i attends the keys j < nk, and with
 * causal != 0 those with j <= i + nk - nq: the last query stands at the last key, keys in
 * front of the queries are a past that is held already, and with nk < nq the first queries
 * attend nothing.  What a tensor holds in rows of no sequence reaches no result; inside a
 * sequence, keys are expected to be finite: a NaN or infinity in v reaches all rows of the
 * query tiles that walk over it, masked or not.  (v of up to 2^60 in magnitude: weights are
 * taken relative to a maximum that may lag behind by 2^32.)
 * Tensors.  bf16 [batch, heads, tokens, 128] with strides in elements, `strides` a host array
 * of (batch, head, token) for each tensor in the order of the arguments: 128 or more,
 * multiples of 8, addresses 16-byte aligned; the stride of an axis of length 1 is free.  So
 * slices of a fused projection's output go in as they are, and outputs may be slices of one
 * buffer.  Outputs must not share elements with inputs or with one another.  (Broadcast
 * tensors, with a stride of 0, are refused: copy them first.)
 * Sizes.  Sq, Sk <= 2^31 - 1025; B * Hq, and the rows of all heads of a tensor, <= 2^40, and
 * fewer than 2^31 tiles of 128 rows; more is refused.
 * Long sums.  Products add up in fp32 in the tensor core, which drops of a term what lies some
 * 2^25 below the sum.  Where all keys of a walk weigh alike, what their v have in common comes out
 * too small by about 2^-28 of itself a key: 0.04 % at 2^18 keys, 0.4 % at 2^20, 1.1 % at 2^21, 10 %
 * at 2^24 (a rounding of out is 0.2 %).  The same holds for dv over the queries, of all heads of a
 * group, that attend a key.  Keys and queries that are cut into ranges count by the range.
 * ------------------------------------------------------------------------------------- */

/* Forward.
 *   q, out  [B or 1, Hq, Sq, D];  k, v  [B or 1, Hkv, Sk, D];  Hq a multiple of Hkv, query head
 *           hq reads key/value head hq / (Hq / Hkv).
 *   strides int64 [12]: (batch, head, token) of q, k, v, out.
 *   scale   natural-exp softmax scale (finite, > 0).
 *   lse     [Hq, Sq] (packed) or [B, Hq, Sq] fp32, base 2, contiguous, or NULL.
 *   workspace  vsa_fwd_prompt_workspace_bytes() bytes or more, 16-byte aligned, no
 *           initialisation needed; calls sharing it must not overlap on the GPU.  Where there
 *           are too few queries to keep the GPU busy, the keys are cut into ranges whose
 *           results meet there.  NULL: they are not cut (slower for few queries against many
 *           keys, and other roundings).
 * A row that attends nothing gets out = +0 and lse = VSA_LSE_EMPTY; one whose scores are no
 * numbers, or all -infinity, gets NaN.  Results do not depend on timing.  One kernel, or two
 * where keys are cut. */
VSA_API vsa_status vsa_fwd_prompt(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                                  const int64_t *strides, const int32_t *q_seq,
                                  const int32_t *k_seq, int packed, int B, int Hq, int Hkv, int Sq,
                                  int Sk, int D, int causal, float scale, vsa_bf16 *out,
                                  float *lse, void *workspace, size_t workspace_bytes,
                                  vsa_stream_t stream);

/* Workspace bytes vsa_fwd_prompt cuts keys with: 0 where it does not (or for an invalid shape). */
VSA_API size_t vsa_fwd_prompt_workspace_bytes(int packed, int B, int Hq, int Hkv, int Sq, int Sk);

/* Gradient: dq, dk, dv of vsa_fwd_prompt for an upstream gradient dout.  With p, lse of the
 * forward, D_i = dout_i . out_i and ds_ij = p_ij (dout_i . v_j - D_i):
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
 * dk and dv summed over the query heads of a key/value head.  Rows that attend nothing get
 * dq = 0 and reach no dk or dv, whatever q and dout hold there; keys that nothing attends get
 * dk = dv = 0; rows of no sequence as in the forward (packed: not written; padded: 0).  Of rows
 * that attend something, a NaN or infinity in q or dout reaches dk and dv of all keys of the key
 * tiles that their query tile walks over.
 *   q, k, v, q_seq, k_seq, sizes, causal, scale: as given to the forward; out, lse what it
 *           returned; dout as out.  Where k and v are a part of the keys that a row attends (a
 *           piece of a long past, or another rank's), out and lse are those over all parts,
 *           joined: p and D are then the whole's, dk and dv the part's, and dq adds up over the
 *           parts.
 *   strides int64 [24]: (batch, head, token) of q, k, v, out, dout, dq, dk, dv.
 *   workspace  vsa_bwd_prompt_workspace_bytes() bytes, 16-byte aligned, no initialisation
 *           needed; calls sharing it must not overlap on the GPU.
 * No atomics: results do not depend on timing.  Two kernels, and one more for each of dq and
 * (dk, dv) where there are too few tiles of them to keep the GPU busy. */
VSA_API vsa_status vsa_bwd_prompt(const vsa_bf16 *q, const vsa_bf16 *k, const vsa_bf16 *v,
                                  const vsa_bf16 *out, const vsa_bf16 *dout, const float *lse,
                                  const int64_t *strides, const int32_t *q_seq,
                                  const int32_t *k_seq, int packed, int B, int Hq, int Hkv, int Sq,
                                  int Sk, int D, int causal, float scale, vsa_bf16 *dq,
                                  vsa_bf16 *dk, vsa_bf16 *dv, void *workspace,
                                  size_t workspace_bytes, vsa_stream_t stream);

/* Workspace bytes vsa_bwd_prompt needs for this shape (0 for an invalid one). */
VSA_API size_t vsa_bwd_prompt_workspace_bytes(int packed, int B, int Hq, int Hkv, int Sq, int Sk);

/* Synchronises `stream`, then reads and clears the device status word of the current
 * device: VSA_OK, or VSA_ERR_DEVICE_TIMEOUT if a kernel gave up on a wait since the
 * last call (`detail`, if not NULL, receives the recorded code). */
VSA_API vsa_status vsa_device_status(vsa_stream_t stream, unsigned int *detail);

/* Number of kernel launches the most recent successful forward call on this thread
 * enqueued (for accounting in benchmarks). */
VSA_API int vsa_last_launch_count(void);

/* Test hooks for the timeout path (failure detection without a GPU fault).  Both are
 * process-wide settings read when a forward or backward kernel is launched; they change
 * no result of a launch that completes.  (The pages have no counterpart.)
 *   vsa_set_wait_limit_ns(ns): the limit of every internal wait that is not a drain
 *     (a drain waits for the kernel's own copies and MMAs in flight and always keeps the
 *     full limit of about one second, so nothing is in flight when a CTA exits).
 *     0 restores the full limit (vsa_fwd_prompt: a second more for every 2^25 keys).  A short
 *     limit makes waits run out on ordinary work.
 *   vsa_set_stall_test(enable): while nonzero, the MMA warp of every CTA first waits on
 *     a barrier that nothing ever completes; that wait runs out after the limit above,
 *     records its code in the device status word (forward 0x11f, backward 0x15f), and
 *     every role of the CTA returns.  The launch's outputs are then undefined and
 *     vsa_device_status() reports VSA_ERR_DEVICE_TIMEOUT. */
VSA_API void vsa_set_wait_limit_ns(unsigned long long ns);
VSA_API void vsa_set_stall_test(int enable);

/* Static text for a status code. */
VSA_API const char *vsa_status_str(vsa_status s);

#ifdef __cplusplus
}
#endif

#endif /* VSA_GB300_H */
