/*
 * paged_attn.h -- C ABI of libpagedattn.so: paged (block-table) KV-cache
 * append and attention on one NVIDIA GB300 (sm_103a).
 *
 * The operations follow the I/O contract of onnxruntime/mobius PR #395
 * "Add paged / block-table KV cache export" (sections "How it works (per
 * attention layer)" and "ONNX I/O contract"): new K/V rows are scattered
 * into a per-layer page pool at slot_mapping (ScatterND), and attention
 * reads a sequence's pages through block_table (Gather) with causal and
 * padding masking given by nonpad_kv_seqlen (here: seq_lens).  The batched,
 * row-padded block_table, seq_lens and query_start_loc follow the vLLM-shaped
 * metadata of ROCm/maxtext PR #93 "[Draft] kv paged kernels" (the
 * attention='gpu_paged' commit).
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensor arguments are DEVICE pointers on the current CUDA device,
 *   owned by the caller.  The library allocates no device memory and keeps
 *   no per-call state.  Its state: one device-side error word per device
 *   (see paged_device_error); a process-wide note of whether the runtime
 *   accepts the decode kernel's cooperative launch (learnt on the first eager
 *   decode launch); and, for paged_attention_decode_cascade only, one extra
 *   stream and two events per (host thread, device), created by the first
 *   cascade call on that thread and kept for the thread's life.
 * - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *   default stream).  Host-side argument checks run before any launch; on a
 *   non-PA_OK return nothing was launched.
 * - Kernels are launched with programmatic stream serialization, and wait for
 *   the kernel before them (griddepcontrol.wait) ahead of every read, with one
 *   exception: the paged_attention_decode and paged_attention_prefill calls
 *   without a window (and their other forms) read lengths and page tables, and
 *   the prefills queries, ahead of it.  A caller's kernel directly before such a
 *   call that writes one of these must not let its dependents start early
 *   (griddepcontrol.launch_dependents); the library's kernels that write them do
 *   not.
 * - Pool layout (NHD): key_pool and value_pool are each
 *   [num_pages, page_size, num_kv_heads, head_dim], contiguous, element type
 *   `dtype`.  The flat slot s = page_id * page_size + offset addresses row s
 *   of the pool viewed as [num_pages * page_size, num_kv_heads, head_dim].
 * - GQA/MQA: num_q_heads must be a multiple of num_kv_heads; query head h
 *   reads KV head h / (num_q_heads / num_kv_heads).
 * - The softmax scale is a required argument (there is no default 1/sqrt(d)):
 *   a query that already carries its scale is passed with scale = 1.0.
 * - There is no attention-bias or ALiBi argument: those are unsupported, not
 *   silently ignored.  A sliding window is an argument of the _window calls
 *   only.
 * - Device-side checks: a block_table entry outside [0, num_pages), a slot
 *   >= num_pages * page_size, or a seq_len outside [0, max_blocks_per_seq *
 *   page_size] is recorded in the device error word and the offending read
 *   or write is skipped (no trap, no hang).
 */
#ifndef PAGED_ATTN_H_
#define PAGED_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PA_ABI_VERSION 2

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_NULL = 1,         /* a required pointer is NULL                        */
  PA_ERR_SHAPE = 2,        /* inconsistent or negative sizes                    */
  PA_ERR_DTYPE = 3,        /* unknown dtype                                     */
  PA_ERR_RANGE = 4,        /* a size is beyond what the kernels index (int32)   */
  PA_ERR_UNSUPPORTED = 5,  /* valid but not implemented (head_dim, page_size)   */
  PA_ERR_CUDA = 6,         /* a CUDA runtime call failed (launch, attribute)    */
  PA_ERR_WORKSPACE = 7,    /* workspace missing or smaller than required        */
  PA_ERR_ALIGN = 8         /* a pointer is not aligned as the dtype requires    */
} pa_status;

typedef enum pa_dtype {
  PA_DTYPE_F32 = 0,        /* float32 pool, q and out                           */
  PA_DTYPE_BF16 = 1,       /* bfloat16 pool, q and out; fp32 accumulation       */
  PA_DTYPE_FP8_E4M3 = 2,   /* e4m3 pool with k_scale / v_scale; bf16 q, out and
                              appended rows                                     */
  PA_DTYPE_INT8 = 3        /* int8 pool with a scale for each block of tokens and
                              KV head (pa_kv_scales); bf16 q, out and appended
                              rows.  Taken by the _int8 calls,
                              paged_attention_decode_mass and
                              paged_kv_copy_pages only                          */
} pa_dtype;

/* One layer's KV page pool (mobius PR #395 "ONNX I/O contract":
 * key_pool.{i} / value_pool.{i}).  All fields are read-only to the library
 * except the pool contents, which paged_kv_append updates in place. */
typedef struct pa_kv_pool {
  void* key_pool;          /* device [num_pages, page_size, num_kv_heads, head_dim] */
  void* value_pool;        /* device, same shape and dtype                           */
  int64_t num_pages;       /* > 0; num_pages * page_size < 2^31                      */
  int32_t page_size;       /* tokens per page, > 0                                   */
  int32_t num_kv_heads;    /* > 0                                                    */
  int32_t head_dim;        /* > 0                                                    */
  int32_t dtype;           /* pa_dtype                                               */
  /* e4m3 pools only (ignored otherwise): a stored code c stands for
   * e4m3(c) * scale; finite and > 0.  The pages name an fp8 KV cache (mobius
   * build features, maxtext pool-sizing table) without a scheme; one scale per
   * pool and tensor is the plainest one. */
  float k_scale;
  float v_scale;
} pa_kv_pool;

/*
 * paged_kv_append -- the ScatterND write (mobius PR #395, "How it works",
 * step 1; the aiter AppendKvJA step of maxtext PR #93).
 *
 *   for t in [0, num_tokens):  if slot_mapping[t] >= 0:
 *       key_pool.flat[slot_mapping[t]]   = key[t]
 *       value_pool.flat[slot_mapping[t]] = value[t]
 *
 * key, value    device [num_tokens, num_kv_heads, head_dim], pool dtype
 *               (bf16 for an e4m3 pool, 16-byte aligned: each element x is
 *               stored as e4m3_rn_satfinite(float32(x) / float32(scale)) --
 *               round to nearest even, magnitudes past 448 saturate, NaN
 *               stays NaN -- with the pool's k_scale / v_scale).
 * slot_mapping  device int64 [num_tokens]; entry = page_id * page_size +
 *               offset.  A negative entry marks a padding token (skipped).
 *               Entries must be unique within one call (otherwise which
 *               row lands is unspecified).  An entry >= num_pages*page_size
 *               is recorded in the device error word and skipped.
 * num_tokens    >= 0; 0 launches nothing.
 * The write is a bit copy (for f32 / bf16 pools): the pool afterwards is
 * bit-identical to the ScatterND result.
 */
pa_status paged_kv_append(const pa_kv_pool* pool, const void* key, const void* value,
                          const int64_t* slot_mapping, int64_t num_tokens, void* stream);

/*
 * paged_attention_decode -- one query token per sequence, attending to all
 * seq_lens[b] keys of its pages (mobius PR #395: Gather(pool, block_table)
 * then Attention with nonpad_kv_seqlen; decode is the one-token case).
 *
 *   out[b, h] = sum_j softmax_j(scale * q[b,h] . K_b[j, h/G]) V_b[j, h/G],
 *   j in [0, seq_lens[b]),  K_b[j] = key_pool[block_table[b, j / page_size],
 *                                             j % page_size]
 *
 * q, out        device [batch, num_q_heads, head_dim], pool dtype.  out may
 *               not alias q.  A sequence with seq_lens[b] == 0 gets out = 0.
 * block_table   device int32 [batch, max_blocks_per_seq], row-padded; entries
 *               past ceil(seq_lens[b] / page_size) are never read.
 * seq_lens      device int32 [batch], the KV length including this step's
 *               appended token (append first, then attend).
 * max_seq_len   host upper bound of seq_lens (used to size the launch).
 * workspace     device scratch of at least
 *               paged_attention_decode_workspace_size(...) bytes (may be NULL
 *               when that size is 0), 16-byte aligned, owned by the caller and
 *               not shared by calls in flight at the same time.  Its
 *               contents need no initialisation: each call writes every
 *               partial it reads, and the per-segment arrival counters that
 *               schedule the merge of a segment cut across CTAs carry a tag
 *               derived from a per-launch epoch kept at the workspace's start
 *               (each launch reads it and stores the next), so a word left by
 *               any earlier launch, a CUDA graph replay included, or never
 *               written counts as zero.  The merge runs inside the one
 *               decode kernel (no second launch).
 * The decode kernel is a persistent grid of at most one CTA per SM, launched
 * cooperatively (all CTAs resident at once: the CTAs that computed the parts
 * of a cut segment each merge a slice of it), so its start can wait for SMs
 * held by kernels on other streams.  Where the runtime refuses that launch,
 * the CTA that counts a segment's last part merges the whole segment.
 * bf16 path (tensor cores): page_size a power of two >= 8, head_dim in
 * {64, 128}, at most 32 query heads per KV head, q 16-byte aligned, at most
 * 2^31 - 1 slots (num_pages * page_size) per pool and batch *
 * ceil(max_seq_len / 16) below 2^31 (PA_ERR_RANGE beyond);
 * e4m3 pools: the bf16 limits; q and out are bf16; the attention is that of
 * the values the codes stand for (scale * k_scale * q . e4m3(K), outputs
 * times v_scale), computed with f16 products (every e4m3 value is an f16);
 * CUDA-core path (fp32 arithmetic, one key at a time; correct, not fast):
 * f32 pools, and bf16 pools of any other page_size (1, 2, 4, or not a power
 * of two); head_dim <= 256, no workspace used.
 */
size_t paged_attention_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             int32_t dtype);

pa_status paged_attention_decode(const pa_kv_pool* pool, const void* q, void* out,
                                 int32_t batch, int32_t num_q_heads,
                                 const int32_t* block_table, int32_t max_blocks_per_seq,
                                 const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * CSR page tables.  paged_attention_decode_csr / paged_attention_prefill_csr
 * are paged_attention_decode / paged_attention_prefill with each sequence's
 * pages given in the compressed form of NVIDIA/recsys-examples PR #400
 * (KVCacheMetadata: kv_indices, kv_indptr, kv_last_page_len) instead of a
 * row-padded block_table and seq_lens:
 *
 *   pages of sequence b = kv_indices[kv_indptr[b] .. kv_indptr[b+1]),
 *   L_b = (kv_indptr[b+1] - kv_indptr[b] - 1) * page_size + kv_last_page_len[b]
 *         (0 when the sequence has no page),
 *
 * i.e. the last page holds kv_last_page_len[b] tokens, 1 .. page_size.
 *
 * kv_indptr         device int32 [batch + 1], non-decreasing, kv_indptr[0] >= 0,
 *                   kv_indptr[batch] <= num_kv_indices.
 * kv_indices        device int32 [num_kv_indices], physical page ids.
 * kv_last_page_len  device int32 [batch].
 * max_seq_len       host upper bound of every L_b.
 * Device contents the host cannot check: a slice of kv_indptr outside
 * [0, num_kv_indices] or running backwards is treated as an empty sequence and
 * a kv_last_page_len outside [1, page_size] is clamped; both are recorded in
 * the device error word (code 3, see paged_device_error).  Every other argument, and the
 * workspace of the decode call (paged_attention_decode_workspace_size), is as
 * for the row-padded calls.
 */
pa_status paged_attention_decode_csr(const pa_kv_pool* pool, const void* q, void* out,
                                     int32_t batch, int32_t num_q_heads,
                                     const int32_t* kv_indptr, const int32_t* kv_indices,
                                     int64_t num_kv_indices, const int32_t* kv_last_page_len,
                                     int32_t max_seq_len, float scale, void* workspace,
                                     size_t workspace_bytes, void* stream);

pa_status paged_attention_prefill_csr(const pa_kv_pool* pool, const void* q, void* out,
                                      int32_t batch, int32_t num_q_heads,
                                      const int32_t* query_start_loc, int64_t total_q,
                                      int32_t max_q_len, const int32_t* kv_indptr,
                                      const int32_t* kv_indices, int64_t num_kv_indices,
                                      const int32_t* kv_last_page_len, int32_t max_seq_len,
                                      float scale, void* stream);

/*
 * paged_attention_decode_cascade -- decode for a batch whose sequences all
 * begin with the same prefix on the same physical pages (block tables that
 * alias the pages of a common prompt prefix: the RadixAttention case of
 * mobius PR #395, summary; the page-granular prefix index of ROCm/maxtext
 * PR #93, prefix cache (M5) commit).  Sequence b attends to
 *
 *   the prefix_len tokens on prefix_block_ids, then
 *   its own seq_lens[b] tokens on block_table[b, ...],
 *
 * i.e. exactly paged_attention_decode over the concatenated key lists.  The
 * prefix is read once for all B query rows (one tensor-core pass with its keys
 * cut into chunks, fp32 partials) instead of once per sequence; each sequence's
 * own tokens go through the split-KV decode, and the partials of both are
 * merged per row.  The prefix pass runs on a second stream of the library's,
 * forked from `stream` and joined back to it with events (so stream order and
 * stream capture hold); that stream is created by the first cascade call on a
 * host thread, which must therefore come before any stream capture there.
 *
 * prefix_block_ids  device int32 [ceil(prefix_len / page_size)], the shared
 *                   pages in order (the prefix may end inside its last page).
 * prefix_len        tokens of the shared prefix, >= 0; 0 runs plain decode.
 * block_table, seq_lens, max_blocks_per_seq, max_seq_len
 *                   the sequences' OWN pages and token counts (excluding the
 *                   prefix); a sequence with seq_lens[b] == 0 attends to the
 *                   prefix alone.
 * q, out, scale     as for paged_attention_decode.
 * workspace         device scratch of at least
 *                   paged_attention_decode_cascade_workspace_size(...) bytes,
 *                   16-byte aligned; contents need no initialisation.
 * bf16 pools only (PA_ERR_UNSUPPORTED for f32), with the tensor-core limits
 * of paged_attention_decode (a page_size that is not a power of two >= 8
 * gives PA_ERR_UNSUPPORTED when prefix_len > 0).
 */
size_t paged_attention_decode_cascade_workspace_size(int32_t batch, int32_t num_q_heads,
                                                     int32_t num_kv_heads, int32_t head_dim,
                                                     int32_t dtype);

pa_status paged_attention_decode_cascade(const pa_kv_pool* pool, const void* q, void* out,
                                         int32_t batch, int32_t num_q_heads,
                                         const int32_t* prefix_block_ids, int32_t prefix_len,
                                         const int32_t* block_table, int32_t max_blocks_per_seq,
                                         const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * paged_attention_decode_append -- one decode step in one launch: the append
 * of this step's K/V rows (paged_kv_append with one token per sequence) and
 * the decode that attends to them (mobius PR #395, "How it works (per
 * attention layer)": step 1 writes the new rows, step 2 attends).  The
 * result equals paged_kv_append(pool, key, value, slot_mapping, batch)
 * followed by paged_attention_decode(...) with the same arguments, provided
 *   (a) slot_mapping[b] >= 0 is the slot of sequence b's last key, position
 *       seq_lens[b] - 1 (block_table[b][(L-1)/page_size] * page_size +
 *       (L-1) % page_size) -- the new token of a decode step; and
 *   (b) no slot written by the call is a key of another sequence.
 * The new rows are written to the pool and, for each sequence, attended to
 * straight from key/value (the pool row is not read back).  An entry
 * breaking (a) is recorded in the device error word (code 2, detail = the
 * slot) and that sequence's output then attends to the new row in place of
 * its last key.  slot_mapping[b] < 0: sequence b has no new token (its keys
 * are all in the pool already).
 *
 * key, value    device [batch, num_kv_heads, head_dim] bf16 (f32 for f32
 *               pools), 16-byte aligned; e4m3 pools store their codes
 *               (quantised as paged_kv_append does).
 * slot_mapping  device int64 [batch], 8-byte aligned.
 * Every other argument, limit and the workspace are those of
 * paged_attention_decode.  The CUDA-core path (f32 pools, bf16 pools of
 * other page sizes) runs the append and the decode as two launches.
 */
pa_status paged_attention_decode_append(const pa_kv_pool* pool, const void* key, const void* value,
                                        const int64_t* slot_mapping, const void* q, void* out,
                                        int32_t batch, int32_t num_q_heads,
                                        const int32_t* block_table, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * paged_attention_decode_static_scratch -- paged_attention_decode without a
 * caller-provided workspace.  The pages have no counterpart of this call: it
 * exists for callers that cannot allocate device memory, such as a plugin in
 * an inference runtime that owns all device memory and hands its plugins no
 * allocator, or a latency-critical serving loop that may not take
 * cudaMalloc's implicit synchronisation mid-step.
 *
 * The split-KV partials go to a file-scope device array of
 * PA_DECODE_STATIC_SCRATCH_BYTES that the library holds on every GPU that
 * loads it, until the process exits.  The call allocates nothing (no
 * cudaMalloc, no cudaFree, no allocating library routine).
 * - The first call on a device looks up the array's device address with
 *   that device current (cudaGetSymbolAddress); make that first call before
 *   any stream capture on the device.
 * - All calls share the one array, which keeps the last call's contents;
 *   calls whose kernels overlap on the GPU (different streams, or unordered
 *   host threads) race on it.  No part of it needs to start zeroed.
 * - The stream must belong to the current device (the array's address is
 *   that device's); a stream of another device gives PA_ERR_CUDA and nothing
 *   is launched.
 * - bf16 and e4m3 pools only (PA_ERR_UNSUPPORTED for f32, whose decode needs no
 *   workspace anyway).  A call whose partials would not fit, i.e. when
 *   paged_attention_decode_workspace_size(...) exceeds
 *   PA_DECODE_STATIC_SCRATCH_BYTES, returns PA_ERR_WORKSPACE and launches
 *   nothing.
 * Arguments, layout and results are those of paged_attention_decode.
 */
#define PA_DECODE_STATIC_SCRATCH_BYTES (8u << 20)

pa_status paged_attention_decode_static_scratch(const pa_kv_pool* pool, const void* q, void* out,
                                                int32_t batch, int32_t num_q_heads,
                                                const int32_t* block_table,
                                                int32_t max_blocks_per_seq,
                                                const int32_t* seq_lens, int32_t max_seq_len,
                                                float scale, void* stream);

/*
 * paged_attention_prefill -- varlen causal attention for a packed batch of
 * new tokens (query_start_loc layout of maxtext PR #93's vLLM-shaped
 * metadata; causal + padding masks from is_causal=1 and nonpad_kv_seqlen of
 * mobius PR #395).
 *
 * Sequence b owns packed rows [query_start_loc[b], query_start_loc[b+1]) of
 * q; with n_b rows and L_b = seq_lens[b], its row i is the token at absolute
 * position p = L_b - n_b + i and attends to keys 0..p of its pages (the new
 * tokens are the last n_b of the sequence, already appended).  A row with
 * p < 0 gets out = 0.
 *
 * q, out           device [total_q, num_q_heads, head_dim], pool dtype.
 * query_start_loc  device int32 [batch + 1], non-decreasing, [0] = 0,
 *                  [batch] = total_q.
 * max_q_len        host upper bound of n_b (sizes the launch).
 * block_table, seq_lens, max_seq_len, scale: as for decode.
 * bf16 path (tensor cores): page_size a power of two >= 8, head_dim in
 * {64, 128}, at most 32 query heads per KV head;
 * e4m3 pools: the bf16 limits, q 16-byte aligned; q and out are bf16; the
 * attention is that of the values the codes stand for (scale * k_scale *
 * q . e4m3(K), outputs times v_scale), computed with f16 products: q is
 * rounded to f16 (exact for bf16 values of magnitude 2^-14 .. 65504; larger
 * ones become infinite), the codes are exact in f16, and the softmax weights are
 * rounded to f16;
 * CUDA-core path (fp32 arithmetic): f32 pools, and bf16 pools of any other
 * page_size; head_dim <= 256.
 */
pa_status paged_attention_prefill(const pa_kv_pool* pool, const void* q, void* out,
                                  int32_t batch, int32_t num_q_heads,
                                  const int32_t* query_start_loc, int64_t total_q,
                                  int32_t max_q_len, const int32_t* block_table,
                                  int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                  int32_t max_seq_len, float scale, void* stream);

/*
 * paged_attention_decode_window / paged_attention_prefill_window --
 * paged_attention_decode / paged_attention_prefill with a sliding window and
 * sinks: a query at absolute position p (decode: p = seq_lens[b] - 1) attends
 * to key j iff
 *
 *   j <= p  and  (j > p - window  or  j < num_sinks),
 *
 * i.e. to the last `window` keys up to its own and to the sequence's first
 * num_sinks keys.  The pages have no counterpart of these calls.
 *
 * window        >= 1 (1: a query's own key and the sinks).
 * num_sinks     >= 0.  Position indices are those of the whole sequence: keys
 *               are not renumbered.
 * block_table   as for the plain calls, with one difference: an entry whose
 *               page holds no key that some query row of the sequence attends
 *               to is never read, so the pages between the sinks and the
 *               window may have been freed (any value, -1 included).  An
 *               entry out of range elsewhere is recorded (code 1) and the keys
 *               of its page take no part (slower; a row without a key left
 *               gives 0).
 * Slots of read pages that no query row of the sequence attends to may hold
 * anything, NaN included.  Keys and values that a row of the sequence attends
 * to must be finite, as for the plain calls.
 * Every other argument, limit, type, the workspace and the results are those
 * of the plain calls; where the window reaches every key (window or num_sinks
 * >= max_seq_len) the plain kernels run, and only there is the workspace used.
 * Tensor-core pools: out is 8-byte aligned (decode), q and out are 16-byte
 * aligned (prefill, which takes at most 2^31 - 1 slots per pool).  As in the
 * plain calls the softmax weights go into the second product as bf16 (e4m3
 * pools: f16), and the queries of an e4m3 pool into the first as f16: they are
 * at most 65504 in magnitude.
 */
pa_status paged_attention_decode_window(const pa_kv_pool* pool, const void* q, void* out,
                                        int32_t batch, int32_t num_q_heads,
                                        const int32_t* block_table, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                        int32_t window, int32_t num_sinks, void* workspace,
                                        size_t workspace_bytes, void* stream);

pa_status paged_attention_prefill_window(const pa_kv_pool* pool, const void* q, void* out,
                                         int32_t batch, int32_t num_q_heads,
                                         const int32_t* query_start_loc, int64_t total_q,
                                         int32_t max_q_len, const int32_t* block_table,
                                         int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                         int32_t max_seq_len, float scale, int32_t window,
                                         int32_t num_sinks, void* stream);

/*
 * paged_qk_norm_rope_append -- what a layer does between its qkv product and
 * its attention, in one pass over the rows: the RMS norm of each query and key
 * head, the rotation by position, and the append of the new K/V rows.  The
 * pages have no counterpart of this call.  For token t with
 * s = slot_mapping[t] >= 0 and p = positions[t]:
 *
 *   q_out[t, h]        = R_p(norm(q[t, h], q_weight))
 *   key_pool.flat[s]   = R_p(norm(key[t, h], k_weight))    for every KV head h
 *   value_pool.flat[s] = value[t]
 *   norm(x, w)         = x / sqrt(mean(x^2) + eps) * w   (x itself when w is NULL)
 *
 * R_p turns the pairs of the first rotary_dim dims, with c_i =
 * cos_sin[p, i] and s_i = cos_sin[p, rotary_dim / 2 + i]:
 *   (x_a, x_b) -> (x_a c_i - x_b s_i, x_b c_i + x_a s_i),
 *   (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved = 1;
 * the other dims pass through.  All arithmetic is fp32 with one rounding to
 * the output's type; an e4m3 pool stores the code of the fp32 quotient by its
 * scale (as paged_kv_append rounds).  The value rows are what paged_kv_append
 * writes.
 *
 * q, key, value  device rows of num_q_heads / num_kv_heads heads of head_dim
 *                contiguous elements (f32 for f32 pools, else bf16); token t
 *                starts at t * q_stride (key_stride, value_stride) elements, so
 *                slices of one qkv product can be passed.  Strides are at
 *                least a row long.
 * q_out          device [num_tokens, num_q_heads, head_dim], the rows' type; q
 *                itself when its rows are contiguous, else memory that no row
 *                of q, key or value overlaps (PA_ERR_SHAPE).  No input overlaps
 *                the pools.
 * q_weight, k_weight  device [head_dim], the rows' type, or NULL: no norm.
 * eps            >= 0, finite.
 * positions      device int32 [num_tokens], each in [0, max_position).
 * cos_sin        device f32 [max_position, rotary_dim].
 * rotary_dim     a multiple of 8, at most head_dim; 0: no rotation (positions
 *                and cos_sin may be NULL).
 * slot_mapping   as for paged_kv_append; a negative entry marks a padding
 *                token: its position may be anything and nothing of it is
 *                written (its q_out row is left as it was).
 * A slot or position out of range is recorded in the device error word (codes
 * 2 and 6) and that token is skipped like a padding token.
 * head_dim a multiple of 8, at most 256 (PA_ERR_UNSUPPORTED); any alignment
 * of the element type.  The fast path: 16-byte aligned rows of f32 heads, or of
 * bf16 heads whose head_dim and rotary_dim are multiples of 16; for many tokens
 * (four an SM or more) also a token's rows of q, key, value and cos_sin of at most
 * 14,336 bytes together (32 + 8 + 8 bf16 heads of 128 take 12,800; wider ones run
 * at 0.71 to 0.87 of the copy rate, not 0.85).
 */
pa_status paged_qk_norm_rope_append(const pa_kv_pool* pool, const void* q, int64_t q_stride,
                                    const void* key, int64_t key_stride, const void* value,
                                    int64_t value_stride, void* q_out, int32_t num_q_heads,
                                    const void* q_weight, const void* k_weight, float eps,
                                    const int32_t* positions, const float* cos_sin,
                                    int64_t max_position, int32_t rotary_dim, int32_t interleaved,
                                    const int64_t* slot_mapping, int64_t num_tokens, void* stream);

/*
 * paged_kv_copy_pages -- copy whole pages inside the pools of all layers: in
 * every pool of `pools`, K and V, page dst_pages[i] becomes page src_pages[i].
 * A fork of a sequence shares its full pages and copies the page that both
 * sequences will go on writing; defragmentation moves pages.  The pages name
 * no such call.
 *
 * pools         host array of num_pools descriptors (at most 1024), e.g. one
 *               per layer, read before the call returns: all of one geometry
 *               and dtype, no two tensors of them overlapping (PA_ERR_SHAPE).
 *               Any dtype: pages are copied bit for bit.
 * src_pages, dst_pages  device int32 [num_copies].  A pair with a negative
 *               entry is padding (skipped); a pair with src = dst copies
 *               nothing; an entry >= num_pages is recorded in the device error
 *               word (code 1) and the pair is skipped.  The pairs run in no
 *               order: a destination page must appear once and must not be the
 *               source of another pair (else which contents land there is
 *               unspecified).
 */
pa_status paged_kv_copy_pages(const pa_kv_pool* pools, int32_t num_pools, const int32_t* src_pages,
                              const int32_t* dst_pages, int64_t num_copies, void* stream);

/*
 * paged_kv_compact -- keep a part of each sequence's rows, moved together in
 * place, in the pools of all layers: eviction of cached keys, or the accepted
 * tokens of a verified draft.  With keep_b = keep[keep_indptr[b] ..
 * keep_indptr[b+1]) and n_b its length, row base[b] + i of sequence b (through
 * its block_table row) becomes its old row keep_b[i], i in [0, n_b), and
 *
 *   new_seq_lens[b] = base[b] + n_b.
 *
 * Rows below base[b] stay; rows at or past the new length are left as they
 * were, and the pages past ceil(new_seq_lens[b] / page_size) are free for other
 * use.  Keys move as stored: a rotation by position stays that of the old
 * position.  The pages name no such call.
 *
 * pools         as for paged_kv_copy_pages, at least one.
 * block_table   device int32 [batch, max_blocks_per_seq]; pages that hold rows
 *               written here must not be shared by two sequences (copy them
 *               first).  batch <= 65535.
 * seq_lens      device int32 [batch]: the lengths before the call.
 * base          device int32 [batch] in [0, seq_lens[b]], or NULL: all 0.
 * keep_indptr   device int32 [batch + 1], non-decreasing, within [0, num_keep].
 * keep          device int32 [num_keep]: old positions, strictly ascending per
 *               sequence, in [base[b], seq_lens[b]).
 * new_seq_lens  device int32 [batch], written; NULL: not wanted.  May not
 *               overlap the inputs (PA_ERR_SHAPE).
 * A position that is not ascending or out of range is recorded in the device
 * error word (code 7) and its row is not moved; a sequence whose length or base
 * (code 3) or slice of keep (code 7) is out of range is left as it was, with
 * its length; a block_table entry out of range (code 1) skips the row.
 */
pa_status paged_kv_compact(const pa_kv_pool* pools, int32_t num_pools, const int32_t* block_table,
                           int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch,
                           const int32_t* base, const int32_t* keep_indptr, const int32_t* keep,
                           int64_t num_keep, int32_t* new_seq_lens, void* stream);

/*
 * int8 pools.  key_pool and value_pool hold int8 codes (PA_DTYPE_INT8, the
 * layout of every pool); code c of slot s and KV head h stands for
 *
 *   c * scales[s / block_tokens, h],
 *
 * with scales of their own for keys and values.  A scale counts as
 * min(max(scale, 2^-40), 2^40).  The pages have no counterpart of these calls.
 *
 * key_scales, value_scales  device f32 [num_pages * page_size / block_tokens,
 *               num_kv_heads], 16-byte aligned.
 * block_tokens  a power of two, 16 .. page_size.
 * All calls on int8 pools: page_size a power of two >= 16, head_dim in
 * {64, 128} (PA_ERR_UNSUPPORTED else), at most 2^31 - 1 slots, pools 16-byte
 * aligned.  paged_kv_copy_pages copies their pages; their scales are a pool of
 * dtype f32, page_size page_size / block_tokens and head_dim 1 to it.
 * paged_kv_compact refuses them: rows that share a scale cannot move alone
 * (paged_kv_evict_pages drops whole pages).
 */
typedef struct pa_kv_scales {
  float* key_scales;
  float* value_scales;
  int32_t block_tokens;
} pa_kv_scales;

/*
 * paged_kv_append_int8 -- write each token's K/V rows into an int8 pool and keep
 * the scales of the blocks that they lie in.  For a block of which this call
 * writes rows, a KV head and a tensor, with a the largest magnitude of those rows
 * (NaN aside) in that head:
 *
 *   n = min(max(a / 127, 2^-40), 2^40)
 *   new scale s = n                when the call writes the block's first slot,
 *               = max(scale, n)    else;
 *   the rows written get the codes rint(x / s), at most 127 in magnitude (NaN
 *   becomes 0); where s is larger than the scale before, the codes c of the
 *   block's other rows become rint(c * (scale / s)).
 *
 * Arithmetic is fp32 (one division, rounding to nearest even).  A row's code is off by
 * half a step of the scale that it is written under, and by half a step more of each
 * larger scale that it is re-encoded under later, once a call that raises it.  A block's first
 * slot is the first that a sequence writes, so a page taken into use again
 * starts anew; its slots not yet written may hold anything, and are left or
 * re-encoded.
 *
 * key, value    device bf16 rows of num_kv_heads heads of head_dim contiguous
 *               elements, 16-byte aligned; token t starts at t * key_stride
 *               (value_stride) elements, multiples of 8, at least a row.
 * slot_mapping  as for paged_kv_append.  The tokens of one block must follow one
 *               another in the call (as those of a sequence do; up to 31 padding
 *               tokens may stand between two): else the block's codes and scale
 *               are unspecified, its other rows' codes among them, and nothing is
 *               recorded.  Two tokens of one slot: which of them lands is
 *               unspecified, as for paged_kv_append.
 */
pa_status paged_kv_append_int8(const pa_kv_pool* pool, const pa_kv_scales* scales, const void* key,
                               int64_t key_stride, const void* value, int64_t value_stride,
                               const int64_t* slot_mapping, int64_t num_tokens, void* stream);

/*
 * paged_attention_decode_int8 / paged_attention_prefill_int8 --
 * paged_attention_decode / paged_attention_prefill over an int8 pool: the
 * attention of the values that the codes stand for.  Products are f16 with fp32
 * sums: the codes are exact, the queries are rounded to f16 (exact for bf16 values
 * of magnitude 2^-14 .. 65504, their largest), and so is each softmax weight times
 * its V scale, relative to the largest such product among the keys that the row sees.
 * The keys of a page that is out of range take no part.
 * out is 8-byte aligned (decode), q and out are 16-byte aligned (prefill).  Every
 * other argument, limit, the workspace (dtype PA_DTYPE_INT8) and the results are
 * those of the plain calls.
 */
pa_status paged_attention_decode_int8(const pa_kv_pool* pool, const pa_kv_scales* scales,
                                      const void* q, void* out, int32_t batch, int32_t num_q_heads,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                      void* workspace, size_t workspace_bytes, void* stream);

pa_status paged_attention_prefill_int8(const pa_kv_pool* pool, const pa_kv_scales* scales,
                                       const void* q, void* out, int32_t batch, int32_t num_q_heads,
                                       const int32_t* query_start_loc, int64_t total_q,
                                       int32_t max_q_len, const int32_t* block_table,
                                       int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                       int32_t max_seq_len, float scale, void* stream);

/*
 * paged_attention_decode_mass -- a decode that also gives the attention weight of
 * every key, summed over the query heads and added to what the key had:
 *
 *   mass_out[b, j] = decay * mass_in[b, j] + sum_h softmax_j(scale * q[b,h] . K_b[j, h/G]),
 *   j in [0, seq_lens[b]); entries at and past seq_lens[b] are left as they were.
 *   The keys of a page that is out of range take no part, whatever the pool's type: their
 *   weight is 0.
 *
 * Summed over the layers or steps that share a block table, it says which keys
 * the queries still look at (paged_kv_evict_rows, paged_kv_evict_pages).  The sum
 * is fp32, in an order of its own that is the same on every run.  The pages have no
 * counterpart of this call.
 *
 * pool, scales  bf16, e4m3 (scales NULL) or int8 pools, with the limits of their
 *               decode calls; PA_ERR_UNSUPPORTED for f32 pools and for pages that
 *               the tensor-core kernels do not take.
 * mass_in       device f32 [batch, mass_stride] rows, mass_out itself, or NULL: 0.
 *               Rows that overlap mass_out otherwise are refused (PA_ERR_SHAPE).
 * decay         finite; 1 adds, between 1 and 0 old weights fade, 0: mass_in is not read.
 * mass_out      device f32, rows mass_stride >= max_seq_len apart.
 * max_seq_len   at most 2^31 - 1024 (PA_ERR_RANGE); a longer sequence is cut to it and
 *               recorded (code 3).  The workspace has 4 bytes for each query head and
 *               key up to it: pass the longest length rather than what the table holds.
 * workspace     paged_attention_decode_mass_workspace_size(...) bytes, 16-byte
 *               aligned, contents need no initialisation.
 * out is 8-byte aligned.  Every other argument is as for paged_attention_decode.
 */
size_t paged_attention_decode_mass_workspace_size(int32_t batch, int32_t num_q_heads,
                                                  int32_t num_kv_heads, int32_t head_dim,
                                                  int32_t dtype, int32_t max_seq_len);

pa_status paged_attention_decode_mass(const pa_kv_pool* pool, const pa_kv_scales* scales,
                                      const void* q, void* out, int32_t batch, int32_t num_q_heads,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                      const float* mass_in, float decay, float* mass_out,
                                      int64_t mass_stride, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * paged_kv_evict_rows -- choose the rows that stay, by their accumulated weight:
 * a sequence of more than `budget` rows keeps its first num_sinks, its last
 * num_recent and, of the others, the heaviest budget - num_sinks - num_recent
 * (equal ones by the lower position; NaN counts as the lightest).  The result is
 * what paged_kv_compact takes:
 *
 *   base[b] = num_sinks and keep[keep_indptr[b] ..] = the other rows that stay,
 *   ascending (budget - num_sinks of them), for a sequence over its budget;
 *   base[b] = seq_lens[b] and an empty list for one that stays whole;
 *   new_mass[b, :] = the masses of the rows that stay, in order, then zeros up to
 *   `width`: what the next steps add to.
 *
 * The pages have no counterpart of these calls.
 *
 * mass, new_mass  device f32 [batch, width], rows mass_stride / new_mass_stride >=
 *               width apart; a sequence longer than width is cut to it and
 *               recorded (code 3).  width is at most 2^31 - 65536 (PA_ERR_RANGE).
 * budget        >= num_sinks + num_recent (PA_ERR_SHAPE).
 * keep_indptr   device int32 [batch + 1], written.   base  device int32 [batch], written.
 * keep          device int32 [num_keep], num_keep >= batch * (budget - num_sinks) (0
 *               when width <= budget); entries past keep_indptr[batch] are left.
 * Outputs overlap neither inputs nor one another (PA_ERR_SHAPE).
 */
pa_status paged_kv_evict_rows(const float* mass, int64_t mass_stride, const int32_t* seq_lens,
                              int32_t batch, int32_t width, int32_t budget, int32_t num_sinks,
                              int32_t num_recent, int32_t* keep_indptr, int32_t* keep,
                              int64_t num_keep, int32_t* base, float* new_mass,
                              int64_t new_mass_stride, void* stream);

/*
 * paged_kv_evict_pages -- the same by whole pages, for pools of any type; no row is
 * moved.  A sequence of more than `budget` pages keeps those that hold its first
 * num_sinks and its last max(num_recent, 1) rows and the heaviest of the others, a
 * page's weight being the sum of its rows' (x[0 .. n/2) + x[n/2 .. n) again and
 * again, rows at and past seq_lens[b] counting 0).
 *
 *   new_block_table[b, :] = the pages that stay, in order, then those that go, in
 *   order, then the entries behind the sequence as they were;
 *   new_seq_lens[b] = seq_lens[b] - page_size * (pages that go): entries from
 *   ceil(new_seq_lens[b] / page_size) to the old number of pages are free;
 *   new_mass as above.
 *
 * Keys keep the rotation of their old position, as with paged_kv_compact.
 * page_size     a power of two, at most 1024 (PA_ERR_UNSUPPORTED).
 * budget        in pages, at least ceil(num_sinks / page_size) + 1 +
 *               (max(num_recent, 1) + page_size - 2) / page_size (PA_ERR_SHAPE): the most
 *               pages that the rows kept in any case lie in.
 * At most 327,424 pages a sequence and 2^31 - 65536 columns of the table (PA_ERR_RANGE).
 */
pa_status paged_kv_evict_pages(const float* mass, int64_t mass_stride, const int32_t* block_table,
                               int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch,
                               int32_t width, int32_t page_size, int32_t budget, int32_t num_sinks,
                               int32_t num_recent, int32_t* new_block_table, int32_t* new_seq_lens,
                               float* new_mass, int64_t new_mass_stride, void* stream);

/*
 * paged_device_error -- read and clear the device error word of the current
 * device.  Synchronises the device.  *code = 0 when no violation was seen,
 * else 1 = block_table / kv_indices entry out of range, 2 = slot out of
 * range, 3 = seq_len (or CSR kv_indptr / kv_last_page_len) out of range,
 * 4 = query_start_loc inconsistent, 5 = a bounded wait inside a kernel gave
 * up, 6 = position out of range, 7 = compaction list inconsistent; *detail
 * holds the offending value.  Either pointer may be NULL.
 */
pa_status paged_device_error(int64_t* code, int64_t* detail);

/*
 * pa_testing_decode_part_wait -- TEST HOOK, not for production use: the pages
 * have no counterpart.  paged_attention_decode (bf16 and e4m3 pools, same
 * arguments, same workspace) with the one wait inside the decode kernel that
 * depends on other CTAs -- a CTA holding part of a sequence's keys waits for
 * the other CTAs' parts before merging its slice of the rows -- given the
 * limit `wait_ns` (1 us .. 2 s; every public call uses 2 s) and
 * `extra_parts` (0 .. 1024) parts added to the count each such wait expects.
 * With extra_parts > 0 those parts never arrive, so every such wait runs out
 * after wait_ns: the kernel records code 5 (a bounded wait gave up) in the
 * device error word, finishes without those parts and returns; the outputs
 * of the affected sequences are then unspecified.  It exists so that the
 * failure path of the bounded wait can be exercised without a fault or a
 * hang; a later call on the same workspace is unaffected.  PA_ERR_RANGE for
 * a limit or count outside the ranges above.
 */
pa_status pa_testing_decode_part_wait(const pa_kv_pool* pool, const void* q, void* out,
                                      int32_t batch, int32_t num_q_heads,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                      void* workspace, size_t workspace_bytes, uint64_t wait_ns,
                                      int32_t extra_parts, void* stream);

/* Human-readable name of a status code (static storage). */
const char* pa_status_string(int32_t status);

/* PA_ABI_VERSION of the loaded library. */
int32_t pa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_H_ */
