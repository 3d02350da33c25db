/*
 * pkv.h -- C ABI of the paged-KV continuous-batching decode step (GB300, sm_103a).
 *
 * One decode step appends one token to every row of a batch and attends over
 * each row's cached keys/values.  It has four device parts and one host part:
 *
 *   a0  host block allocator: positions, slot_mapping, seq_lens, block tables
 *   a1  pkv_rope               rotate-half RoPE of the new q and k at per-row positions
 *   a2  pkv_append             write rotated k and raw v into the cache slot
 *   a3  pkv_decode_attn_split  grouped-query attention through block tables,
 *                              split over a page-balanced partition, online softmax
 *   a4  pkv_lse_merge          log-sum-exp merge of the split partials
 *
 * Sources: "neurogrid releases" v0.7.0 (paged KV cache in fixed 16-token blocks,
 * O(1) block allocator with per-sequence block tables, paged attention with GQA),
 * v0.6.0 (flash decode: online softmax over KV tiles), v0.8.0 (kv_len =
 * position + 1 computed on the GPU, zero device-to-host copies, every kernel on
 * one caller stream); helexa issue 121 "continuous batching -- batched decode +
 * engine", slice 1 (per-row RoPE positions, rotate-half, keys stored post-RoPE,
 * additive (B,1,1,S) mask over each row's padding gap); "cortex-engine writeup",
 * block-sparse attention kernel (a row with zero softmax denominator outputs
 * zeros instead of NaN).
 *
 * Conventions
 *  - Every call returns PKV_OK (0) or a PKV_ERR_* code; pkv_last_error()
 *    returns a message for the calling thread's last failure.
 *  - The library never allocates device memory.  The caller owns every device
 *    buffer and the CUDA stream.  Device calls are asynchronous on `stream`
 *    (a cudaStream_t passed as void*, NULL = legacy default stream), make no
 *    device-to-host copy (the host-step calls at the end of this header are
 *    the exception: they return the result in host memory) and check
 *    cudaGetLastError after each launch.
 *  - Every tensor is dense and row-major in the layout stated.  dtype is
 *    PKV_F32 or PKV_BF16 and applies to q, k, v, the caches and the output.
 *  - dev_err_flag (nullable, device int32): kernels that meet an out-of-range
 *    block id, slot or length atomically OR a PKV_DEVERR_* bit into it and skip
 *    that access instead of faulting.  The caller clears it.
 *  - The allocator is host-only and not thread-safe: one owner per allocator.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define PKV_OK 0
#define PKV_ERR_INVALID_ARG 1   /* null pointer, bad size, bad stride, duplicate row */
#define PKV_ERR_OUT_OF_BLOCKS 2 /* the free list cannot satisfy the request; nothing changed */
#define PKV_ERR_UNKNOWN_SEQ 3   /* sequence id not live */
#define PKV_ERR_UNSUPPORTED 4   /* dtype, head_dim, group size or block size not built */
#define PKV_ERR_CUDA 5          /* a CUDA runtime/driver call failed; see pkv_last_error */

#define PKV_F32 0
#define PKV_BF16 1

#define PKV_BLOCK_SIZE 16       /* tokens per KV block ("neurogrid releases" v0.7.0) */

/* bits OR-ed into dev_err_flag */
#define PKV_DEVERR_BAD_BLOCK 1  /* a block table entry outside [0, num_blocks) */
#define PKV_DEVERR_BAD_SLOT 2   /* a slot outside [0, num_blocks * 16) */
#define PKV_DEVERR_BAD_LEN 4    /* seq_len < 0, or longer than bt_stride*16 or bias_stride */
#define PKV_DEVERR_TIMEOUT 8    /* an internal pipeline wait gave up (never expected) */
#define PKV_DEVERR_BAD_PLAN 16  /* a plan does not fit the call, or (PKV_ATTN_CHECK_PLAN) it
                                   disagrees with the metadata */

/* flags for the attention calls */
#define PKV_ATTN_SIMT 1         /* use the CUDA-core consumer instead of mma.sync (bf16 only;
                                   f32 always uses CUDA cores) */
#define PKV_ATTN_SEPARATE_MERGE 2 /* leave the split partials for pkv_lse_merge instead of
                                     merging them in the split kernel's epilogue */
#define PKV_STEP_FUSED 4          /* pkv_decode_step: run a1+a2 inside the attention kernel
                                     (one launch per step) instead of as their own kernel */
#define PKV_ATTN_SHORT_WAITS 8    /* diagnostic: every wait inside the attention kernel gives
                                     up after ~64 SM clocks instead of ~1 s, so the timeout
                                     path can be exercised (PKV_DEVERR_TIMEOUT is set, the
                                     output is incomplete, every copy the kernel issued still
                                     lands before it exits); the workspace must be zero-filled
                                     again before its next use */
#define PKV_ATTN_CHECK_PLAN 16    /* with a plan: also derive the partition from the metadata
                                     in the kernel, set PKV_DEVERR_BAD_PLAN where the plan
                                     disagrees and use the derived one there */
#define PKV_LAYERS_MERGE_HELPERS 32 /* pkv_decode_step_layers: launch each layer's attention
                                     kernel cooperatively, so that the merge of a unit split
                                     over many parts is shared by its last parts as in a
                                     single-layer call (otherwise its last part merges it
                                     alone).  Worth it for long rows; the next layer's
                                     attention kernel then starts only once the previous one
                                     has left the GPU.  Ignored by the other calls. */

/* Message for the calling thread's last failed call ("" if none). */
const char *pkv_last_error(void);
/* ABI version of this header (bumped on any signature change). */
int pkv_abi_version(void);

/* ======================================================================== */
/* a0: host block allocator                                                  */
/* ======================================================================== */
/*
 * Policy ("neurogrid releases" v0.7.0: constant-time block allocation and
 * release, one block table per sequence; v0.8.0: kv_len = position + 1):
 *  - The free list is a stack, seeded bottom-to-top with `initial_free` (a
 *    permutation of 0..num_blocks-1; NULL = 0,1,2,...).  Pop takes the top.
 *  - join pops ceil(prefix_len/16) blocks in table order and takes the
 *    smallest free sequence id; leave pushes the sequence's blocks in table
 *    order and frees its id.
 *  - prepare_step appends one token to each listed sequence: position = L
 *    (cached length before the step); if L % 16 == 0 a block is popped first;
 *    slot = table[L/16]*16 + L%16; the length becomes L+1.
 *  - A request that cannot be met returns PKV_ERR_OUT_OF_BLOCKS and changes
 *    nothing.  Each pop/push is O(1).
 */
typedef struct pkv_alloc pkv_alloc;

/* block_size must be 16.  max_blocks_per_seq bounds each block table.
 * On success *out owns the allocator (free with pkv_alloc_destroy). */
int pkv_alloc_create(int32_t num_blocks, int32_t block_size, int32_t max_seqs,
                     int32_t max_blocks_per_seq, const int32_t *initial_free,
                     pkv_alloc **out);
void pkv_alloc_destroy(pkv_alloc *a);

/* A new sequence whose first prefix_len tokens are already in its blocks
 * (their contents are written by the caller, e.g. by a prefill). */
int pkv_seq_join(pkv_alloc *a, int32_t prefix_len, int32_t *seq_id);
int pkv_seq_leave(pkv_alloc *a, int32_t seq_id);

/* Several joins in one call (one host call per step for a serving loop that
 * admits many sequences): the same as pkv_seq_join(prefix_lens[i]) for i = 0..n-1
 * in order, into seq_ids[i].  If positions and slot_mapping are given they receive,
 * packed one sequence after another, the positions and cache slots of every
 * joiner's prefix tokens [0, prefix_lens[i]) (sum(prefix_lens) entries, as
 * pkv_seq_slots gives them): the input of pkv_prefill_kv.  All or nothing: if
 * the sequence ids, the pool or a table cannot take every joiner, nothing
 * changes (PKV_ERR_OUT_OF_BLOCKS when the pool is short). */
int pkv_seqs_join(pkv_alloc *a, const int32_t *prefix_lens, int32_t n, int32_t *seq_ids,
                  int32_t *positions, int64_t *slot_mapping);
/* Several leaves in one call: pkv_seq_leave(seq_ids[i]) for i = 0..n-1 in order.
 * All or nothing: every id must be live and listed once, else nothing changes. */
int pkv_seqs_leave(pkv_alloc *a, const int32_t *seq_ids, int32_t n);

/*
 * Host part of one decode step for the B listed (distinct, live) sequences.
 * Outputs (host arrays, row b = seq_ids[b]):
 *   positions[B]      int32  position of the new token (= cached length before, plus the
 *                            sequence's offset, pkv_seq_set_offset)
 *   slot_mapping[B]   int64  cache slot of the new token
 *   seq_lens[B]       int32  length after the append (what attention reads)
 *   block_tables[B*bt_stride] int32, row-major, padded with -1
 * Atomic: on any error nothing changes.
 */
int pkv_prepare_step(pkv_alloc *a, const int32_t *seq_ids, int32_t B,
                     int32_t *positions, int64_t *slot_mapping, int32_t *seq_lens,
                     int32_t *block_tables, int32_t bt_stride);
/* The same step, for a block_tables buffer that is rewritten step after step:
 * row_state (int32 [B*3], all -1 before the first call on a fresh buffer, then
 * kept by the caller with that buffer) records which sequence, join and table
 * length each row of the buffer holds, and only the entries that differ are
 * written (a row whose sequence stayed gets just its new blocks; a row that
 * changed sequence is rewritten and its stale entries set to -1).  The buffer
 * then holds exactly what pkv_prepare_step would have written.  Every output
 * and all allocator state are the same as pkv_prepare_step's. */
int pkv_prepare_step_cached(pkv_alloc *a, const int32_t *seq_ids, int32_t B,
                            int32_t *positions, int64_t *slot_mapping, int32_t *seq_lens,
                            int32_t *block_tables, int32_t bt_stride, int32_t *row_state);

int pkv_seq_len(const pkv_alloc *a, int32_t seq_id, int32_t *len);
/* Copies up to cap block ids of the sequence's table into out; *n = table length. */
int pkv_seq_blocks(const pkv_alloc *a, int32_t seq_id, int32_t *out, int32_t cap,
                   int32_t *n);
/* Positions and cache slots of tokens [start, start+count) of a live sequence
 * (already covered by its blocks: start+count <= its length), for writing a
 * prefix chunk with pkv_prefill_kv.  positions[i] = start+i,
 * slot_mapping[i] = table[p/16]*16 + p%16.  PKV_ERR_INVALID_ARG if the range
 * is negative or beyond the length; nothing is changed. */
int pkv_seq_slots(const pkv_alloc *a, int32_t seq_id, int32_t start, int32_t count,
                  int32_t *positions, int64_t *slot_mapping);
/* Positions that run ahead of the cached length.  A sequence's next token sits at
 * position length + offset (0 at join): pkv_seq_set_offset sets the offset (a
 * sequence behind a shared prefix: the prefix's length; offset >= 0), and
 * pkv_prepare_step's positions include it.  Slots, lengths and tables do not. */
int pkv_seq_set_offset(pkv_alloc *a, int32_t seq_id, int32_t offset);
int pkv_seq_offset(const pkv_alloc *a, int32_t seq_id, int32_t *offset);
/* After pkv_evict: sequence seq_ids[i] now holds keep_lens[i] tokens (if it held
 * more; else nothing changes for it).  The blocks behind them return to the free
 * list in table order, and the offset grows by the tokens dropped, so that
 * positions go on where they were.  All or nothing: every id must be live and
 * listed once, every keep_lens[i] >= 0, and a sequence that gets shorter must share no
 * block (pkv_seq_fork): its tokens have moved within them. */
int pkv_seqs_evict(pkv_alloc *a, const int32_t *seq_ids, const int32_t *keep_lens, int32_t n);
/* Forks of a sequence (several samples of one prompt, beams): n new sequences with the
 * parent's tokens and offset, into child_ids[0..n-1] (smallest free ids, ascending).  Whole
 * blocks are shared: a block then belongs to several sequences and is free when the last
 * of them has given it back.  A last block that is not full is the parent's alone: every
 * child gets a block of its own for it, and pair i of the *n_copies pairs copy_src,
 * copy_dst (room for n each; they may be NULL where the length is a multiple of 16) says
 * which to copy (pkv_copy_blocks, in every layer, before the next step).  All or nothing.
 * So the block that a sequence appends to is always its own. */
int pkv_seq_fork(pkv_alloc *a, int32_t seq_id, int32_t n, int32_t *child_ids, int32_t *copy_src,
                 int32_t *copy_dst, int32_t *n_copies);
/* Sequences cut back to lens[i] tokens (at most what they have): the tokens behind are
 * forgotten, positions go on from there, and the blocks behind return to the free list in
 * table order (after pkv_tree_accept: the drafted tokens that were not accepted).  A
 * sequence that then ends inside a block which it shares gets a block of its own, to be
 * copied as in pkv_seq_fork (copy_src, copy_dst: room for n, or NULL where no block is
 * shared).  All or nothing; PKV_ERR_OUT_OF_BLOCKS unless the free list has a block for
 * each such sequence. */
int pkv_seqs_truncate(pkv_alloc *a, const int32_t *seq_ids, const int32_t *lens, int32_t n,
                      int32_t *copy_src, int32_t *copy_dst, int32_t *n_copies);
/*
 * Host part of a step that appends counts[b] tokens (0 or more) to each of the B listed
 * (distinct, live) sequences: T = sum(counts) new tokens (the nodes of a tree of drafted
 * tokens, a chunk of a prompt), packed row after row.  Outputs (host arrays):
 *   positions[T]      length before + offset + depths[i] (depths NULL: the token's number
 *                     in its row)
 *   slot_mapping[T]   int64 cache slots of the new tokens
 *   node_starts[B+1]  row b's new tokens are [node_starts[b], node_starts[b+1])
 *   seq_lens[B], block_tables[B*bt_stride] as pkv_prepare_step, after the append
 * Atomic: on any error nothing changes.
 */
int pkv_prepare_nodes(pkv_alloc *a, const int32_t *seq_ids, int32_t B, const int32_t *counts,
                      const int32_t *depths, int32_t *positions, int64_t *slot_mapping,
                      int32_t *node_starts, int32_t *seq_lens, int32_t *block_tables,
                      int32_t bt_stride);
/* Another size of the pool.  Larger: the new blocks come onto the free list, the last of
 * them on top.  Smaller: blocks in use from num_blocks on move to free ones ahead of it,
 * taken from the top of the free list; pair i of the *n pairs src, dst (room for cap) says
 * what to copy (pkv_copy_blocks, in every layer), sequences in the order of their ids,
 * blocks in table order; the rest of the free list keeps its order.  Then tables hold the
 * new ids.  All or nothing: PKV_ERR_OUT_OF_BLOCKS if more blocks are in use than num_blocks,
 * PKV_ERR_INVALID_ARG if cap is too small (*n is then what it must be).  Not for an allocator
 * that a pkv_server manages (its captured steps name the caches). */
int pkv_alloc_resize(pkv_alloc *a, int32_t num_blocks, int32_t *src, int32_t *dst, int32_t cap,
                     int32_t *n);
/* The pairs that pkv_alloc_resize with these arguments would give (and its refusals); nothing
 * changes.  For a caller who copies into the new pools first and takes the new size once
 * that has succeeded. */
int pkv_alloc_resize_pairs(const pkv_alloc *a, int32_t num_blocks, int32_t *src, int32_t *dst,
                           int32_t cap, int32_t *n);
/* shared[i]: the blocks of sequence seq_ids[i] that belong to another one too.  (To be asked
 * before anything moves tokens within a sequence's blocks: pkv_evict.) */
int pkv_seqs_shared(const pkv_alloc *a, const int32_t *seq_ids, int32_t n, int32_t *shared);
/* Sequences that a block belongs to (0: it is free). */
int pkv_block_refs(const pkv_alloc *a, int32_t block, int32_t *refs);
int pkv_num_free(const pkv_alloc *a, int32_t *n);
/* Pool auto-sizing ("neurogrid releases" v0.7.0: the pool is sized from the
 * VRAM budget): the number of 16-token blocks whose K and V, for every KV head
 * and every one of n_layers layers, fit in budget_bytes (floor; host only). */
int pkv_pool_blocks(uint64_t budget_bytes, int32_t n_layers, int32_t Hkv, int32_t d,
                    int32_t dtype, int32_t *num_blocks);
/* Copies the free stack bottom-to-top (up to cap entries); *n = its size. */
int pkv_alloc_dump(const pkv_alloc *a, int32_t *free_stack, int32_t cap, int32_t *n);

/* Device calls.  Tensors are device memory, except that the integer index
 * arrays (positions, slot_mapping, seq_lens, block_tables) -- and the new q, k,
 * v of pkv_decode_step -- may instead be page-locked host memory at its mapped
 * address (pkv_mapped_pointer): the kernels then read them in place over the
 * CPU-GPU link, and the host must not rewrite them until those kernels have
 * finished.  All calls are asynchronous
 * on `stream` (a cudaStream_t; NULL = the legacy default stream). */

/* ======================================================================== */
/* a1: RoPE (helexa issue 121, slice 1: batch_cos_sin at per-row positions,   */
/*     rotate-half apply)                                                    */
/* ======================================================================== */
/*
 * q [B,Hq,d], k [B,Hkv,d] -> q_out [B,Hq,d], k_out [B,Hkv,d] (device, dtype).
 * For pair i < d/2 at position p = positions[b]:
 *   theta = p * base^(-2i/d)
 *   out[i]     = x[i] cos(theta) - x[i+d/2] sin(theta)
 *   out[i+d/2] = x[i+d/2] cos(theta) + x[i] sin(theta)
 * theta is formed modulo 2*pi exactly (64-bit fixed-point turns from a
 * double-precision host table), then rotated in float32 and rounded once to
 * dtype.  In-place (q_out == q) is allowed.
 * d even, 2 <= d <= 256.
 */
int pkv_rope(const void *q, const void *k, void *q_out, void *k_out,
             const int32_t *positions, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
             float base, int32_t dtype, void *stream);

/* ======================================================================== */
/* a2: append ("neurogrid releases" v0.7.0: fixed 16-token blocks)           */
/* ======================================================================== */
/*
 * k_cache, v_cache: [num_blocks, Hkv, 16, d] (device, dtype).
 * For each row b with slot = slot_mapping[b] >= 0:
 *   k_cache[slot/16, h, slot%16, :] = k_rot[b, h, :]
 *   v_cache[slot/16, h, slot%16, :] = v[b, h, :]
 * A negative slot appends nothing (padding row).  A slot >= num_blocks*16 sets
 * PKV_DEVERR_BAD_SLOT and is skipped.  d*sizeof(dtype) must be a multiple of 16.
 */
int pkv_append(const void *k_rot, const void *v, const int64_t *slot_mapping,
               void *k_cache, void *v_cache, int32_t B, int32_t Hkv, int32_t d,
               int32_t num_blocks, int32_t dtype, int32_t *dev_err_flag, void *stream);

/*
 * a1 + a2 fused: one launch that rotates q and k as pkv_rope does and writes
 * the rotated key and the raw value into the cache slot as pkv_append does
 * (k_out still receives the rotated key).  Same argument rules as the two calls.
 */
int pkv_rope_append(const void *q, const void *k, const void *v, void *q_out, void *k_out,
                    const int32_t *positions, const int64_t *slot_mapping, void *k_cache,
                    void *v_cache, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                    int32_t num_blocks, float base, int32_t dtype, int32_t *dev_err_flag,
                    void *stream);

/*
 * Prefix KV of joining sequences (chunked prefill's cache write): T tokens,
 * each with its raw key k[t, Hkv, d], value v[t, Hkv, d], position
 * positions[t] and cache slot slot_mapping[t] (pkv_seq_slots gives both for a
 * chunk of one sequence; chunks of several sequences may be concatenated).
 * The key is rotated at its position exactly as pkv_rope_append rotates a
 * decode token (bit-identical rows), then both are written to the slot.
 * Same argument rules as pkv_rope_append; there is no query and no rotated-key
 * output.  Writes nothing but the T slots; a negative slot writes nothing.
 */
int pkv_prefill_kv(const void *k, const void *v, const int32_t *positions,
                   const int64_t *slot_mapping, void *k_cache, void *v_cache, int32_t T,
                   int32_t Hkv, int32_t d, int32_t num_blocks, float base, int32_t dtype,
                   int32_t *dev_err_flag, void *stream);

/* ======================================================================== */
/* a3 + a4: split-KV paged GQA decode attention and its LSE merge            */
/* ("neurogrid releases" v0.7.0 paged attention with GQA, v0.6.0 flash       */
/*  decode; "cortex-engine writeup" zero-denominator guard)                  */
/* ======================================================================== */
/*
 * Row b attends over its first seq_lens[b] tokens (the token appended in this
 * step included).  Token t of row b is row t%16 of block
 * block_tables[b*bt_stride + t/16].  Query head h uses KV head h / (Hq/Hkv).
 *   s_t   = (q_rot[b,h] . k_t) * scale + attn_bias[b*bias_stride + t]
 *   out   = sum_t softmax(s)_t v_t            (float32 accumulation)
 * attn_bias (device float32, nullable) is additive; -inf excludes a token (the
 * value at an excluded token must still be finite).  A row with no tokens, or
 * whose tokens are all excluded, outputs zeros.
 *
 * Partition: the (row, KV head) units, in row-major order, are laid end to
 * end as positions: a unit of n pages takes n + A positions, the first A
 * without a page (A, the cost of a unit boundary in pages: 4 at d = 64, 2 at
 * d = 128).  With P positions in all, part c of num_parts owns positions
 * [floor(c*P/num_parts), floor((c+1)*P/num_parts)) and the pages in them, and
 * runs as one CTA, so parts balance pages plus unit boundaries.  A unit whose
 * pages lie in one part is written to `out` directly.  Every other
 * unit leaves one float32 (o, lse) partial per part it touches in `workspace`;
 * the LSE merge (M = max lse; out = sum exp(lse_s - M) o_s / sum exp(lse_s - M))
 * then combines them.  By default the merge runs in the epilogue of
 * pkv_decode_attn_split, so `out` is complete when the call's kernel ends:
 * the last H parts of a unit to finish each merge a slice of its output
 * columns (H <= 32, at least 8 float4 columns each).  H > 1 only when the
 * grid fits on the GPU at once (num_parts <= the resident CTAs, which the
 * default partition always does): the kernel is then launched cooperatively,
 * so the helpers may wait for each other; otherwise the last part to finish
 * merges the unit alone.  With PKV_ATTN_SEPARATE_MERGE the
 * split kernel stops at the partials and pkv_lse_merge must follow with the
 * same arguments.  pkv_lse_merge may also be called after a fused call: it
 * recomputes the same merge from the partials left in the workspace.
 *
 * Workspace: pkv_attn_workspace_bytes(...) bytes, 256-byte aligned, owned by
 * the caller, ZERO-FILLED ONCE after allocation (it holds the fused merge's
 * per-unit counters, which every call leaves at zero).  Calls that share a
 * workspace must not overlap on the GPU.
 *
 * Supported: dtype PKV_BF16 or PKV_F32; d in {64, 128}; Hq/Hkv in {1,2,4,8};
 * B <= 65536.  q_rot [B,Hq,d] (16-byte aligned); out [B,Hq,d] (device, dtype,
 * 16-byte aligned).
 * num_parts <= 0 selects pkv_attn_default_parts(d, Hq, Hkv, dtype, flags) for the
 * current device (every SM holding as many CTAs as fit: the kernel variant,
 * and so the count, depends on the head dimension, the group size Hq/Hkv, the
 * dtype and PKV_ATTN_SIMT); at most 4096 parts.
 */
int pkv_attn_default_parts(int32_t d, int32_t Hq, int32_t Hkv, int32_t dtype, int32_t flags,
                           int32_t *num_parts);
int pkv_attn_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                             int32_t num_parts, size_t *bytes);

int pkv_decode_attn_split(const void *q_rot, const void *k_cache, const void *v_cache,
                          int32_t num_blocks, const int32_t *block_tables,
                          int32_t bt_stride, const int32_t *seq_lens,
                          const float *attn_bias, int32_t bias_stride, int32_t B,
                          int32_t Hq, int32_t Hkv, int32_t d, float scale,
                          int32_t num_parts, void *workspace, size_t workspace_bytes,
                          void *out, int32_t dtype, int32_t flags,
                          int32_t *dev_err_flag, void *stream);

/*
 * Attention without a caller-provided workspace.  This call has no
 * counterpart in the pages the method comes from; it exists for callers that
 * cannot allocate device memory (code running under another runtime's memory
 * manager, plugins that are handed only their input and output tensors, or
 * paths that must never reach an allocator).  It computes the same result as
 * pkv_decode_attn_split followed by its fused merge (same arguments, minus
 * the workspace) and takes its scratch from a 16 MiB array compiled into this
 * library; calls needing more scratch than that fail with
 * PKV_ERR_UNSUPPORTED.  It performs no device allocation or free.
 *  - Every GPU that loads the library holds the 16 MiB array until the
 *    process exits.
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - All calls share the one array, which keeps the previous call's contents;
 *    each call clears the bytes it uses first (an asynchronous memset on
 *    `stream`).  Calls that overlap on the GPU (other streams, other host
 *    threads) race on the array and give wrong results: serialise them.
 *  - PKV_ATTN_SEPARATE_MERGE is rejected (the merge always runs in-kernel).
 */
int pkv_decode_attn_static(const void *q_rot, const void *k_cache, const void *v_cache,
                           int32_t num_blocks, const int32_t *block_tables, int32_t bt_stride,
                           const int32_t *seq_lens, const float *attn_bias, int32_t bias_stride,
                           int32_t B, int32_t Hq, int32_t Hkv, int32_t d, float scale,
                           int32_t num_parts, void *out, int32_t dtype, int32_t flags,
                           int32_t *dev_err_flag, void *stream);

/*
 * Host-planned partition.  Without a plan, every CTA of the attention kernel
 * first reads all row lengths (to find where its part starts) and then the
 * block ids of its first pages: two dependent reads before its first page
 * load, each a round trip over the CPU-GPU link when the step's metadata is
 * read in place from host memory.  The host that prepared the metadata (a0)
 * can state the same partition instead: pkv_plan_parts writes one record of
 * PKV_PLAN_INTS int32 per part, and the kernel then makes one read before it
 * loads pages.  Record c (part c of num_parts):
 *   [0] first row b0 of the part (-1: the part owns no position)
 *   [1] positions of the rows before b0, per KV head (sum of n_b + A over
 *       rows b < b0 with n_b > 0 pages; A = 4 at d = 64, 2 at d = 128)
 *   [2] seq_lens[b0], [3] seq_lens[b0 + 1] (0 past the last row)
 *   [4], [5] P, the total position count (int64, low word first)
 *   [6], [7] zero
 *   [8 + i], i < 16: block id of page j0 + i of the part's first unit segment
 *       (j0 its first page there); entries past the segment's last page are
 *       not written (and not read)
 * The plan is a pure function of (seq_lens, block tables, B, Hkv, d,
 * bt_stride, bias_stride, num_parts): it must come from the very metadata the
 * kernel reads, and be rebuilt whenever that changes.  PKV_ATTN_CHECK_PLAN
 * makes the kernel verify it.  Host-only; plan is [num_parts * PKV_PLAN_INTS].
 */
#define PKV_PLAN_INTS 24
int pkv_plan_parts(const int32_t *seq_lens, int32_t B, int32_t Hkv, int32_t d,
                   const int32_t *block_tables, int32_t bt_stride, int32_t bias_stride,
                   int32_t num_parts, int32_t *plan);

/* pkv_decode_attn_split with a plan from pkv_plan_parts (device or mapped
 * pointer; num_parts must be the plan's).  Same results, bit for bit.  Without
 * PKV_ATTN_CHECK_PLAN and without attn_bias the launch runs a smaller build of
 * the kernel (no row-length scan, plan check or bias code), which is faster:
 * the plan is the fast path. */
int pkv_decode_attn_planned(const void *q_rot, const void *k_cache, const void *v_cache,
                            int32_t num_blocks, const int32_t *block_tables,
                            int32_t bt_stride, const int32_t *seq_lens,
                            const float *attn_bias, int32_t bias_stride, int32_t B,
                            int32_t Hq, int32_t Hkv, int32_t d, float scale,
                            int32_t num_parts, const int32_t *plan, void *workspace,
                            size_t workspace_bytes, void *out, int32_t dtype, int32_t flags,
                            int32_t *dev_err_flag, void *stream);

/* bt_stride and bias_stride (0 when no bias was given) are the values passed to
 * pkv_decode_attn_split: they decide which rows are valid, exactly as there. */
int pkv_lse_merge(const void *workspace, size_t workspace_bytes, const int32_t *seq_lens,
                  int32_t bt_stride, int32_t bias_stride, int32_t B, int32_t Hq,
                  int32_t Hkv, int32_t d, int32_t num_parts, void *out, int32_t dtype,
                  void *stream);

/* ======================================================================== */
/* rotary positions in other layouts and scalings, with the append           */
/* ======================================================================== */
/*
 * What pkv_rope_append does for whole heads in the rotate-half layout, for the
 * other ways in which heads carry positions.  Pair i < rot_dim/2 of a head at
 * position p turns by theta = p * f_i:
 *   PKV_ROTARY_HALF         (x1, x2) = (x[i], x[i + rot_dim/2])
 *   PKV_ROTARY_INTERLEAVED  (x1, x2) = (x[2i], x[2i+1])
 *   x1' = amplitude * (x1 cos - x2 sin),  x2' = amplitude * (x2 cos + x1 sin)
 * Elements from rot_dim on are copied.  With g_i = base^(-2i/rot_dim):
 *   PKV_ROTARY_PLAIN   f_i = g_i
 *   PKV_ROTARY_LINEAR  f_i = g_i / factor
 *   PKV_ROTARY_NTK     f_i = g_i with base * factor^(rot_dim/(rot_dim-2)) for base
 *   PKV_ROTARY_RAMP    f_i = g_i (1-w) + g_i/factor w, w = clamp((i-lo)/(hi-lo), 0, 1),
 *                      lo = max(0, floor(D(high))), hi = min(rot_dim-1, ceil(D(low))),
 *                      D(t) = rot_dim ln(original_len/(2 pi t)) / (2 ln base): the pair
 *                      that makes t turns over original_len (hi - lo is at least 0.001)
 *   PKV_ROTARY_BANDS   f_i = s g_i + (1-s) g_i/factor, s = clamp((t_i-low)/(high-low), 0, 1),
 *                      t_i = original_len g_i/(2 pi), the turns of pair i
 * Angles are formed modulo 2*pi exactly, as pkv_rope forms them (positions may
 * be negative here), rotated in float32 and rounded once to dtype; PLAIN over
 * the whole head in the HALF layout gives pkv_rope's values bit for bit.
 */
#define PKV_ROTARY_HALF 0
#define PKV_ROTARY_INTERLEAVED 1
#define PKV_ROTARY_PLAIN 0
#define PKV_ROTARY_LINEAR 1
#define PKV_ROTARY_NTK 2
#define PKV_ROTARY_RAMP 3
#define PKV_ROTARY_BANDS 4

typedef struct pkv_rotary_spec {
  int32_t rot_dim;                   /* rotated elements at the front of a head: even, 2..d */
  int32_t layout;                    /* PKV_ROTARY_HALF, PKV_ROTARY_INTERLEAVED */
  int32_t scaling;                   /* PKV_ROTARY_PLAIN .. PKV_ROTARY_BANDS */
  int32_t original_len;              /* RAMP, BANDS: the trained length, > 0 */
  double base;                       /* >= 1 (> 1 for RAMP) */
  double factor;                     /* >= 1 (unused by PLAIN) */
  double low, high;                  /* RAMP, BANDS: turns, 0 < low < high */
  double amplitude;                  /* > 0 and finite in float32; 1 for none */
} pkv_rotary_spec;

/* What the kernels need of a spec, filled by pkv_rotary_init (host only) and
 * kept by the caller; it owns nothing. */
typedef struct pkv_rotary {
  int32_t d, rot_dim, layout;
  float amplitude;
  uint64_t turns[128];               /* 2^64 * f_i / (2 pi) */
  uint32_t check;                    /* set by pkv_rotary_init, pkv_rotary_axes_init */
} pkv_rotary;
int pkv_rotary_init(const pkv_rotary_spec *spec, int32_t d, pkv_rotary *out);

/*
 * Positions with several axes (time, height and width of an image's or a video's patches):
 * pair i turns by p_a * f_i, where a = axis[i] and p_a is the token's position on that axis.
 * Axis a has sections[a] pairs (sum: rot_dim/2), in the order
 *   PKV_AXES_BLOCKED  all of the first axis, then all of the second, ...
 *   PKV_AXES_CYCLIC   dealt to the axes in turn, as long as they have pairs left
 * and f_i is
 *   PKV_AXES_SHARED   that of pair i of the whole head, as without axes
 *   PKV_AXES_OWN      for the k-th pair of an axis, that of pair k of a head that rotates
 *                     2 * sections[a] elements
 * with the spec's layout, scaling and amplitude.  pkv_rotary_axes_init (host only) fills
 * both structs; they belong together: pkv_rotary_axes_append refuses a pair of other origin,
 * pkv_rotary_append a table with axes.
 */
#define PKV_ROTARY_MAX_AXES 8
#define PKV_AXES_BLOCKED 0
#define PKV_AXES_CYCLIC 1
#define PKV_AXES_SHARED 0
#define PKV_AXES_OWN 1
typedef struct pkv_rotary_axes {
  int32_t n_axes, pairs;
  uint8_t axis[128];                 /* of every pair */
  uint32_t check;                    /* set by pkv_rotary_axes_init */
} pkv_rotary_axes;
int pkv_rotary_axes_init(const pkv_rotary_spec *spec, int32_t d, const int32_t *sections,
                         int32_t n_axes, int32_t order, int32_t ladder, pkv_rotary *out,
                         pkv_rotary_axes *axes);

typedef struct pkv_rotary_args {
  const pkv_rotary *rotary;          /* host */
  const void *q, *k, *v;             /* T tokens of [Hq,d], [Hkv,d], [Hkv,d]; a token's heads
                                        are dense, tokens lie q_stride, k_stride, v_stride
                                        elements apart (slices of one projection's output) */
  int64_t q_stride, k_stride, v_stride;
  void *q_out, *k_out;               /* rotated q and k (k_out nullable when appending) */
  int64_t q_out_stride, k_out_stride;
  const int32_t *positions;          /* [T] */
  const int64_t *slot_mapping;       /* [T], or NULL: nothing is appended */
  void *k_cache, *v_cache;           /* [num_blocks,Hkv,16,d]; used with slot_mapping */
  int32_t num_blocks, T, Hq, Hkv, d, dtype;
  int32_t *dev_err_flag;             /* nullable */
} pkv_rotary_args;
/*
 * Rotates the queries and keys of T tokens (a decode step's rows or a prompt's
 * tokens) and, with slot_mapping, writes the rotated keys and the values into
 * the cache as pkv_append does (negative slot: nothing; a slot beyond the pool
 * sets PKV_DEVERR_BAD_SLOT).  The tokens of a call name different slots: where two
 * name one, its rows are left holding pieces of either's.
 * Hq or Hkv may be 0.  In place (q_out == q with the same stride, k_out == k) is
 * allowed; no other overlap is.  d even, 2..256; appending needs
 * d * sizeof(dtype) and the caches' addresses to be multiples of 16 bytes.
 */
int pkv_rotary_append(const pkv_rotary_args *args, void *stream);
/* The same with axes: args->positions holds [n_axes][T] positions, an axis' tokens dense,
 * the axes axis_stride (>= T) entries apart. */
int pkv_rotary_axes_append(const pkv_rotary_args *args, const pkv_rotary_axes *axes,
                           int64_t axis_stride, void *stream);

/* ======================================================================== */
/* decode attention over shared prefixes, with per-token weights             */
/* ======================================================================== */
/*
 * Rows that begin with the same tokens (a system prompt, a document) keep those
 * tokens in blocks of their own, once: row b attends over the tokens of prefix
 * row_prefix[b] followed by its own seq_lens[b] tokens, which are all that its
 * block table names.  Each prefix's keys and values are read once for all of its
 * rows, as matrix products over the rows' queries; the rows' own tokens go
 * through the split-KV kernel, and the two are joined by log-sum-exp:
 *   out[b,h] = sum_t softmax_t(q_rot[b,h] . k_t * scale + bias_t) v_t
 * over t in prefix ++ own (the bias, if any, covers own tokens only; -inf, or a
 * value below -2.35e38 such as float32's lowest, excludes a token, whatever its key
 * and value hold).  A row with no token at all, or none that is not excluded, outputs
 * zeros and lse = -inf; a query, key or value of NaN or infinity in what counts gives
 * NaN where the formula does.
 *
 * Scores, sums and accumulators are float32.  In bf16 the softmax weights are rounded to
 * bf16, once, ahead of the product with V (the tensor cores' operand type; the sums take
 * them before it), except in the one-kernel form for short contexts (pkv_shared_short),
 * which keeps them in float32.
 *
 * Positions are the caller's: a row's own token i sits at position
 * prefix length + i (pkv_seq_set_offset lets the allocator count that way).
 *
 * pkv_shared_plan (host only) groups the rows by prefix and splits the work
 * over num_ctas CTAs; it depends on which row has which prefix and on the
 * prefixes' lengths, so a plan stays valid until one of those changes.  Row b
 * has prefix row_prefix[b] in [0, n_prefixes), or none if that is negative;
 * prefix p has prefix_lens[p] >= 0 tokens.  plan receives at most plan_cap
 * int32, *plan_ints of them used; pkv_shared_plan_cap gives a sufficient
 * capacity.  The plan's own description of its size is what
 * pkv_shared_workspace_bytes needs: *slots, the partial results it keeps.
 * num_ctas <= 0 stands for the number of SMs of the current device.
 */
int pkv_shared_plan_cap(int32_t B, int32_t n_prefixes, int32_t Hq, int32_t Hkv,
                        int32_t num_ctas, int32_t *plan_cap, int32_t *max_slots);
int pkv_shared_plan(const int32_t *row_prefix, int32_t B, const int32_t *prefix_lens,
                    int32_t n_prefixes, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                    int32_t num_ctas, int32_t *plan, int32_t plan_cap, int32_t *plan_ints,
                    int32_t *slots);
/* The partition pkv_decode_attn_shared takes for num_parts <= 0 where the contexts are
 * not short (pkv_shared_short; in float32 behind prefixes at most one part to an SM): that of
 * pkv_attn_default_parts, but at least 8 positions (pages and unit boundaries, see
 * pkv_attn_default_parts' partition) to a part if every table were full. */
int pkv_shared_default_parts(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                             int32_t bt_stride, int32_t *num_parts);
/* Whether pkv_decode_attn_shared with num_parts <= 0 and no flags takes its one-kernel
 * form for short contexts: few (row, KV head) pairs whose tables have few entries
 * (pt_stride 0: no prefixes). */
int pkv_shared_short(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                     int32_t bt_stride, int32_t pt_stride, int32_t *short_form);
/* Workspace of pkv_decode_attn_shared: the bytes of pkv_attn_workspace_bytes plus
 * the row sums and, with prefixes, the partials of `slots` (0 without; max_slots above
 * serves every plan of those sizes) and the prefix CTAs' account of them.  Same rules: 256-byte aligned, zero-filled once
 * for a given B and num_parts (the counters' places follow from them, so again before
 * calls with others), calls that share it, or scores, must not overlap. */
int pkv_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t num_parts, int32_t slots, size_t *bytes);

typedef struct pkv_shared_args {
  const void *q_rot;                 /* [B,Hq,d] */
  const void *k_cache, *v_cache;     /* [num_blocks,Hkv,16,d] */
  const int32_t *block_tables;       /* [B*bt_stride] own tokens */
  const int32_t *seq_lens;           /* [B] own tokens */
  const float *attn_bias;            /* nullable [B*bias_stride], own tokens */
  const int32_t *plan;               /* nullable: pkv_plan_parts of the own tokens */
  const int32_t *prefix_tables;      /* [n_prefixes*pt_stride], or NULL: no prefixes */
  const int32_t *prefix_plan;        /* device copy of pkv_shared_plan's output (int32[plan_ints],
                                        16-byte aligned), required with prefix_tables */
  float *mass;                       /* nullable [num_blocks,Hkv,16]: accumulated weights */
  float *scores;                     /* with mass: scratch [num_blocks,Hkv,16,Hq/Hkv], 16-byte
                                        aligned */
  const int32_t *mass_lens;          /* with mass: nullable [B] */
  void *workspace;
  size_t workspace_bytes;
  void *out;                         /* [B,Hq,d] */
  float *lse_out;                    /* nullable [B,Hq]: natural log-sum-exp */
  int32_t *dev_err_flag;             /* nullable */
  int32_t num_blocks, bt_stride, bias_stride, n_prefixes, pt_stride, plan_ints, slots;
  int32_t B, Hq, Hkv, d, dtype, flags, num_parts, num_ctas;
  float scale, mass_decay;
} pkv_shared_args;
/*
 * With mass, every own token's weight is added to its accumulator: for token t
 * of row b in block k, row r, KV head g,
 *   mass[k,g,r] = (t < mass_lens[b] ? mass_decay * mass[k,g,r] : 0)
 *                 + sum over the group's heads of softmax weight of t
 * (mass_lens NULL stands for seq_lens[b] - 1: the step's new token starts from
 * zero, whatever its block held before).  The weights are relative to prefix and
 * own tokens together.  A block may then belong to one row only.
 *
 * Sizes as pkv_decode_attn_split; flags: PKV_ATTN_CHECK_PLAN,
 * PKV_ATTN_SHORT_WAITS.  out must not overlap q_rot.  A block id outside the pool sets
 * PKV_DEVERR_BAD_BLOCK and its tokens are left out.  plan_ints, slots and
 * num_ctas are pkv_shared_plan's.  A prefix_plan made for another call (its B,
 * num_ctas, Hkv or Hq/Hkv) sets PKV_DEVERR_BAD_PLAN and the rows attend over
 * their own tokens alone; so does a row whose prefix lies outside prefix_tables,
 * and, where partials are kept (not in the one-kernel form), a plan with more of
 * them than slots or whose records leave some out.
 * Where a wait of the prefix kernel gives up (PKV_DEVERR_TIMEOUT), the rows
 * with a prefix are NaN.  Records of `plan` that do not fit set
 * PKV_DEVERR_BAD_PLAN and are skipped (their rows' outputs are then incomplete).
 */
int pkv_decode_attn_shared(const pkv_shared_args *args, void *stream);

/* ======================================================================== */
/* eviction by accumulated weight                                            */
/* ======================================================================== */
/*
 * Row b of L = seq_lens[b] tokens keeps K = keep_lens[b] of them, for each KV
 * head its own choice: its last r = min(recent, K) tokens, its first
 * s = min(sink, K - r), and of those between the K - r - s with the largest
 * mass (equal ones: the lowest index; NaN counts as the largest).  The kept
 * tokens' keys, values and mass move, in their order, to the front of the row's
 * blocks (in place: slots 0..K-1 of its block table); what lies behind is left
 * as it was.  Keys stay rotated at their own positions.  A row with L <= K is
 * left alone.  kept[b,g,j] receives the index of the j-th kept token (-1 from
 * min(L,K) on), for all kept_stride entries of every row.
 *
 * A row with a bad length (L < 0, L > 16*bt_stride, K < 0, or min(L,K) >
 * kept_stride) sets PKV_DEVERR_BAD_LEN, one with a block id outside the pool
 * PKV_DEVERR_BAD_BLOCK; such a row is left alone, its kept entries are -1.  A
 * block may appear once among the rows' tables.  The host then shortens the
 * sequences with pkv_seqs_evict.
 * d * sizeof(dtype) a multiple of 16, at most 1024; caches and mass 16-byte
 * aligned; B <= 65536.  Workspace: pkv_evict_workspace_bytes(...) bytes, 256-byte
 * aligned, any contents; calls that share it must not overlap.
 */
int pkv_evict_workspace_bytes(int32_t B, int32_t Hkv, int32_t d, int32_t dtype,
                              int32_t kept_stride, size_t *bytes);
typedef struct pkv_evict_args {
  void *k_cache, *v_cache;           /* [num_blocks,Hkv,16,d] */
  float *mass;                       /* [num_blocks,Hkv,16] */
  const int32_t *block_tables;       /* [B*bt_stride] */
  const int32_t *seq_lens;           /* [B] */
  const int32_t *keep_lens;          /* [B] */
  int32_t *kept;                     /* [B,Hkv,kept_stride] */
  void *workspace;
  size_t workspace_bytes;
  int32_t *dev_err_flag;             /* nullable */
  int32_t num_blocks, bt_stride, kept_stride, sink, recent;
  int32_t B, Hkv, d, dtype;
} pkv_evict_args;
int pkv_evict(const pkv_evict_args *args, void *stream);

/* ======================================================================== */
/* drafted tokens: attention of a tree, its accepted path, copies of blocks  */
/* ======================================================================== */
/*
 * Several new tokens a row in one step: a tree of drafted tokens to verify, or a chunk of
 * a prompt.  They are appended like any token (pkv_prepare_nodes, then pkv_rotary_append:
 * row b's blocks hold seq_lens[b] tokens, of which the last n_b = node_starts[b+1] -
 * node_starts[b] are its nodes), and each attends over what is ahead of the nodes and over
 * those nodes that its mask names:
 *   node i, query head h:  s_t = (q_rot[node_starts[b]+i,h] . k_t) * scale
 *   out[node_starts[b]+i,h] = sum_t softmax_t(s) v_t
 * over tokens t < seq_lens[b] - n_b and nodes j (token seq_lens[b] - n_b + j) with bit
 * j % 32 of mask[(node_starts[b]+i)*mask_words + j/32] set (bits from n_b on are not
 * looked at).  Without a mask node i sees the nodes up to itself.  Node i's own bit is
 * like any other.  A token that a node does not see may hold anything.  A node that sees
 * nothing outputs zeros and lse = -inf; NaN and infinities in what it sees give NaN where
 * the formula does.  Keys are in the caches as rotated; positions are the caller's
 * (a node's: the tokens ahead of the nodes plus its depth).
 *
 * Scores, sums and accumulators are float32; in bf16 the softmax weights are rounded to
 * bf16, once, ahead of the product with V (the tensor cores' operand type; the sums take
 * them before it).
 *
 * q_rot, out [T,Hq,d]; query rows outside node_starts[0..B] are left as they were, and so
 * are a row's that does not fit the call (PKV_DEVERR_BAD_LEN: starts that do not ascend
 * within [0, T], more nodes than tokens or mask bits, seq_lens[b] > 16*bt_stride); rows that
 * add up to 2^31 steps of 64 tokens and more set it too, and nothing is computed.  A block
 * id outside the pool sets PKV_DEVERR_BAD_BLOCK and its tokens are left out (a node to
 * which none is left is NaN).  Rows may share blocks (pkv_seq_fork, shared prefixes); a
 * query row belongs to one batch row.  Where a wait inside the kernel gives up
 * (PKV_DEVERR_TIMEOUT), the outputs that it was for are NaN.
 *
 * Types, heads and head sizes as pkv_decode_attn_split; out must not overlap q_rot.
 * flags: 0 or PKV_ATTN_SHORT_WAITS.  Workspace: pkv_tree_workspace_bytes(...) bytes for the
 * current device, 256-byte aligned, any contents (a call leaves nothing in it that a later
 * one reads); calls that share it must not overlap.
 */
int pkv_tree_workspace_bytes(int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, size_t *bytes);
typedef struct pkv_tree_args {
  const void *q_rot;                 /* [T,Hq,d] */
  const void *k_cache, *v_cache;     /* [num_blocks,Hkv,16,d] */
  const int32_t *block_tables;       /* [B*bt_stride] */
  const int32_t *seq_lens;           /* [B] */
  const int32_t *node_starts;        /* [B+1] */
  const int32_t *mask;               /* nullable [T*mask_words] bits */
  void *workspace;
  size_t workspace_bytes;
  void *out;                         /* [T,Hq,d] */
  float *lse_out;                    /* nullable [T,Hq]: natural log-sum-exp */
  int32_t *dev_err_flag;             /* nullable */
  int32_t num_blocks, bt_stride, mask_words;
  int32_t B, T, Hq, Hkv, d, dtype, flags;
  float scale;
} pkv_tree_args;
int pkv_decode_attn_tree(const pkv_tree_args *args, void *stream);

/*
 * The accepted path of each row's tree to the front of its nodes' slots, in place, in all
 * n_pools pools (keys and values of every layer) at once: with base = seq_lens[b] - n_b,
 * token base + j becomes what token base + path[b*path_stride + j] held, for
 * j < accept_lens[b].  A path ascends strictly (parents come ahead of their children) within
 * [0, n_b).  Tokens from base + accept_lens[b] on hold nothing of use afterwards:
 * pkv_seqs_truncate to base + accept_lens[b] frees them.  Keys stay rotated: a node's
 * position is its depth's, which is its place on the path.
 * A row that does not fit (lengths as in pkv_decode_attn_tree, accept_lens[b] outside
 * [0, min(n_b, path_stride)], a path that does not ascend) sets PKV_DEVERR_BAD_LEN, one with
 * a block id outside the pool among those that it needs PKV_DEVERR_BAD_BLOCK; it is left
 * alone.  The blocks of a row's nodes belong to that row only.
 */
#define PKV_MAX_POOLS 256
typedef struct pkv_accept_args {
  void *const *pools;                /* host array of n_pools device pointers, each
                                        [num_blocks,Hkv,16,d], 16-byte aligned */
  const int32_t *block_tables;       /* [B*bt_stride] */
  const int32_t *seq_lens;           /* [B] */
  const int32_t *node_starts;        /* [B+1] */
  const int32_t *path;               /* [B*path_stride] */
  const int32_t *accept_lens;        /* [B] */
  int32_t *dev_err_flag;             /* nullable */
  int32_t n_pools, num_blocks, bt_stride, path_stride, B, T, Hkv, d, dtype;
} pkv_accept_args;
int pkv_tree_accept(const pkv_accept_args *args, void *stream);

/*
 * Copies of whole blocks, in n_pools pools at once: block dst_blocks[i] of dst[p] becomes
 * block src_blocks[i] of src[p], for i < n and every pool p.  src[p] may be dst[p] (forks)
 * or another pool (a pool of another size, one in mapped host memory); a destination
 * overlaps no other pool.  A pair with a negative id copies nothing; an id beyond its pool
 * sets PKV_DEVERR_BAD_BLOCK and its pair is skipped.  A block may be the destination of
 * one pair only and, within one pool, not the source of another (else what it holds is
 * undefined).
 */
typedef struct pkv_copy_args {
  const void *const *src;            /* host arrays of n_pools device pointers, 16-byte aligned */
  void *const *dst;
  const int32_t *src_blocks, *dst_blocks;   /* [n] */
  int32_t *dev_err_flag;             /* nullable */
  int64_t block_bytes;               /* of one block of one pool: a multiple of 16 */
  int32_t n_pools, n, src_num_blocks, dst_num_blocks;
} pkv_copy_args;
int pkv_copy_blocks(const pkv_copy_args *args, void *stream);

/* ======================================================================== */
/* the whole device step: a1 -> a2 -> a3 -> a4 on one stream                */
/* ======================================================================== */
typedef struct pkv_step_args {
  const void *q, *k, *v;             /* new tokens: [B,Hq,d], [B,Hkv,d], [B,Hkv,d] */
  void *q_rot, *k_rot;               /* RoPE outputs (device scratch owned by the caller) */
  void *k_cache, *v_cache;           /* [num_blocks,Hkv,16,d] */
  int32_t num_blocks;
  const int32_t *positions;          /* [B] */
  const int64_t *slot_mapping;       /* [B] */
  const int32_t *seq_lens;           /* [B] lengths after the append */
  const int32_t *block_tables;       /* [B*bt_stride] */
  int32_t bt_stride;
  const float *attn_bias;            /* nullable, [B*bias_stride] */
  int32_t bias_stride;
  int32_t B, Hq, Hkv, d;
  float scale, rope_base;
  int32_t dtype, flags, num_parts;
  void *workspace;                   /* pkv_attn_workspace_bytes(...) bytes */
  size_t workspace_bytes;
  void *out;                         /* [B,Hq,d] */
  int32_t *dev_err_flag;             /* nullable */
  const int32_t *plan;               /* nullable: pkv_plan_parts of this step's metadata
                                        for num_parts parts (num_parts must then be > 0) */
} pkv_step_args;

/* All pointers in *args are device pointers or host memory the GPU can reach
 * (pinned / mapped: q, k, v, positions, slot_mapping, seq_lens and block_tables
 * may live there so that a step needs no host-to-device copy -- the kernels read
 * them in place -- and out so that it needs no copy back; give the mapped
 * address, pkv_mapped_pointer); asynchronous on stream.
 * Runs pkv_rope_append, then pkv_decode_attn_split launched as a programmatic
 * dependent (its prologue overlaps the RoPE kernel), and pkv_lse_merge when
 * flags has PKV_ATTN_SEPARATE_MERGE.  With PKV_STEP_FUSED the whole step is
 * one kernel instead: the attention kernel also rotates q and k and appends
 * the rotated key and the value (the part that owns a row's last page writes
 * that row's slot before it loads the page; rows with seq_len 0 are not
 * appended).  Both forms give bit-identical results.  q_rot/k_rot receive the
 * rotated q and k.  Each row's slot must be its position seq_len-1 in its own
 * blocks, as pkv_prepare_step produces. */
int pkv_decode_step(const pkv_step_args *args, void *stream);

/*
 * A decode step through n_layers layers, each with its own caches
 * ("neurogrid releases" v0.7.0: per-layer caches; the block tables, slots,
 * positions and lengths are the same for every layer, so layers[l] differ in
 * q, k, v, q_rot, k_rot, k_cache, v_cache, out and workspace).  Layer l runs
 * after layer l-1 on `stream`: its RoPE/append kernel is launched as a
 * programmatic dependent of layer l-1's attention kernel (its angles are
 * formed early; its q/k/v reads and cache writes wait for that kernel), and
 * its attention kernel as a dependent of its RoPE/append kernel, so each
 * layer's start overlaps the previous layer's tail.  Consecutive layers must
 * not share a workspace (two alternating workspaces suffice).
 * PKV_STEP_FUSED is rejected.  Stops at the first failing layer.  The layers'
 * attention kernels are not launched cooperatively unless a layer's flags have
 * PKV_LAYERS_MERGE_HELPERS, so by default each unit's merge is done by its last
 * part alone (the next layer's kernels may then start on SMs the previous layer
 * has freed); with it, each layer merges like pkv_decode_step (bit-identical to
 * one single-layer step per layer).
 */
int pkv_decode_step_layers(const pkv_step_args *layers, int32_t n_layers, void *stream);

/*
 * The dense right-padded batch that paging replaces, kept as a comparator
 * (helexa issue 121: slice 1 assemble_batch, slice 3a extract_row).  All KV
 * buffers use the block layout [blocks, Hkv, 16, d] (dtype): a snapshot is one
 * sequence's tokens [0, len) in ceil(len/16) blocks; a dense batch of B rows
 * and cap tokens per row (cap a multiple of 16) is B*cap/16 blocks, row b owning
 * blocks [b*cap/16, (b+1)*cap/16), so the attention call reads it as a pool
 * with block table row b = b*cap/16 + j and an additive -inf bias on the gap.
 * k_snaps, v_snaps: host arrays of device pointers.  Buffers must be large
 * enough for the tokens named; nothing else is checked on the device.
 * Hkv * d * sizeof(dtype) must be at most 16 KB.
 *
 * pkv_dense_assemble: dense row b = snapshot b's tokens [0, lens[b]) followed by
 * zeros up to padded_len (lens[b] <= padded_len <= cap); tokens from
 * padded_len on are left for the decode columns.
 * pkv_dense_extract: for each i, snapshot i = dense row rows[i]'s prefix
 * [0, prefix_lens[i]) followed by its decode columns [padded_len,
 * padded_len + steps) (the gap is dropped).
 */
int pkv_dense_assemble(const void *const *k_snaps, const void *const *v_snaps,
                       const int32_t *lens, int32_t B, int32_t padded_len, void *k_dense,
                       void *v_dense, int32_t cap, int32_t Hkv, int32_t d, int32_t dtype,
                       void *stream);
int pkv_dense_extract(const void *k_dense, const void *v_dense, int32_t cap,
                      const int32_t *rows, const int32_t *prefix_lens, int32_t n_rows,
                      int32_t padded_len, int32_t steps, void *const *k_snaps,
                      void *const *v_snaps, int32_t Hkv, int32_t d, int32_t dtype,
                      void *stream);

/* The address under which kernels read the page-locked host buffer at
 * host_ptr (allocated pinned, or registered with the mapped flag), so that the
 * per-step metadata of pkv_decode_step can stay in host memory and be read by
 * the kernels over the CPU-GPU link instead of being copied first.  The buffer
 * must not change until the kernels that read it have finished.  Returns
 * PKV_ERR_INVALID_ARG for a NULL pointer and PKV_ERR_CUDA when the memory is
 * not mapped for the current device. */
int pkv_mapped_pointer(const void *host_ptr, void **device_ptr);

/* Host-side buffers for pkv_decode_step_host (pinned memory recommended). */
#define PKV_HOST_IN_PLACE 1   /* pkv_step_host_io.flags: the kernels read the host
                                 inputs and write the host output in place
                                 instead of going through device copies */

typedef struct pkv_step_host_io {
  const void *q, *k, *v;             /* [B,Hq,d], [B,Hkv,d], [B,Hkv,d] */
  const int32_t *positions;
  const int64_t *slot_mapping;
  const int32_t *seq_lens;
  const int32_t *block_tables;       /* [B*bt_stride] */
  void *out;                         /* [B,Hq,d] */
  int32_t flags;                     /* 0 or PKV_HOST_IN_PLACE */
  const int32_t *plan;               /* nullable: the step's plan (pkv_plan_parts), read in
                                        place or copied to dev->plan like the metadata */
} pkv_step_host_io;

/*
 * End-to-end step from host memory: copies the host inputs into the device
 * buffers named by *dev (q, k, v, positions, slot_mapping, seq_lens,
 * block_tables), runs pkv_decode_step, copies dev->out back to host->out and
 * waits for the stream.  Returns after the result is in host memory.  With
 * PKV_HOST_IN_PLACE the inputs and host->out must be page-locked host memory;
 * the step's kernels read the inputs and write the result over the CPU-GPU
 * link at their mapped addresses (no staging or result copies; dev's input
 * pointers and dev->out are not used).  The mapped address of each host buffer is looked up once per
 * device and remembered (a buffer freed and re-registered at the same address
 * must keep its mapping).
 */
int pkv_decode_step_host(const pkv_step_args *dev, const pkv_step_host_io *host,
                         void *stream);

/*
 * The work of pkv_decode_step_host(dev, host) -- staging copies or in-place
 * reads per host->flags, the step's kernels, the copy of the output back --
 * captured once as a CUDA graph for these exact buffers (their addresses are
 * fixed in it: each launch reads whatever the host last wrote there, typically
 * pkv_prepare_step's outputs and the new q/k/v).  A serving loop then pays one
 * graph launch per step instead of every launch and copy.  *out owns the graph
 * (free with pkv_step_graph_destroy).  Nothing runs at creation.
 */
typedef struct pkv_step_graph pkv_step_graph;
int pkv_step_graph_create(const pkv_step_args *dev, const pkv_step_host_io *host,
                          pkv_step_graph **out);
/* Launches the captured step on stream and waits for it (host->out is then set). */
int pkv_step_graph_launch(pkv_step_graph *g, void *stream);
/*
 * The same launch without the wait, and the wait on its own.  Each graph
 * records its own completion event after every enqueue, so a loop over two
 * graphs (two sets of host buffers) keeps the GPU busy: prepare step i into
 * set i%2 (a0, the plan, the new q/k/v), enqueue its graph, then wait for the
 * graph of step i-1 and read its output while the GPU runs step i.  Host
 * buffers a queued or running launch reads or writes must not be touched until
 * pkv_step_graph_wait has returned for that graph.  The graphs of one loop
 * share the device buffers of dev (scratch, caches), so they go on one stream.
 * Errors: PKV_ERR_INVALID_ARG for a NULL graph; PKV_ERR_CUDA if the launch or
 * the event record fails (the message names the call).
 */
int pkv_step_graph_enqueue(pkv_step_graph *g, void *stream);
/* Waits (blocking the calling thread) for the last pkv_step_graph_enqueue of
 * g; host->out then holds that step's output.  Returns at once if g was never
 * enqueued.  Errors: PKV_ERR_INVALID_ARG for a NULL graph; PKV_ERR_CUDA if the
 * step failed on the device (a sticky CUDA error: the context is then lost). */
int pkv_step_graph_wait(pkv_step_graph *g);
/* Frees the graph and its event (NULL is ignored); no launch of g may be in
 * flight. */
void pkv_step_graph_destroy(pkv_step_graph *g);

/* ======================================================================== */
/* native serving loop: continuous batching, one host call per step          */
/* ======================================================================== */
/*
 * The continuous-batching loop of helexa issue 121, slice 3b (admit joiners,
 * prefill them, rebatch, decode every live sequence in lockstep) over the
 * paged cache of "neurogrid releases" v0.7.0 (joining or leaving edits block
 * tables only; no KV moves), the step replayed as one CUDA graph that reads
 * the host-written metadata in place (v0.8.0).  A joiner takes over the row of
 * a sequence that left, so the batch keeps its B rows and two captured graphs
 * (one per pinned metadata buffer, used alternately) serve every step.
 *
 * The caller owns every buffer and keeps each alive and in place for the
 * server's lifetime (the server allocates no device memory):
 *  - step: pkv_decode_step's device buffers and sizes for B rows.  step.q,
 *    step.k, step.v are the graph's input buffers.  Its metadata and plan
 *    pointers are ignored (the server points them into meta_host); num_parts
 *    must be > 0; attn_bias must be NULL.
 *  - alloc: the block allocator; rows[b] (B entries) are live sequences of it,
 *    which the server then manages (joins and leaves go through the server).
 *  - meta_host[2]: page-locked host buffers of pkv_server_meta_bytes(B,
 *    bt_stride, num_parts) bytes, 16-byte aligned (positions, slots, lengths,
 *    block tables and the partition plan of a step).
 *  - prefix_host[2]: page-locked host buffers of
 *    pkv_server_prefix_bytes(max_prefix_tokens) bytes (joiners' prefix
 *    positions and slots), or NULL when max_prefix_tokens is 0.
 * Creation captures the two graphs; nothing runs.
 */
typedef struct pkv_server pkv_server;
typedef struct pkv_server_desc {
  pkv_step_args step;
  pkv_alloc *alloc;
  const int32_t *rows;               /* [step.B] live sequence ids, one per row */
  void *meta_host[2];
  void *prefix_host[2];
  int32_t max_prefix_tokens;         /* most prefix tokens joining in one step */
} pkv_server_desc;
size_t pkv_server_meta_bytes(int32_t B, int32_t bt_stride, int32_t num_parts);
size_t pkv_server_prefix_bytes(int32_t max_prefix_tokens);
int pkv_server_create(const pkv_server_desc *desc, pkv_server **out);
/*
 * One step, enqueued on stream.  The sequences of rows leave_rows[0..n-1]
 * retire and n joiners take those rows, joiner i with a prefix of
 * prefix_lens[i] tokens whose raw keys and values are prefix_k, prefix_v
 * (device, [sum(prefix_lens), Hkv, d], joiner after joiner): they are rotated
 * at their positions and written into the joiners' blocks (pkv_prefill_kv).
 * Then every row decodes one token: q, k, v (device, [B,Hq,d], [B,Hkv,d],
 * [B,Hkv,d]; NULL or the step's own input buffers: nothing to copy) are copied
 * into the step's input buffers, a0 (pkv_prepare_step_cached) and the plan
 * (pkv_plan_parts) are written into a metadata buffer, and the captured step
 * is launched: the result is in step.out when the stream gets there.  The
 * call waits only for the step two calls back, which used the same host
 * buffers.  Argument errors change nothing; a failure after the leaves (the
 * pool cannot take the joiners: PKV_ERR_OUT_OF_BLOCKS) leaves the server
 * unusable, and every later step returns PKV_ERR_INVALID_ARG.
 */
int pkv_server_step(pkv_server *s, const int32_t *leave_rows, const int32_t *prefix_lens,
                    int32_t n, const void *prefix_k, const void *prefix_v, const void *q,
                    const void *k, const void *v, void *stream);
/* The sequence id of every row ([B]). */
int pkv_server_rows(const pkv_server *s, int32_t *rows);
/* Frees the server (not the caller's buffers or allocator); call after its
 * last step has finished on the GPU. */
void pkv_server_destroy(pkv_server *s);

#ifdef __cplusplus
}
#endif
#endif /* PKV_H */
