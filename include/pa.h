/*
 * pa.h — C ABI of libpa: paged KV-cache attention kernels for GB300 (sm_103a).
 *
 * The operations are the ones the paged-attention pages describe:
 *
 *   [KVS] "19.2 KV Cache 系统化管理" (paper.xwysyy.cn, llm-fullstack-book):
 *         §19.2.2 block pool / block table, Fig 19-5 block-wise attention,
 *         Fig 19-8 copy-on-write; §19.2.3 the simplified implementation
 *         (pool layout, slot writes, block-table append, paged attention with
 *         an online softmax checked against dense softmax attention);
 *         §19.2.4 KV quantisation (FP8); §19.2.6 swapping blocks to CPU
 *         memory on preemption.
 *   [OS]  "LLM 推理引擎的内存管理与调度：PagedAttention、Prefix Cache 与
 *         Continuous Batching" (zhouzhq2021.github.io): §三 the kernel looks a
 *         logical block up in the block table and forms the physical address
 *         and in-block offset; §四 shared blocks and copy-on-write; §8.1
 *         chunked prefill.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Pool layout (from [KVS] §19.2.3): k_cache and v_cache are each
 *    [num_blocks, block_size, num_kv_heads, head_dim], row-major, contiguous,
 *    one layer.  Call once per layer for a multi-layer cache.
 *  - Element type: PA_F32 or PA_BF16; K, V, Q and the output share it,
 *    except for the e4m3 pool calls (pa_reshape_and_cache_fp8,
 *    pa_decode_fp8 and the block-scaled cache's), whose pools hold
 *    PA_FP8_E4M3 codes with fp32 scales.
 *    Accumulation is fp32 whatever the storage type (the tensor-core forms
 *    round their product operands as each call's description states); bf16
 *    results are rounded to nearest even.
 *  - Supported sizes (the latent cache and the rotary calls state their own):
 *    head_dim in {32, 64, 128}; block_size in {4, 8, 16, 32}; num_heads a
 *    multiple of num_kv_heads.  Query head h reads KV head
 *    h / (num_heads / num_kv_heads) (grouped-query attention).
 *  - Every pointer argument is a DEVICE pointer unless stated otherwise; the
 *    caller owns all memory and the library allocates nothing per call.
 *    K/V pools, queries and outputs must be 16-byte aligned.
 *  - `stream` is a cudaStream_t (NULL: the legacy default stream).  Every
 *    call only enqueues work on it and returns without synchronising.
 *  - CUDA graphs: every argument the kernels read is a device pointer or a
 *    size, so a captured call replays with whatever the pointed-to buffers
 *    hold at replay time.  The first call with a new combination of sizes
 *    and pool (kernel variant, tensor map) does host-side set-up (function
 *    attributes, occupancy query, tensor-map encoding, cached afterwards):
 *    make one call outside the capture first.
 *  - Return value: 0 on success, or a negative PA_ERR_* code when the host
 *    side rejects the arguments — in that case nothing was launched.
 *  - Conditions only the device can see (a block id outside the pool, a slot
 *    outside the pool, a context longer than its block-table row, a
 *    pipeline wait that ran out) never trap: the affected item is skipped or
 *    zero-filled and a bit is OR-ed into a sticky device word that
 *    pa_last_error() returns and clears.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* PA_FP8_E4M3 is a storage type for K/V pools only: 8-bit e4m3 codes (4
 * exponent bits with bias 7, 3 mantissa bits, largest finite value 448)
 * with one fp32 scale per token for its K vector and one for its V vector
 * (pa_reshape_and_cache_fp8, pa_decode_fp8), or one per (block, KV head)
 * (pa_append_fp8_blocks and the calls after it). */
typedef enum { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2 } pa_dtype;

/* host-detected errors (negative return values) */
#define PA_OK             0
#define PA_ERR_NULL      (-1) /* a required pointer is NULL */
#define PA_ERR_SHAPE     (-2) /* unsupported or inconsistent sizes */
#define PA_ERR_DTYPE     (-3) /* unknown pa_dtype */
#define PA_ERR_ALIGN     (-4) /* a K/V/Q/out pointer is not 16-byte aligned */
#define PA_ERR_WORKSPACE (-5) /* workspace missing or smaller than needed */
#define PA_ERR_CUDA      (-6) /* a CUDA runtime call failed (launch, attributes) */

/* device-detected conditions (bits of pa_last_error()'s positive result) */
#define PA_DEV_BAD_BLOCK  1u  /* block-table entry or pair id outside [0, num_blocks) */
#define PA_DEV_BAD_SLOT   2u  /* slot_mapping entry >= num_blocks * block_size */
#define PA_DEV_BAD_LEN    4u  /* context length < 0 or > max_blocks_per_seq * block_size */
#define PA_DEV_TIMEOUT    8u  /* a shared-memory pipeline wait exceeded its time limit */
#define PA_DEV_BAD_GROUP 16u  /* pa_decode_shared: a group descriptor that does not cover the batch,
                                or a member whose row does not hold its group's shared blocks */

/*
 * KV append ("reshape_and_cache").  [KVS] §19.2.3: a new token's key and
 * value are written into a slot of a physical block; the slot comes from the
 * block table (logical block = tokens so far / block_size, offset = tokens so
 * far % block_size).  Fig 19-6: decode appends into the partly filled block.
 *
 *   key, value     [num_tokens, num_kv_heads, head_dim]   (read)
 *   slot_mapping   [num_tokens] int64: physical_block * block_size + offset.
 *                  A negative slot is padding and is skipped.  Slots must be
 *                  distinct within one call (duplicates: unspecified winner).
 *   k_cache, v_cache  pool (written only at the addressed slots)
 *
 * Exact byte copy.  A slot >= num_blocks * block_size is skipped and sets
 * PA_DEV_BAD_SLOT.  num_tokens == 0 launches nothing.
 */
int pa_reshape_and_cache(const void* key, const void* value,
                         const int64_t* slot_mapping, int num_tokens,
                         void* k_cache, void* v_cache,
                         int num_blocks, int block_size, int num_kv_heads, int head_dim,
                         pa_dtype dtype, void* stream);

/*
 * Paged decode attention.  [KVS] §19.2.3 / Fig 19-5 and [OS] §三: for each
 * sequence b and query head h (KV head g = h / (num_heads/num_kv_heads)),
 *
 *   out[b,h,:] = sum_{t < L_b} softmax_t(scale * <q[b,h,:], K_b[t,g,:]>) V_b[t,g,:]
 *
 * where token t of sequence b sits in physical block
 * block_tables[b*max_blocks_per_seq + t/block_size] at slot t % block_size,
 * and L_b = context_lens[b] counts the newest token (append it first).
 * Only the valid slots of the last block are read; L_b == 0 gives zeros.
 *
 *   out            [num_seqs, num_heads, head_dim]        (written)
 *   query          [num_seqs, num_heads, head_dim]
 *   block_tables   [num_seqs, max_blocks_per_seq] int32
 *   context_lens   [num_seqs] int32
 *   scale          the pages use 1/sqrt(head_dim)
 *   partition_size split-K partition in tokens: 0 = automatic (256 tokens
 *                  when num_heads == num_kv_heads; 2048 for grouped-query
 *                  attention, unless num_seqs * ceil(num_kv_heads / 4) <
 *                  912, the unsplit work items being fewer than three per
 *                  CTA of the grid: then the largest power of two from
 *                  256 to 2048 not above max_blocks_per_seq * block_size *
 *                  num_seqs * ceil(num_kv_heads / 4) / 2432, or 256), < 0 = never
 *                  split, > 0 = a multiple of block_size.  A sequence longer
 *                  than one partition is processed as independent partitions
 *                  whose (max, sum, unnormalised output) states are merged by
 *                  log-sum-exp in a second kernel (outside stream capture it
 *                  is launched as a programmatic dependent of the first and
 *                  waits for it on the device; inside a capture, a plain
 *                  launch).
 *   workspace      device scratch of at least pa_decode_workspace_bytes()
 *                  with the same sizes (may be NULL when that is 0).  Its
 *                  contents on entry do not matter; calls that share one
 *                  workspace must be ordered (same stream).  Its last 256
 *                  bytes hold a work-item counter: a one-thread kernel clears
 *                  it, then the decode kernel's CTAs take their work items
 *                  from it as they free up (on eager calls the decode kernel
 *                  is that kernel's programmatic dependent and waits for it
 *                  on the device).  Without a workspace (no split needed) the
 *                  items are divided among the CTAs in advance.
 *
 * Output is fp32-accumulated; bf16 output is rounded to nearest even.  With
 * bf16, head_dim 64 or 128, block_size >= 8 and a power-of-two group G >= 2,
 * the G query heads of a KV head are computed together on tensor cores
 * (m16n8k16 bf16 products, fp32 accumulation; P is rounded to bf16 for the
 * P*V product): for G <= 8 the block's tokens are the M rows and the heads
 * the N columns; for G >= 16, subgroups of 16 heads are the M rows.
 * Everything else runs on CUDA cores in fp32.
 */
int pa_decode(void* out, const void* query,
              const void* k_cache, const void* v_cache,
              const int32_t* block_tables, int max_blocks_per_seq,
              const int32_t* context_lens, int num_seqs,
              int num_heads, int num_kv_heads, int head_dim,
              int block_size, int num_blocks, float scale, int partition_size,
              void* workspace, size_t workspace_bytes,
              pa_dtype dtype, void* stream);

/*
 * Paged decode attention for sequences that share prompt blocks.  [KVS]
 * §19.2.2 (Fig 19-8) and §19.2.5, [OS] §四: samples drawn from one prompt
 * (parallel sampling, beam search, a common system prompt) point their
 * block tables at the same physical blocks for the prompt, shared by
 * reference count.  The result is that of pa_decode on the same arguments;
 * the shared blocks' keys and values are read from memory once per group
 * for all of its members' query heads (one dense tensor-core product per
 * (shared block, KV head)) instead of once per member.
 *
 *   group_start    [num_groups + 1] int32, device: group g is sequences
 *                  group_start[g] .. group_start[g+1]-1 (non-decreasing,
 *                  from 0 to num_seqs; a sequence alone is a group of one)
 *   shared_blocks  [num_groups] int32, device: the number of leading
 *                  block-table entries every member of group g holds in
 *                  common.  The shared part used is
 *                    S_g = min(shared_blocks[g], floor(L_b / block_size)
 *                              over the group's members b)
 *                  whole blocks, read through the FIRST member's table row;
 *                  each member's tokens from S_g * block_size on are read
 *                  through its own row.  The two attention states are
 *                  merged by log-sum-exp (exact up to rounding: the online
 *                  softmax is associative).
 *   partition_size 0: automatic: partitions of the shared blocks of 1024,
 *                  512, 256 or 128 tokens, the largest that gives at least
 *                  152 shared items if every group shared its whole longest
 *                  context (host arithmetic on num_seqs, num_groups,
 *                  num_kv_heads and max_blocks_per_seq); the private tails
 *                  as pa_decode's automatic choice;
 *                  > 0: a multiple of block_size used for both; < 0: no
 *                  split of either.
 *   workspace      at least pa_decode_shared_workspace_bytes() with the same
 *                  sizes, 16-byte aligned (PA_ERR_ALIGN otherwise); contents
 *                  on entry do not matter
 *   other arguments as for pa_decode
 *
 * Device-detected conditions (PA_DEV_BAD_GROUP): a descriptor that is not
 * non-decreasing from 0 to num_seqs is ignored (the call computes plain
 * decode); a member whose row differs from the first member's within the
 * shared blocks is flagged and its shared part follows the first member's
 * row.  PA_BF16 with head_dim 64 or 128, block_size >= 8, G =
 * num_heads / num_kv_heads <= 8, num_seqs <= 1024 and 1 <= num_groups <=
 * 1024 run the shared path (tensor cores, m16n8k16 bf16 products with fp32
 * accumulation, P rounded to bf16); other arguments run pa_decode unchanged
 * (same result, no sharing exploited).  On the stream: a one-thread kernel
 * that clears the work-item counter the call keeps in the workspace, the
 * decode kernel (its CTAs take work items from that counter as they free
 * up, larger ones first; private tails largest first) and a merge kernel;
 * on eager calls the last two are launched as programmatic dependents of
 * the kernel before them and wait for it on the device.
 */
int pa_decode_shared(void* out, const void* query,
                     const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int num_seqs,
                     const int32_t* group_start, const int32_t* shared_blocks, int num_groups,
                     int num_heads, int num_kv_heads, int head_dim,
                     int block_size, int num_blocks, float scale, int partition_size,
                     void* workspace, size_t workspace_bytes,
                     pa_dtype dtype, void* stream);

/* Bytes of workspace pa_decode_shared needs for these sizes (never less than
 * pa_decode_workspace_bytes()).  Pure host arithmetic; no CUDA call. */
size_t pa_decode_shared_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                        int max_blocks_per_seq, int block_size, int partition_size,
                                        int num_groups);

/*
 * KV append into an e4m3 pool.  The write of pa_reshape_and_cache, with each
 * token's K vector and V vector ([num_kv_heads, head_dim], every head)
 * quantised on its own ([KVS] §19.2.4: per-token scaled quantisation, FP8
 * at one byte per element).  The formula is not in the extracted page; the
 * reading implemented is absmax scaling onto the e4m3 range:
 *
 *   amax  = max |x| over the token's vector
 *   scale = amax / 448                 (fp32, correctly rounded)
 *   code  = e4m3(x * (448 / amax))     (fp32 product, nearest-even rounding,
 *                                       saturating at +-448)
 *
 * and amax == 0 gives scale 0 and all-zero codes.  A dequantised element is
 * e4m3_value(code) * scale.  Non-finite inputs give unspecified codes.
 *
 *   key, value        [num_tokens, num_kv_heads, head_dim], src_dtype
 *                     PA_BF16 or PA_F32
 *   slot_mapping      as for pa_reshape_and_cache
 *   k_cache, v_cache  e4m3 pools [num_blocks, block_size, num_kv_heads,
 *                     head_dim], one byte per element
 *   k_scale, v_scale  [num_blocks, block_size] fp32 (16-byte aligned): the
 *                     scale of the token in each slot
 */
int pa_reshape_and_cache_fp8(const void* key, const void* value,
                             const int64_t* slot_mapping, int num_tokens,
                             void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                             int num_blocks, int block_size, int num_kv_heads, int head_dim,
                             pa_dtype src_dtype, void* stream);

/*
 * Paged decode attention over an e4m3 pool: the result of pa_decode over
 * the dequantised pool (K = e4m3_value(code) * k_scale[slot], likewise V).
 * The per-token scales are applied exactly in fp32: the K scale multiplies
 * the token's score, the V scale its softmax weight in the P*V sum (the
 * softmax normaliser uses the unscaled weights).  Halves the bytes read per
 * token against bf16 ([KVS] §19.2.4).
 *
 *   query, out        dtype must be PA_BF16
 *   k_cache, v_cache  e4m3 pools; k_scale, v_scale as written by
 *                     pa_reshape_and_cache_fp8 (16-byte aligned)
 *   partition_size    as for pa_decode, but the automatic choice is 512
 *                     tokens when num_heads == num_kv_heads (grouped-query
 *                     attention as for pa_decode); pa_decode_fp8_partition_size
 *                     returns the size used
 *   workspace         pa_decode_workspace_bytes() with the same sizes is
 *                     enough (the automatic partition here is never shorter
 *                     than pa_decode's, so no more partials are written)
 *   other arguments   as for pa_decode
 *
 * Power-of-two query groups (G >= 2; subgroups of 16 above 16) with
 * head_dim 128 and block_size >= 8 run on tensor cores: f16 m16n8k16 products of the exactly converted codes with
 * fp32 accumulation, Q scaled per work item by a power of two into f16
 * range, P carrying the V scale relative to a power-of-two reference (f16,
 * in [0, 1]).  Everything else runs on CUDA cores in fp32.
 */
int pa_decode_fp8(void* out, const void* query,
                  const void* k_cache, const void* v_cache,
                  const float* k_scale, const float* v_scale,
                  const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, int num_seqs,
                  int num_heads, int num_kv_heads, int head_dim,
                  int block_size, int num_blocks, float scale, int partition_size,
                  void* workspace, size_t workspace_bytes,
                  pa_dtype dtype, void* stream);

/*
 * The block-scaled e4m3 cache: an e4m3 pool with one fp32 scale per (block,
 * KV head) for K and one for V.
 *
 *   k_cache, v_cache  codes [num_blocks, block_size, num_kv_heads, head_dim]
 *   k_scale, v_scale  [num_blocks, PA_SCALE_ROW(num_kv_heads)] fp32, 16-byte
 *                     aligned: entry h of a block's row belongs to KV head h
 *                     (a row is padded to whole 16-byte chunks; the padding
 *                     is read, never used and never written)
 *
 * A dequantised element is e4m3_value(code) * scale.  The calls below write
 * powers of two; pa_decode_fp8_blocks, pa_decode_weights and
 * pa_prefill_fp8_blocks read any finite scale >= 0.  Blocks are copied and
 * swapped with pa_copy_blocks / pa_swap_blocks on the codes and again, with
 * the same pairs, on (k_scale, v_scale) as fp32 pools of block_size 4,
 * num_kv_heads = PA_SCALE_ROW(num_kv_heads) / 4 and head_dim 1.
 * A table row of these calls, and of pa_decode_weights over any pool, holds at
 * most 2^30 tokens (PA_ERR_SHAPE above).
 */
#define PA_SCALE_ROW(num_kv_heads) (((num_kv_heads) + 3) / 4 * 4)

/*
 * Quantising append into a block-scaled e4m3 cache.  Sequence b's new tokens
 * are rows query_start[b] .. query_start[b+1]-1 of key and value: the last
 * n_b tokens of its context (context_lens counts them).  For every block they
 * touch and every head, K and V each on their own:
 *
 *   a     = max |x| over the block's new finite elements of the head
 *   need  = the smallest power of two with a <= 448 * need, at least 2^-100
 *           (0 when a is 0)
 *   s     = max(need, the block's scale), the latter only if the block holds
 *           earlier tokens of the sequence; a block begun by this call starts
 *           from need
 *   codes = e4m3(x / s), nearest even, saturating; codes of the earlier tokens
 *           become e4m3(value(code) * old_scale / s)
 *
 * Powers of two make x / s exact and a raised scale exact for every code whose
 * value stays a normal one, so the tokens' split into calls hardly shows.  (Under a
 * scale of the caller's own that is no power of two, x / s is off by 2^-23 of itself
 * before it is rounded to a code.)
 * A NaN gives a NaN code; an infinity gives +-448 codes, or NaN codes where the
 * block's head holds nothing that is finite and not zero.
 *
 *   key, value     [total_tokens, num_kv_heads, head_dim], src_dtype PA_F32 or
 *                  PA_BF16
 *   query_start    [num_seqs + 1] int32, non-decreasing from 0 to total_tokens
 *                  (a sequence may add none)
 *
 * Blocks that receive tokens must belong to one sequence only (copy shared
 * ones first), named once in its table row.  A sequence whose rows or lengths
 * are inconsistent (rows outside [0, total_tokens], more rows than tokens, a
 * context longer than its table row) writes nothing and sets PA_DEV_BAD_LEN;
 * a block id outside the pool is skipped and sets PA_DEV_BAD_BLOCK.
 */
int pa_append_fp8_blocks(const void* key, const void* value,
                         const int32_t* query_start, int total_tokens,
                         const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, int num_seqs,
                         void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         int num_blocks, int block_size, int num_kv_heads, int head_dim,
                         pa_dtype src_dtype, void* stream);

/*
 * Paged decode attention over a block-scaled e4m3 cache: the result of
 * pa_decode over the dequantised pool.  The K scale multiplies the scores of a
 * block's tokens, the V scale their softmax weights (the normaliser uses the
 * unscaled weights), both in fp32.
 *
 *   query, out      PA_BF16
 *   partition_size  as for pa_decode, but for the automatic choice:
 *                   pa_decode_fp8_blocks_partition_size returns the size used
 *   workspace       at least pa_decode_fp8_blocks_workspace_bytes() with the
 *                   same sizes, 16-byte aligned (may be NULL when that is 0)
 *   other arguments as for pa_decode
 *
 * With block_size 8 to 32 and num_kv_heads * head_dim a multiple of 128 it runs
 * on the tcgen05 tensor cores, the codes as they are (8-bit products, fp32
 * accumulation): Q enters as two e4m3 terms, off by at most 2^-21 of the head's
 * largest element; the products of softmax weight and V scale as three e5m2 terms,
 * which hold a product to 2^-9 of itself (bf16's precision) down to 2^-26 of the
 * head's largest, and to 2^-35 of that largest below.  Everything else runs on CUDA
 * cores in fp32.
 */
int pa_decode_fp8_blocks(void* out, const void* query,
                         const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale,
                         const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, int num_seqs,
                         int num_heads, int num_kv_heads, int head_dim,
                         int block_size, int num_blocks, float scale, int partition_size,
                         void* workspace, size_t workspace_bytes,
                         pa_dtype dtype, void* stream);

/* Bytes of workspace pa_decode_fp8_blocks needs for these sizes, and the
 * partition size (tokens) it uses.  Pure host arithmetic; no CUDA call. */
size_t pa_decode_fp8_blocks_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                            int max_blocks_per_seq, int block_size, int partition_size);
int pa_decode_fp8_blocks_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                        int max_blocks_per_seq, int block_size, int partition_size);

/*
 * Causal attention of each sequence's newest tokens over a block-scaled e4m3
 * cache: pa_prefill_varlen's rows and positions, for every head_dim,
 * block_size and query group that pa_decode takes (num_seqs unlimited).  The
 * tokens' K/V are already appended.  Rows at negative positions are zeros.
 *
 *   out, query     [total_queries, num_heads, head_dim], PA_BF16
 *   query_start    [num_seqs + 1] int32, non-decreasing from 0 to total_queries
 *                  (a bad pair sets PA_DEV_BAD_LEN, and that sequence writes
 *                  nothing)
 *   scale          > 0
 *
 * A NaN value makes NaN of its head dim in the rows at and past its token, a NaN
 * key of those rows whole; the rows before are not touched by either.
 *
 * With head_dim 128, block_size 8 to 32 and at most 128 query heads per KV head it
 * runs on the tcgen05 tensor cores: a query row enters as an e4m3 and an e5m2 term,
 * off by at most 2^-20 of the row's largest element (exact down to 2^-13 of it); the
 * softmax weights and the dequantised values are rounded to bf16 once each (which a
 * power of two as the scale leaves exact).  Everything else runs in fp32.
 */
int pa_prefill_fp8_blocks(void* out, const void* query, const int32_t* query_start, int total_queries,
                          const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale,
                          const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* context_lens, int num_seqs,
                          int num_heads, int num_kv_heads, int head_dim,
                          int block_size, int num_blocks, float scale,
                          pa_dtype dtype, void* stream);

/*
 * Decode that keeps account of what attention looks at.  out is pa_decode's
 * (or pa_decode_fp8_blocks') result; besides, with w[b,h,t] the softmax weight
 * of token t for query head h of sequence b,
 *
 *   weights[b, g, t] += sum over the query heads h of KV head g of w[b,h,t]
 *
 * for t < L_b (the rest of a row is untouched), in fp32 and in head order: the
 * same call gives the same totals.  A token's total starts from what the
 * caller put there: 0 for a new token (pa_evict leaves zeros behind).
 *
 *   weights         [num_seqs, num_kv_heads] rows of weights_stride floats,
 *                   weights_stride >= max_blocks_per_seq * block_size
 *   dtype           of query and out
 *   kv_dtype        of the pools: dtype itself, or PA_FP8_E4M3 (block-scaled,
 *                   dtype PA_BF16); k_scale, v_scale are used only then
 *   workspace       at least pa_decode_weights_workspace_bytes(), 16-byte
 *                   aligned: the split-K partials and an fp32 score per (query
 *                   head, table slot)
 *   other arguments as for pa_decode; num_heads / num_kv_heads <= 1024
 */
int pa_decode_weights(void* out, float* weights, long long weights_stride,
                      const void* query, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim,
                      int block_size, int num_blocks, float scale, int partition_size,
                      void* workspace, size_t workspace_bytes,
                      pa_dtype dtype, pa_dtype kv_dtype, void* stream);

/* Bytes of workspace pa_decode_weights needs for these sizes.  Pure host
 * arithmetic; no CUDA call. */
size_t pa_decode_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                         int max_blocks_per_seq, int block_size, int partition_size,
                                         pa_dtype kv_dtype);

/*
 * Evict: cut the cache of every (sequence, KV head) to `budget` tokens.  Each
 * KV head keeps tokens of its own choice; all heads of a sequence keep the
 * same number, so its new length is min(L_b, budget).
 *
 * Slot t < L_b of (b, g) holds the token at position
 *   pos(t) = token_pos[b,g,t]        for t < kept_lens[b]
 *            seen_lens[b] - L_b + t  for the tokens appended since.
 * Protected are pos < sinks and pos >= seen_lens[b] - recent.  Where
 * L_b > budget, the `budget` tokens stay that come first by: protected, then
 * larger weights[b,g,t] (NaN last), then lower t.  Kept tokens in slots below
 * the budget keep their slot; the i-th kept token (by slot) at or above the
 * budget moves into the i-th slot below it whose token was dropped.  K/V rows,
 * weights and positions move together; attention over the cache does not
 * depend on the order of its rows.  Rows of a PA_FP8_E4M3 (block-scaled) pool
 * are requantised: a block that receives rows takes the largest of its scale
 * and theirs, and its own remaining rows follow it.
 *
 *   kept_lens    [num_seqs] int32: tokens whose token_pos entry is valid, i.e.
 *                new_lens of the sequence's last eviction (0 before the first)
 *   seen_lens    [num_seqs] int32: tokens the sequence has had in all, the
 *                dropped ones included (L_b before its first eviction)
 *   weights, token_pos  [num_seqs, num_kv_heads] rows of row_stride floats /
 *                int32, row_stride >= max_blocks_per_seq * block_size (which is
 *                at most 6291456 tokens)
 *   budget, recent, sinks   >= 1, >= 0, >= 0; recent + sinks <= budget
 *   new_lens     [num_seqs] int32 (written); may be context_lens or kept_lens
 *   weights_out, token_pos_out  rows like weights and token_pos (written: the
 *                kept tokens' entries, then 0 and -1 up to max_blocks_per_seq *
 *                block_size); may be weights and token_pos themselves, with no
 *                other overlap
 *   workspace    at least pa_evict_workspace_bytes(), 16-byte aligned; calls
 *                that share one must be ordered
 *
 * The blocks of a sequence must be its own (copy shared ones first).  Blocks
 * wholly past the new length are the caller's to free.  A context length
 * outside its table row, or a kept length outside the context, is clamped and
 * sets PA_DEV_BAD_LEN; a move from or to a block id outside the pool is skipped
 * and sets PA_DEV_BAD_BLOCK.  A pool with per-token scales
 * (pa_reshape_and_cache_fp8) cannot be evicted by head: one scale there serves
 * all heads of a token.
 */
int pa_evict(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
             const int32_t* block_tables, int max_blocks_per_seq,
             const int32_t* context_lens, const int32_t* kept_lens, const int32_t* seen_lens, int num_seqs,
             const float* weights, const int32_t* token_pos,
             int budget, int recent, int sinks,
             int32_t* new_lens, float* weights_out, int32_t* token_pos_out, long long row_stride,
             int num_blocks, int block_size, int num_kv_heads, int head_dim,
             void* workspace, size_t workspace_bytes, pa_dtype kv_dtype, void* stream);

/* Bytes of workspace pa_evict needs for these sizes.  Pure host arithmetic. */
size_t pa_evict_workspace_bytes(int num_seqs, int num_kv_heads, int max_blocks_per_seq, int block_size, int budget);

/*
 * Swap blocks between two pools (preemption by swapping).  [KVS] §19.2.6:
 * a preempted request's KV cache can be moved out to CPU memory and moved
 * back when GPU memory frees up; [OS] §九 names the same swap-out.  For each
 * pair i, block pairs[2i+1] of the destination pool (dst_k, dst_v) becomes a
 * byte-exact copy of block pairs[2i] of the source pool (src_k, src_v), all
 * slots and heads.  Both pools have the [num_blocks, block_size,
 * num_kv_heads, head_dim] layout; their block counts may differ.
 *
 *   dst_*, src_*  device-accessible addresses: device memory, or page-locked
 *                 host memory the device can address (on GB300 such host
 *                 memory is reached over NVLink-C2C by the copy kernel itself,
 *                 so no staging buffer is needed)
 *   pairs         [num_pairs, 2] int64 (src block, dst block), device memory;
 *                 destination blocks distinct, pools not overlapping
 *
 * A pair naming a block outside its pool is skipped and sets
 * PA_DEV_BAD_BLOCK.  num_pairs == 0 launches nothing.  Shapes and dtypes as
 * for pa_copy_blocks (an e4m3 pool swaps its scale rows by a second call).
 */
int pa_swap_blocks(void* dst_k, void* dst_v, int dst_num_blocks,
                   const void* src_k, const void* src_v, int src_num_blocks,
                   const int64_t* pairs, int num_pairs,
                   int block_size, int num_kv_heads, int head_dim,
                   pa_dtype dtype, void* stream);

/*
 * Decode that allocates nothing and takes no workspace.  This entry point
 * has no counterpart on the paged-attention pages; it exists for callers
 * that cannot allocate device memory at the point of the call — for example
 * a plug-in whose host engine owns every device allocation through its own
 * pool, or a latency-critical path that cannot afford an allocation call
 * that may synchronise the device.
 *
 * Same arguments and result as pa_decode, without workspace: the split-K
 * scratch is a PA_NOALLOC_SCRATCH_BYTES array compiled into the library,
 * held by every device that loads the library until the process exits.
 *  - Sizes whose pa_decode_workspace_bytes() exceeds that limit are rejected
 *    with PA_ERR_WORKSPACE (nothing launched; pa_last_host_error() says how
 *    much was needed).
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it, and so does the first call after
 *    the device's context has changed (e.g. after cudaDeviceReset()); make
 *    such a call before any stream capture.
 *  - Every call on a device shares the one array and it keeps the previous
 *    call's contents: calls whose GPU work overlaps (e.g. on two streams)
 *    race on it and must be ordered by the caller.  Nothing in it needs to
 *    start at zero.
 *  - It calls no cudaMalloc, cudaFree or other allocating routine.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
int pa_decode_noalloc(void* out, const void* query,
                      const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim,
                      int block_size, int num_blocks, float scale, int partition_size,
                      pa_dtype dtype, void* stream);

/* Bytes of workspace pa_decode needs for these sizes (0 when no sequence can
 * span more than one partition).  Pure host arithmetic; no CUDA call. */
size_t pa_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                 int max_blocks_per_seq, int block_size, int partition_size);

/* The partition size (tokens) pa_decode will use for these arguments. */
int pa_decode_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                             int max_blocks_per_seq, int block_size, int partition_size);

/* The partition size (tokens) pa_decode_fp8 will use for these arguments. */
int pa_decode_fp8_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                 int max_blocks_per_seq, int block_size, int partition_size);

/*
 * Copy-on-write block copy.  [KVS] Fig 19-8 and [OS] §四: before a sequence
 * writes into a block that other sequences still share, a new block is
 * allocated and the old contents are copied into it.  For each pair i,
 * block pairs[2i+1] of both k_cache and v_cache becomes a byte-exact copy of
 * block pairs[2i] (all block_size slots, all heads).
 *
 *   pairs   [num_pairs, 2] int64 (src, dst), device memory.  dsts must be
 *           distinct and no dst may be the src of another pair; if they are
 *           not, the contents of the blocks involved are undefined (nothing
 *           is flagged).  A pair whose src equals its dst changes nothing.
 *
 * A pair with an id outside [0, num_blocks) is skipped and sets
 * PA_DEV_BAD_BLOCK.  num_pairs == 0 launches nothing.
 *
 * Pure byte movement, so any dtype (PA_FP8_E4M3 included) and any
 * num_kv_heads, head_dim >= 1 whose block (block_size * num_kv_heads *
 * head_dim * element bytes) is a multiple of 16 bytes.  For an e4m3 pool,
 * copy its scale rows with a second call with the same pairs on
 * (k_scale, v_scale) as an fp32 pool with num_kv_heads = head_dim = 1.
 */
int pa_copy_blocks(void* k_cache, void* v_cache, const int64_t* pairs, int num_pairs,
                   int num_blocks, int block_size, int num_kv_heads, int head_dim,
                   pa_dtype dtype, void* stream);

/*
 * Causal chunked-prefill query tile over the paged cache ([OS] §8.1: a long
 * prompt is processed in chunks, each continuing from the tokens already in
 * the cache).  The tile is the LAST num_queries tokens of each sequence's
 * context, their K/V already appended: query i of sequence b sits at
 * position p = context_lens[b] - num_queries + i and attends to positions
 * 0..p of its paged context (query head h reads KV head h / G).  Rows with
 * p < 0 are written as zeros.
 *
 *   out, query  [num_seqs, num_queries, num_heads, head_dim]
 *   other arguments as for pa_decode.
 *
 * Runs on the tcgen05 tensor cores: PA_BF16, head_dim 128, block_size in
 * {8, 16, 32}, G = num_heads / num_kv_heads in {1, 2, 4, 8, 16}; anything
 * else returns PA_ERR_SHAPE, as does scale <= 0.  P is rounded to bf16 before
 * the P*V product; accumulation is fp32.
 */
int pa_prefill_paged(void* out, const void* query, int num_queries,
                     const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int num_seqs,
                     int num_heads, int num_kv_heads, int head_dim,
                     int block_size, int num_blocks, float scale,
                     pa_dtype dtype, void* stream);

/*
 * Mixed round in one launch: decode requests and prefill chunks together
 * ([OS] §8.1 chunked prefill; §8.2: one round's token budget covers decode
 * tokens, new prefill tokens and chunked-prefill tokens).  Sequence b
 * contributes n_b = query_start[b+1] - query_start[b] query rows, its last
 * n_b tokens (K/V already appended): n_b = 1 for a decode request, the chunk
 * length for a prefill chunk, 0 for a sequence with no work this round.
 * Row i of sequence b sits at position p = context_lens[b] - n_b + i and
 * attends causally to positions 0..p (rows with p < 0 are zeros).
 *
 *   out, query     [total_queries, num_heads, head_dim], rows in sequence
 *                  order: sequence b's rows start at query_start[b]
 *   query_start    [num_seqs + 1] int32, device, non-decreasing, starting
 *                  at 0 and ending at total_queries (a decreasing pair, or
 *                  a start outside 0..total_queries, sets PA_DEV_BAD_LEN
 *                  and that sequence writes nothing)
 *   other arguments as for pa_prefill_paged; num_seqs <= 2048
 *
 * The same tcgen05 kernel as pa_prefill_paged: each (query tile, KV head)
 * is one CTA, tiles of 128 / G query positions; a decode request is a
 * tile with one position.
 */
int pa_prefill_varlen(void* out, const void* query, const int32_t* query_start, int total_queries,
                      const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim,
                      int block_size, int num_blocks, float scale,
                      pa_dtype dtype, void* stream);

/*
 * Rotary positions.  Pair i of a head at position p is turned by the angle
 * p * f_i and multiplied by an amplitude A:
 *
 *   (x, y) -> A (x cos(p f_i) - y sin(p f_i), y cos(p f_i) + x sin(p f_i))
 *
 * for the first rotary_dim elements of the head; the rest stays as it is.
 *
 *   PA_ROPE_HALF         pair i is elements i and i + rotary_dim / 2
 *   PA_ROPE_INTERLEAVED  pair i is elements 2 i and 2 i + 1
 *
 * The frequencies come as a table of steps: steps[i] = round(2^64 f_i / 2 pi),
 * the fraction of a turn that one position makes, so that p * steps[i] modulo
 * 2^64 is the turn's fraction with no angle to reduce: right to 2^-33 of a turn
 * for every int32 position.  (The kernels take it as a float, off by 2^-25 of a
 * turn at most.)  pa_rope_steps fills a HOST table of rotary_dim / 2
 * entries (to be copied to the device) and *amplitude:
 *
 *   PA_ROPE_PLAIN   f_i = base^(-2 i / rotary_dim), A = 1; the other arguments
 *                   are not looked at
 *   PA_ROPE_LINEAR  f_i / factor (positions interpolated)
 *   PA_ROPE_NTK     the base times factor^(rotary_dim / (rotary_dim - 2))
 *   PA_ROPE_YARN    f_i ((1 - r_i) + r_i / factor), r_i rising from 0 to 1
 *                   between the pairs that make beta_fast and beta_slow turns
 *                   over original_len positions, A = 0.1 ln(factor) + 1
 *
 * rotary_dim is a multiple of 16 up to 512, base > 1, factor >= 1,
 * 0 < beta_slow <= beta_fast.  Pure host arithmetic; no CUDA call.
 */
typedef enum { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;
typedef enum { PA_ROPE_PLAIN = 0, PA_ROPE_LINEAR = 1, PA_ROPE_NTK = 2, PA_ROPE_YARN = 3 } pa_rope_scaling;
int pa_rope_steps(uint64_t* steps, float* amplitude, int rotary_dim, double base, pa_rope_scaling scaling,
                  double factor, double original_len, double beta_fast, double beta_slow);

/*
 * Rotate queries and keys.  Both are strided [num_tokens, heads, head_dim]
 * tensors (strides in elements, the innermost 1; a view into a fused
 * projection's output will do).  An output may be its input (same pointer and
 * strides: the elements past rotary_dim are then not touched) and must not
 * overlap it otherwise, nor itself, nor the other side.  A part of a head other
 * than its first elements is rotated through a pointer to it, with head_dim =
 * rotary_dim.
 *
 *   positions    [num_tokens] int32, any value
 *   num_heads, num_kv_heads  0 to 2^20: 0 leaves that side out
 *   head_dim     a multiple of 16 up to 512; rotary_dim <= head_dim likewise
 *   steps        device copy of the table of pa_rope_steps
 *   dtype        PA_F32 or PA_BF16; products in fp32, rounded once
 *
 * Pointers and strides are multiples of 16 bytes (PA_ERR_ALIGN); a token has at
 * most 2^28 bytes to move (PA_ERR_SHAPE).
 */
int pa_rope(void* q_out, long long q_out_token_stride, long long q_out_head_stride,
            const void* q, long long q_token_stride, long long q_head_stride, int num_heads,
            void* k_out, long long k_out_token_stride, long long k_out_head_stride,
            const void* k, long long k_token_stride, long long k_head_stride, int num_kv_heads,
            const int32_t* positions, int num_tokens, int head_dim, int rotary_dim,
            pa_rope_layout layout, const uint64_t* steps, float amplitude,
            pa_dtype dtype, void* stream);

/*
 * pa_rope and pa_reshape_and_cache in one launch: the queries rotated, the
 * keys rotated into their slots of k_cache, the values copied into v_cache.
 * Strides, positions, steps as for pa_rope; slots, pools and their conditions
 * as for pa_reshape_and_cache (a token without a slot has its queries rotated
 * all the same).  num_heads 0 leaves the queries out.
 */
int pa_rope_and_cache(void* q_out, long long q_out_token_stride, long long q_out_head_stride,
                      const void* q, long long q_token_stride, long long q_head_stride, int num_heads,
                      const void* key, long long key_token_stride, long long key_head_stride,
                      const void* value, long long value_token_stride, long long value_head_stride,
                      int num_kv_heads, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                      void* k_cache, void* v_cache, int num_blocks, int block_size, int head_dim, int rotary_dim,
                      pa_rope_layout layout, const uint64_t* steps, float amplitude,
                      pa_dtype dtype, void* stream);

/*
 * The latent cache: one vector a token for all heads.
 *
 *   cache  [num_blocks, block_size, latent_dim + rope_dim], row-major: the
 *          token's latent vector, then its rotated key
 *
 * latent_dim in {128, 256, 384, 512}, rope_dim in {16, 32, 48, 64}, block_size
 * in {8, 16, 32}.  Blocks are copied and swapped with pa_copy_blocks /
 * pa_swap_blocks, num_kv_heads = 1 and head_dim = latent_dim + rope_dim, two
 * layers' pools a call (or one pool as both).
 *
 * Append: row t of latent goes to slot slot_mapping[t] as it is, row t of
 * key_rope rotated behind it, and the rotary part of the token's queries
 * (strided [num_tokens, num_heads, rope_dim]) is rotated into query_out in the
 * same launch (num_heads 0 leaves it out).  Row strides in elements; alignment,
 * positions, steps and layouts as for pa_rope, slots as for
 * pa_reshape_and_cache.
 */
int pa_latent_append(const void* latent, long long latent_stride, const void* key_rope, long long key_rope_stride,
                     void* query_out, long long query_out_token_stride, long long query_out_head_stride,
                     const void* query, long long query_token_stride, long long query_head_stride, int num_heads,
                     const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                     void* cache, int num_blocks, int block_size, int latent_dim, int rope_dim,
                     pa_rope_layout layout, const uint64_t* steps, float amplitude,
                     pa_dtype dtype, void* stream);

/*
 * Attention over a latent cache in its absorbed form: every head's queries
 * meet the cached rows themselves, and the rows' latent part is the values.
 * With c_t row t of the context and q of latent_dim + rope_dim elements (the
 * query times the key's up-projection, then its rotated part),
 *
 *   out[r,h,:] = sum_t softmax_t(scale * <q[r,h,:], c_t>) c_t[:latent_dim]
 *
 * (to be multiplied by the value's up-projection).  Rows and positions are
 * pa_prefill_varlen's: sequence b's rows are query_start[b] ..
 * query_start[b+1]-1, the last of its context, and see it causally; rows at
 * negative positions are zeros, rows of no sequence are left as they were.
 *
 *   out            [total_queries, num_heads, latent_dim] (written)
 *   query          [total_queries, num_heads, latent_dim + rope_dim]
 *   query_start    [num_seqs + 1] int32, non-decreasing from 0 to
 *                  total_queries, or NULL: one row a sequence (total_queries =
 *                  num_seqs).  A bad pair sets PA_DEV_BAD_LEN, and that
 *                  sequence writes nothing.
 *   scale          > 0
 *   workspace      at least pa_latent_decode_workspace_bytes() with the same
 *                  sizes, 16-byte aligned; contents on entry do not matter,
 *                  calls that share one must be ordered
 *   dtype          PA_BF16
 *
 * A context length outside its table row is clamped and sets PA_DEV_BAD_LEN, a
 * block id outside the pool is read as block 0 and sets PA_DEV_BAD_BLOCK.  A
 * table row holds at most 2^30 tokens, total_queries * num_heads < 2^31, and
 * (total_queries * num_heads / G + num_seqs) * (a table row's tiles of 128
 * tokens) < 2^31 (PA_ERR_SHAPE), where G is 16 up to 16 (query, head) rows a
 * sequence, 32 up to 32, else 64 (total_queries / num_seqs, rounded up, times
 * num_heads).
 * Accumulation is fp32; the softmax weights are rounded to bf16 for their
 * product with the values.  A cached row that holds a NaN makes NaN of the rows
 * that see it, whole, and one that holds an infinity likewise or, for a row whose
 * score it makes -inf, of its elements; the rows before it are not touched.
 * Sums of weights (1 at most) times values are fp32 and divided at the end:
 * values whose sum passes 3.4e38 overflow.  A score of -inf is a weight of zero,
 * and a row of such scores alone is zeros, as in the other attention calls.
 *
 * The batch's tokens are divided evenly among the SMs by the lengths on the
 * device, and what a cut divides is joined by a second kernel (outside stream
 * capture its launch is a programmatic dependent of the first's): the same call
 * gives the same bits, another batch around a sequence may round it otherwise.
 */
int pa_latent_decode(void* out, const void* query, const int32_t* query_start, int total_queries,
                     const void* cache, const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int num_seqs, int num_heads, int latent_dim, int rope_dim,
                     int block_size, int num_blocks, float scale,
                     void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream);

/* Bytes of workspace pa_latent_decode needs for these sizes (whatever the
 * table's).  Pure host arithmetic; no CUDA call. */
size_t pa_latent_decode_workspace_bytes(int total_queries, int num_seqs, int num_heads, int latent_dim);

/*
 * Attention over latent vectors in their expanded form (prompts): keys and
 * values of every head, as the up-projection writes them, and one rotated key
 * shared by all heads.  With k[t,h,:] = (kv[t,h,:key_dim], key_rope[t,:]) and
 * v[t,h,:] = kv[t,h,key_dim:],
 *
 *   out[r,h,:] = sum_t softmax_t(scale * <q[r,h,:], k[t,h,:]>) v[t,h,:]
 *
 * over ragged sequences: sequence b's context is rows kv_start[b] ..
 * kv_start[b+1]-1 of kv and key_rope, its queries rows query_start[b] ..
 * query_start[b+1]-1, the last tokens of that context, causal.  (A chunk that
 * continues a cached context takes the cached rows back first: they are rows
 * of the latent pool, to be multiplied by the up-projection again.)
 *
 *   out             [total_queries, num_heads, value_dim] (written)
 *   query           [total_queries, num_heads, key_dim + rope_dim]
 *   kv              [total_kv, num_heads, key_dim + value_dim]
 *   key_rope        [total_kv, rope_dim], rows key_rope_stride elements apart
 *                   (a multiple of 16 bytes)
 *   query_start, kv_start  [num_seqs + 1] int32, non-decreasing from 0 to
 *                   total_queries / total_kv.  A bad pair, or a context of
 *                   more than 2^26 tokens, sets PA_DEV_BAD_LEN, and that
 *                   sequence writes nothing.  Rows at negative
 *                   positions (more rows than context) are zeros; rows of no
 *                   sequence are left as they were.
 *   key_dim, value_dim  32, 64 or 128; rope_dim 16, 32, 48 or 64
 *   scale           > 0
 *   dtype           PA_BF16; accumulation fp32, softmax weights rounded to
 *                   bf16 for their product with the values
 *
 * num_seqs <= 2048.  A NaN value makes NaN of its element in the rows that see
 * it, an infinite one makes it infinite (NaN beside one of the other sign, or
 * where its token's weight has underflowed: either), a NaN key makes NaN of those
 * rows whole; the rows before it are not touched by any.  Rows next to a value
 * that is not finite are computed a second time, with the (256 rows, head) pair
 * or less that they belong to.  Scores of -inf and sums of large values as for
 * pa_latent_decode.
 */
int pa_latent_prefill(void* out, const void* query, const int32_t* query_start, int total_queries,
                      const void* kv, const void* key_rope, long long key_rope_stride, const int32_t* kv_start,
                      int total_kv, int num_seqs, int num_heads, int key_dim, int rope_dim, int value_dim,
                      float scale, pa_dtype dtype, void* stream);

/* Return the sticky device-detected condition bits (PA_DEV_*) and clear
 * them.  Synchronises the current device; 0 means nothing was detected.
 * Returns PA_ERR_CUDA if the device cannot be read. */
int pa_last_error(void);

/* Text of the last host-side failure on the calling thread (which CUDA call
 * failed and why) after a call returned PA_ERR_CUDA; "" if none yet.  The
 * string is owned by the library and overwritten by the next failure. */
const char* pa_last_host_error(void);

/* Human-readable text for a PA_ERR_* code or a PA_DEV_* bit. */
const char* pa_strerror(int code);

/*
 * Health check of the bounded pipeline waits (a library facility; the pages
 * have no counterpart).  Every mbarrier wait in the decode and prefill
 * kernels gives up after 2 s, sets PA_DEV_TIMEOUT and lets the kernel finish,
 * so a stalled pipeline leaves the CUDA context usable and shows up in
 * pa_last_error().  This call exercises that path on its own: it launches one
 * 32-thread CTA that waits on a shared-memory mbarrier nothing arrives at,
 * giving up after limit_ns nanoseconds (1 .. 2e9).  Once the launch has run,
 * pa_last_error() includes PA_DEV_TIMEOUT.  Asynchronous on `stream`; touches
 * no global memory other than the status bit.  A limit outside the range
 * returns PA_ERR_SHAPE and launches nothing.
 */
int pa_selftest_bounded_wait(unsigned long long limit_ns, void* stream);

/* Library ABI version (major*100 + minor). */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
