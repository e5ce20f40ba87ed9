/*
 * tsv.h -- C ABI of libtsv, the GB300 (sm_103a) target-side verification step of
 * tree-based speculative decoding.
 *
 * One verification step is three calls on one CUDA stream, with no host
 * synchronisation between them:
 *   1. tsv_tree_verify_attn    -- attention of the flattened draft tree over the
 *                                 paged KV cache under the ancestor-only tree mask;
 *   2. tsv_tree_reject_sample  -- rejection-sampling walk of the tree (Sequoia-style
 *                                 sampling without replacement) plus a bonus token;
 *   3. tsv_kv_compact_accepted -- KV-cache rewrite of the accepted path
 *      (tsv_tree_reject_sample_compact runs 2 and 3 in one launch).
 * (Step 2 consumes target logits, which in a full model are produced from step
 * 1's output by the layers above attention; the library takes them as input.)
 *
 * Conventions for every entry point
 *  - All array pointers are caller-owned DEVICE memory on the current device,
 *    except where a comment says otherwise.  The library allocates no device
 *    memory and keeps no state between calls; calls are thread-safe.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default).
 *  - Host-side argument errors return TSV_ERR_ARG / TSV_ERR_UNSUPPORTED at once and
 *    launch nothing.  A failed launch returns TSV_ERR_CUDA.  tsv_last_error()
 *    gives a message for the calling thread's last failure.
 *  - Data errors found on the device never trap: they are written as bit masks to
 *    `seq_err[b]` (one int32 per sequence, overwritten by each call) and the
 *    sequence's outputs are poisoned as documented per call.
 *  - Layouts are row-major:  q/out [B, N, Hq, D];  caches [num_blocks, block_size,
 *    Hkv, D];  block_table [B, max_blocks];  seq_lens/ new_seq_lens [B];  parent,
 *    draft_tokens, u_accept, accepted_nodes, out_tokens [B, N];  target_logits,
 *    draft_probs [B, N, V];  u_bonus, accept_len, bonus_token, seq_err [B].
 *  - Logical slot t of sequence b lives at physical row
 *    block_table[b, t / block_size] * block_size + t % block_size of the caches.
 *
 * The tree (sglang report "Speculative decoding on sglang", sections "What is
 * Tree-Attention?" and "Tree-based Speculative Decoding (EAGLE) Implementation
 * Summary": draft candidates flattened to 1-D, verified in one pass under a tree
 * mask) is given per sequence as parent[b, i]: node 0 is the root, i.e. the last
 * accepted token (parent -1), and 0 <= parent[i] < i for i >= 1.  Node i's K/V is
 * already in the cache at logical slot seq_lens[b] + i (written by the caller's
 * projection, as serving engines do); the caller preallocates the blocks, so
 * seq_lens[b] + N <= max_blocks * block_size ("preallocated slots", vLLM PR #2188,
 * "Guide for reviewers").
 */
#ifndef TSV_H
#define TSV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TSV_OK = 0,
    TSV_ERR_ARG = 1,         /* null pointer, bad size, workspace too small */
    TSV_ERR_UNSUPPORTED = 2, /* valid but not built: e.g. D not in {64, 128} */
    TSV_ERR_CUDA = 3         /* a CUDA runtime/driver call or launch failed */
} tsv_status;

typedef enum { TSV_BF16 = 0, TSV_F32 = 1 } tsv_dtype;

/* Device-side data error bits written to seq_err[b]. */
enum {
    TSV_DERR_PARENT = 1,    /* parent array (or accepted path) is not a valid tree/path */
    TSV_DERR_BLOCK = 2,     /* a block id covering slots [0, L_b + N) is outside [0, num_blocks) */
    TSV_DERR_CAPACITY = 4,  /* L_b < 0 or L_b + N > max_blocks * block_size */
    TSV_DERR_TOKEN = 8,     /* a tried draft token is outside [0, V) */
    TSV_DERR_NONFINITE = 16, /* a visited logits row, or a draft row that is read, is not finite */
    TSV_DERR_TIMEOUT = 32,   /* internal: a bounded device-side wait gave up; outputs of the
                                sequence are not valid (never expected; reported, not trapped) */
    TSV_DERR_INTERNAL = 64,  /* checked builds only (-DTSV_CHECKED, a test build): a device-side
                                index check failed and the access was skipped -- a library bug */
    TSV_DERR_POOL = 128,     /* the pool of free blocks is too small, or its count is wrong */
    TSV_DERR_SEQ = 256       /* a sequence index is outside the batch, named twice or not empty; groups
                                that do not cover the batch in order */
};

/* Message for the calling thread's most recent failed call ("" if none). */
const char *tsv_last_error(void);

/* ---------------------------------------------------------------------------
 * Tree-masked GQA attention (sglang report, "What is Tree-Attention?"; the EAGLE
 * "Tree Decoding" step with attention_mask + tree_attention_mask).
 *
 * For query row (b, n, h), kv head g = h / (Hq / Hkv):
 *   keys = prefix slots 0 .. L_b-1  (all visible)
 *        + tree slots L_b + j for every node j on the root-to-n path, n included;
 *   out[b,n,h,:] = softmax_t(scale * q[b,n,h,:] . k[t,g,:]) @ v[t,g,:].
 * q, caches and out share `dtype` (bf16: tensor-core tiles, fp32 accumulation;
 * fp32: exact fp32 FMA path).  D in {64, 128}; 1 <= N <= 128; Hq % Hkv == 0;
 * block_size a power of two in [8, 128].
 * bf16: persistent CTAs split the 128-key tiles of all (sequence, kv head) pairs
 * evenly; a pair that straddles CTAs leaves partial (max, sum, output) in
 * `workspace`, combined by a merge kernel.  fp32: long prefixes are split into key
 * chunks whose partials are merged by a second kernel.  The call's kernels are
 * chained with programmatic dependent launch; each waits for the kernel before it
 * in the stream to complete before reading its inputs.
 * `workspace` must hold tsv_attn_workspace_size(...) bytes (may be NULL when that
 * is 0); it is scratch owned by the caller, and every byte the call reads there is
 * written earlier in the same call (no clearing needed between calls).
 * Rows of a sequence with seq_err != 0 are written as NaN.
 * Cache slots from L_b + N to the end of the sequence's last block are never
 * read into the result (they may hold anything, NaN included).
 * ------------------------------------------------------------------------- */
size_t tsv_attn_workspace_size(int B, int N, int Hq, int Hkv, int D, int block_size, int max_blocks,
                               tsv_dtype dtype);

tsv_status tsv_tree_verify_attn(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_table, const int32_t *seq_lens,
                                const int32_t *parent, void *out, int B, int N, int Hq, int Hkv,
                                int D, int block_size, int max_blocks, int num_blocks, float scale,
                                tsv_dtype dtype, void *workspace, size_t workspace_bytes,
                                int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * tsv_tree_verify_attn with the tree's own K/V appended in the same call (sglang
 * report, "Tree-based Speculative Decoding (EAGLE) Implementation Summary": the KV
 * cache is updated for the tree's tokens before they are verified; vLLM PR #2188,
 * "Guide for reviewers": no host synchronisation inside the step).
 *
 * k_new, v_new [B, N, Hkv, D] (dtype as q) are the tree nodes' K/V rows; node j's row
 * is written to logical slot seq_lens[b] + j of k_cache / v_cache (all kv heads), and
 * the attention then reads it there, exactly as tsv_tree_verify_attn does once the
 * caller has written the rows: same results, same workspace, same errors.  A sequence
 * whose capacity or block ids fail the checks (TSV_DERR_CAPACITY / TSV_DERR_BLOCK)
 * gets no rows written.  The rows are written by the sequence-check kernel, and the
 * attention kernel waits for that kernel (programmatic dependent launch) before its
 * first tile that reaches the tree keys, so the append adds no launch on the bf16
 * path (fp32: one small kernel before the attention).  k_new / v_new must be 16-byte
 * aligned and must not overlap the caches.
 * ------------------------------------------------------------------------- */
tsv_status tsv_tree_verify_attn_append(const void *q, const void *k_new, const void *v_new, void *k_cache,
                                       void *v_cache, const int32_t *block_table,
                                       const int32_t *seq_lens, const int32_t *parent, void *out, int B,
                                       int N, int Hq, int Hkv, int D, int block_size, int max_blocks,
                                       int num_blocks, float scale, tsv_dtype dtype, void *workspace,
                                       size_t workspace_bytes, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * tsv_tree_verify_attn without a caller workspace (the pages have no counterpart
 * of this call; it is an interface convenience).
 *
 * For callers that cannot allocate device memory -- e.g. a plugin inside an engine
 * that owns all device memory and passes only inputs and outputs, or a loop that
 * must not call cudaMalloc because it can synchronise the device.  Same arguments
 * and result as tsv_tree_verify_attn, minus the workspace: the split-K partials go
 * to a scratch array of tsv_noalloc_scratch_bytes() (64 MiB) that the library
 * defines in device memory; every GPU that loads the library holds it until the
 * process exits.  Nothing is allocated per call.
 *  - Shapes whose tsv_attn_workspace_size exceeds the array are rejected with
 *    TSV_ERR_UNSUPPORTED before anything is launched.
 *  - The array used is the CURRENT device's: the current device must be the device
 *    of `stream` and of every buffer (a stream of another device is refused with
 *    TSV_ERR_ARG).
 *  - The first call on a device looks up the array's device address (once per
 *    device, with that device current; again only if the device's context changes,
 *    e.g. after cudaDeviceReset, which reloads the array with the module); make that
 *    first call before any stream capture.  A failed lookup returns TSV_ERR_CUDA and
 *    is retried by the next call.
 *  - All calls share the array: calls that overlap on the GPU race on it and must
 *    be ordered by the caller.  Each call rewrites every scratch byte it reads.
 * ------------------------------------------------------------------------- */
size_t tsv_noalloc_scratch_bytes(void);

tsv_status tsv_tree_verify_attn_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                        const int32_t *block_table, const int32_t *seq_lens,
                                        const int32_t *parent, void *out, int B, int N, int Hq,
                                        int Hkv, int D, int block_size, int max_blocks,
                                        int num_blocks, float scale, tsv_dtype dtype,
                                        int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * Rejection-sampling verification of the tree (statistical-learning-notes ch.07
 * "Speculative Decoding", section "Draft Token Validation"; Sequoia summary,
 * sections "Scalable Speculative Decoding" and "Robust Sampling").
 *
 * Per sequence, starting at the root i = 0:
 *   p = softmax(target_logits[b,i,:] / T), q = draft_probs[b,i,:];
 *   children c of i are tried in increasing index with x = draft_tokens[b,c]:
 *     accept iff u_accept[b,c] < p(x)/q(x)   (q(x) == 0: accept iff p(x) > 0);
 *     on rejection p <- normalize(max(0, p - q)) (kept if that sum is 0),
 *                  q(x) <- 0, q <- normalize(q) (kept if that sum is 0);
 *   the first accepted child becomes i; when no child is accepted (or i is a
 *   leaf) the walk stops and the bonus token is the smallest t with
 *   u_bonus[b] < sum_{v<=t} p(v) over the current p; if there is none (u_bonus >= 1
 *   or NaN, outside the stated [0, 1)), the last t with p(t) > 0.
 * T == 0: a child is accepted iff its token is argmax target_logits[b,i,:]
 * (lowest index on ties) and the bonus is that argmax; draft_probs and the
 * uniforms are not read (draft_probs may be NULL).
 * Outputs: accepted_nodes[b,:] = root-first path, -1 padded; accept_len[b] =
 * drafts accepted (path length - 1); bonus_token[b]; out_tokens[b,:] = accepted
 * draft tokens then the bonus, -1 padded.  A sequence with seq_err != 0 gets
 * accept_len = bonus_token = -1 and all-(-1) rows.
 * Uniforms are pre-drawn by the caller in [0, 1).  T == 0 or T >= 1e-6 (smaller
 * positive T is refused with TSV_ERR_UNSUPPORTED).  Vocabulary-wide sums use fp32
 * per thread and float-float pairs (about 44 significant bits) across threads, warps
 * and CTAs; the ratio p(x)/q(x) is formed in float-float from a compensated exponent
 * argument (relative error a few 1e-7).  V <= 16 * 512 * 32.
 * ------------------------------------------------------------------------- */
tsv_status tsv_tree_reject_sample(const float *target_logits, const float *draft_probs,
                                  const int32_t *draft_tokens, const int32_t *parent,
                                  const float *u_accept, const float *u_bonus, float temperature,
                                  int B, int N, int V, int32_t *accepted_nodes, int32_t *accept_len,
                                  int32_t *bonus_token, int32_t *out_tokens, int32_t *seq_err,
                                  void *stream);

/* ---------------------------------------------------------------------------
 * Variants of the walk (a host struct, read during the call; NULL = the defaults
 * {0, TSV_F32, 0, 1.0f}, i.e. tsv_tree_reject_sample).
 *
 * with_replacement: how the caller's drafter drew the siblings of a node.
 *   0 -- without replacement (Sequoia summary, "Robust Sampling"): the walk above.
 *   1 -- independently from q (the SpecInfer verification that the Sequoia summary's
 *        figure of rejection rates compares against, "More on figures"): after a
 *        rejected sibling only p takes the residual update, p <- normalize(max(0,
 *        p - q)); q is kept (no q(x) <- 0), so siblings may repeat a token.
 *   The walk must match the drafting: each is lossless only for its own drafts.
 * logits_dtype: element type of target_logits, TSV_F32 or TSV_BF16 (the target
 *   model's own output dtype; a bf16 row is half the bytes of an fp32 one).  A bf16
 *   logit is decoded exactly to fp32; everything after the load is the fp32 walk.
 * top_k, top_p: filtered target (the Sequoia summary's table of robustness to
 *   top-p sampling, "More on tables"): at every visited node p is first restricted
 *   to its top_k most probable tokens (top_k = 0: all), then to the smallest prefix
 *   of them, by decreasing p with ties to the lower index, whose mass reaches top_p
 *   (top_p = 1: all), and renormalised; q is the drafter's own (filtered)
 *   distribution as given.  top_k >= V keeps every token.  The cut is found by
 *   bisection over the logits' order (about 35 cluster reductions per visited node,
 *   a few more when the boundary falls inside a run of equal logits), so a filtered
 *   walk costs several times the plain one.  Mass sums are float-float; a cut whose
 *   cumulative mass lies within ~1e-7 of top_p may differ from an exact computation.
 * ------------------------------------------------------------------------- */
typedef struct {
    int with_replacement;
    tsv_dtype logits_dtype;
    int top_k;
    float top_p;
} tsv_walk_options;

/* tsv_tree_reject_sample with options; target_logits has opts->logits_dtype. */
tsv_status tsv_tree_reject_sample_ex(const void *target_logits, const float *draft_probs,
                                     const int32_t *draft_tokens, const int32_t *parent,
                                     const float *u_accept, const float *u_bonus, float temperature,
                                     const tsv_walk_options *opts, int B, int N, int V,
                                     int32_t *accepted_nodes, int32_t *accept_len, int32_t *bonus_token,
                                     int32_t *out_tokens, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * KV-cache rewrite for the accepted path (sglang report: the KV cache must be
 * updated selectively for accepted indices and trees require a rewrite; SGLang
 * "SpeculativeDecoding", prefix match: rejected tokens' KV cache is evicted).
 *
 * For j = 1 .. accept_len[b]: the K and V rows (all kv heads) at logical slot
 * L_b + accepted_nodes[b,j] move to logical slot L_b + j; new_seq_lens[b] =
 * L_b + 1 + accept_len[b].  Slots at or past the new length are evicted by the
 * length cut (their bytes are not cleared; freeing blocks is the caller's).
 * seq_lens is read only, so a repeated call gives the same result.
 * accept_len[b] < 0 leaves the sequence untouched (new_seq_lens[b] = L_b).
 * The path must satisfy 0 = a_0 < a_1 < ... < a_A < N (else TSV_DERR_PARENT).
 * ------------------------------------------------------------------------- */
tsv_status tsv_kv_compact_accepted(void *k_cache, void *v_cache, const int32_t *block_table,
                                   const int32_t *seq_lens, const int32_t *accepted_nodes,
                                   const int32_t *accept_len, int32_t *new_seq_lens, int B, int N,
                                   int Hkv, int D, int block_size, int max_blocks, int num_blocks,
                                   tsv_dtype dtype, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * The walk and the KV-cache rewrite in one launch: the same arguments and results as
 * tsv_tree_reject_sample(...) followed by tsv_kv_compact_accepted(k_cache, v_cache,
 * block_table, seq_lens, accepted_nodes, accept_len, new_seq_lens, ..., compact_err)
 * on the same stream (the rewrite runs in the walk kernel's tail, one CTA per
 * sequence, so it costs no launch of its own).  Walk errors go to seq_err, rewrite
 * errors to compact_err, with the same codes as the two calls.
 * ------------------------------------------------------------------------- */
tsv_status tsv_tree_reject_sample_compact(const float *target_logits, const float *draft_probs,
                                          const int32_t *draft_tokens, const int32_t *parent,
                                          const float *u_accept, const float *u_bonus,
                                          float temperature, int B, int N, int V,
                                          int32_t *accepted_nodes, int32_t *accept_len,
                                          int32_t *bonus_token, int32_t *out_tokens, int32_t *seq_err,
                                          void *k_cache, void *v_cache, const int32_t *block_table,
                                          const int32_t *seq_lens, int32_t *new_seq_lens, int Hkv,
                                          int D, int block_size, int max_blocks, int num_blocks,
                                          tsv_dtype dtype, int32_t *compact_err, void *stream);

/* tsv_tree_reject_sample_compact with the walk options above. */
tsv_status tsv_tree_reject_sample_compact_ex(const void *target_logits, const float *draft_probs,
                                             const int32_t *draft_tokens, const int32_t *parent,
                                             const float *u_accept, const float *u_bonus, float temperature,
                                             const tsv_walk_options *opts, int B, int N, int V,
                                             int32_t *accepted_nodes, int32_t *accept_len,
                                             int32_t *bonus_token, int32_t *out_tokens, int32_t *seq_err,
                                             void *k_cache, void *v_cache, const int32_t *block_table,
                                             const int32_t *seq_lens, int32_t *new_seq_lens, int Hkv, int D,
                                             int block_size, int max_blocks, int num_blocks, tsv_dtype dtype,
                                             int32_t *compact_err, void *stream);

/* ---------------------------------------------------------------------------
 * Operators around the step: the slot plan, the rotary K/V append and single-token
 * attention.  They read and write the same paged cache as the calls above (a block
 * allocator on the device: vLLM PR #2188, "Guide for reviewers", preallocated slots).
 * A decoding step is
 *   tsv_kv_plan_slots -> (projection) tsv_rope_kv_append -> tsv_decode_attn     one token
 *   tsv_kv_plan_slots -> tsv_rope_kv_append -> tsv_tree_verify_attn -> the walk  a tree
 * with seq_lens of tsv_decode_attn = total_lens of the plan, and seq_lens of
 * tsv_tree_verify_attn = seq_lens of the plan (its tree tokens are in the cache already).
 * ------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------
 * Block tables, slot maps and positions from request lengths, on the device.
 *
 * Sequence b has L_b = seq_lens[b] cached tokens, n_b = new_lens[b] tokens about to be
 * written and blocks_held[b] blocks (the first entries of its table row).  With
 * want = ceil((L_b + n_b) / block_size):
 *   1. sequences with want < held give back the blocks of entries want .. held-1, in
 *      order of (b, entry), onto the stack free_blocks[0 .. free_count) (num_blocks
 *      places); a finished request is L_b = n_b = 0.  The entries keep their old values;
 *   2. sequences with want > held take want - held blocks from the top of that stack, in
 *      order of (b, entry), into entries held .. want-1;
 *   3. new token j of sequence b is token i = token_offsets[b] + j of the batch
 *      (token_offsets[0 .. B]: running sums of new_lens) and gets
 *      slot_map[i] = table[b, (L_b + j) / bs] * bs + (L_b + j) % bs   and
 *      positions[i] = L_b + j, or, with `parent` [B, N] (a draft tree, n_b <= N; the
 *      tree's rules are those of the attention call), L_b + depth of node j;
 *      places of slot_map / positions past the last token are -1.
 * blocks_held_out[b] = want, total_lens[b] = L_b + n_b, *free_count_out = blocks left.
 * blocks_held_out, free_count_out and total_lens may be the input arrays blocks_held,
 * free_count and seq_lens (in-place update); nothing else may overlap.  With separate
 * outputs, and no change in between, a repeated call gives the same result.
 *
 * seq_err[b], overwritten: TSV_DERR_CAPACITY (negative length, L_b + n_b > max_blocks * bs,
 * blocks_held[b] outside [0, max_blocks], tokens past max_tokens), TSV_DERR_PARENT
 * (n_b > N), TSV_DERR_POOL (too few free blocks for this sequence after those before it --
 * no later sequence that needs blocks gets any then; *free_count outside [0, num_blocks];
 * more blocks given back than the pool has places for): the sequence keeps its
 * blocks, total_lens[b] = L_b (0 for a negative length), its tokens get slot and position -1,
 * the others are served.  TSV_DERR_BLOCK (a block id outside [0, num_blocks): its tokens'
 * slots are -1; one given back goes onto the stack as it is) and TSV_DERR_PARENT for a
 * parent row that is not a tree (positions of the nodes below the fault are -1) leave
 * the rest of the sequence as planned.
 * Negative lengths count as no tokens.  B = 0: slot_map and positions are -1 throughout, token_offsets[0]
 * is 0 and *free_count_out = *free_count (arrays of B entries and free_blocks may be NULL; with
 * these five NULL too the call writes nothing).  B <= 8192; block_size a power of two in
 * [8, 128]; max_blocks * block_size, max_tokens and num_blocks up to 2^30.
 * ------------------------------------------------------------------------- */
tsv_status tsv_kv_plan_slots(const int32_t *seq_lens, const int32_t *new_lens, const int32_t *parent,
                             int32_t *block_table, const int32_t *blocks_held, int32_t *blocks_held_out,
                             int32_t *free_blocks, const int32_t *free_count, int32_t *free_count_out,
                             int32_t *total_lens, int32_t *token_offsets, int64_t *slot_map,
                             int32_t *positions, int B, int N, int block_size, int max_blocks,
                             int num_blocks, int max_tokens, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * Rotary positions and the K/V append.
 *
 * Token t's rows q[t] [Hq, D], k[t], v[t] [Hkv, D] start q_stride, k_stride, v_stride
 * elements after the one before (heads and elements contiguous), so they may be parts of one
 * projection's rows.  Pair i of a head's first rotary_dim elements turns by
 * theta = positions[axis(i), t] * inv_freq[i] (positions [axes, T], inv_freq
 * [rotary_dim / 2]):  (x, y) <- (x cos - y sin, y cos + x sin); the rest passes through.
 * The turned q goes to q_out[t] (q_out_stride; q_out may be q with the same stride), the
 * turned k and v to cache slot slot_map[t].  The angle is formed to about 2^-22 of a turn while
 * |position| and |position * inv_freq| are below 2^24.  Arithmetic is fp32, rounded once to dtype.
 * slot_map[t] < 0 (padding): nothing is written to the cache and q_out[t] is zero.
 * slot_map[t] >= num_blocks * block_size: nothing is written to the cache, q_out[t] is NaN
 * and tok_err[t] = TSV_DERR_BLOCK (otherwise 0; one int32 per token, overwritten).
 * Slots that are not negative must differ; q, k, v and the caches must not overlap
 * (but for q_out = q).  D in {64, 128}; rotary_dim a multiple of 16; bases and strides
 * 16-byte aligned; Hq * D and Hkv * D up to 2^28.  opts NULL: {D, 0, 1, 0, {D / 2}}.
 * ------------------------------------------------------------------------- */
typedef struct {
    int rotary_dim;  /* elements of a head that turn */
    int neighbours;  /* pairs: 0 -- (i, i + rotary_dim / 2), 1 -- (2i, 2i + 1) */
    int axes;        /* position axes (time, height, width, ...): 1 to 4 */
    int rounds;      /* which axis a pair takes: 0 -- section after section, 1 -- the axes in
                        turn, an axis dropping out when its section is used up */
    int sections[4]; /* pairs of each axis; their sum is rotary_dim / 2 */
} tsv_rope_options;

tsv_status tsv_rope_kv_append(const void *q, const void *k, const void *v, const int32_t *positions,
                              const float *inv_freq, void *q_out, void *k_cache, void *v_cache,
                              const int64_t *slot_map, int T, int Hq, int Hkv, int D, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int64_t q_out_stride, int block_size,
                              int num_blocks, tsv_dtype dtype, const tsv_rope_options *opts,
                              int32_t *tok_err, void *stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per sequence over the paged cache.
 *
 * For query row (b, h), kv head g = h / (Hq / Hkv), keys = slots 0 .. L_b - 1 with
 * L_b = seq_lens[b] (the new token's own K/V row included, already written):
 *   out[b,h,:] = softmax_t(scale * q[b,h,:] . k[t,g,:]) @ v[t,g,:],
 *   lse[b,h] = ln sum_t exp(scale * q[b,h,:] . k[t,g,:])   (lse may be NULL).
 * q, out [B, Hq, D]; lse [B, Hq] fp32.  L_b = 0: out is zero and lse -infinity.  Sums and weights
 * are fp32 (a bf16 call's weights within 2^-15 of themselves); out is rounded once to dtype.
 * Slots past L_b are never read into the result.  The keys of all sequences are divided
 * evenly between the GPU's SMs; pieces of a sequence are joined by log-sum-exp in a fixed order, so a
 * repeated call gives the same bits.  `workspace` as in tsv_tree_verify_attn, with
 * tsv_decode_attn_workspace_size(...) bytes; calls that may overlap on the GPU need one each.
 * out and lse must not overlap the inputs.
 * seq_err[b]: TSV_DERR_CAPACITY (L_b < 0 or > max_blocks * block_size), TSV_DERR_BLOCK (a
 * block id covering [0, L_b) outside [0, num_blocks)); rows of a flagged sequence are NaN.
 * D in {64, 128}; Hq % Hkv == 0; block_size a power of two in [8, 128];
 * max_blocks * block_size and B * Hq up to 2^30; Hq * D up to 2^28; scale > 0, scale * log2(e) finite.
 * ------------------------------------------------------------------------- */
size_t tsv_decode_attn_workspace_size(int B, int Hq, int Hkv, int D, int block_size, int max_blocks,
                                      tsv_dtype dtype);

tsv_status tsv_decode_attn(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_table, const int32_t *seq_lens, void *out, float *lse,
                           int B, int Hq, int Hkv, int D, int block_size, int max_blocks,
                           int num_blocks, float scale, tsv_dtype dtype, void *workspace,
                           size_t workspace_bytes, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * Several continuations of one prompt (samples, beams) on the same paged cache: sequences forked on
 * shared blocks, attention that reads a shared prefix once, log probabilities to rank them by.
 *   tsv_kv_fork_seqs -> tsv_kv_copy_blocks (each layer) -> steps with tsv_prefix_decode_attn
 *   -> tsv_token_logprobs -> tsv_kv_release_seqs, tsv_kv_fork_seqs, ...
 *
 * shares [num_blocks] holds, for each block, the table entries that refer to it beyond the first: 0 for
 * a block of one sequence and for a free one, never negative.  It starts as zeros, and
 * tsv_kv_plan_slots, which takes and gives back blocks of one sequence, needs nothing of it.  Blocks that may be
 * shared go back with tsv_kv_release_seqs, before the plan sees the shorter length (blocks_held is then what is
 * left).  Only full blocks are shared, so a sequence never writes into a shared block unless it is cut back
 * into one; a sequence to be cut back there is forked and released instead.
 *
 * In these calls an output array may be its input array (seq_lens_out, blocks_held_out, shares_out,
 * free_count_out, block_table_out); with separate outputs, and no change in between, a repeated call gives
 * the same result.  Nothing else may overlap.  B <= 8192; block_size a power of two in [8, 128];
 * max_blocks * block_size and num_blocks up to 2^30.
 * ------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------
 * Forks: sequence fork_dst[i], which holds no blocks, becomes a copy of fork_src[i] (batch rows;
 * fork_src[i] < 0: padding).  With L = seq_lens[src]:
 *   entries 0 .. L / bs - 1 of the source's table row go into the destination's, and each such block's
 *   shares grow by one;
 *   if L % bs > 0, a block is taken from the top of the stack free_blocks[0 .. free_count), in
 *   order of i, into entry L / bs, and (copy_src, copy_dst, copy_rows)[i] = (the source's block, the
 *   new one, L % bs); otherwise (-1, -1, 0).  tsv_kv_copy_blocks does the copy, in each layer's cache;
 *   seq_lens_out[dst] = L, blocks_held_out[dst] = ceil(L / bs).  Other rows' entries are copied.
 * Surplus blocks of the source are not shared.  A source may be forked many times.
 * fork_err[i], overwritten: TSV_DERR_SEQ (an index outside the batch, a destination named twice or holding blocks),
 * TSV_DERR_CAPACITY (the source's length negative or past its blocks, its blocks_held outside [0, max_blocks]),
 * TSV_DERR_POOL (too few free blocks: no later fork that needs one gets one then; *free_count outside
 * [0, num_blocks]): the fork is not done.  TSV_DERR_BLOCK (a block id outside [0, num_blocks)): the
 * entry is copied as it is, and nothing is counted or copied for it.
 * F <= 8192 forks.
 * ------------------------------------------------------------------------- */
tsv_status tsv_kv_fork_seqs(const int32_t *fork_src, const int32_t *fork_dst, const int32_t *seq_lens,
                            int32_t *seq_lens_out, int32_t *block_table, const int32_t *blocks_held,
                            int32_t *blocks_held_out, const int32_t *shares, int32_t *shares_out,
                            const int32_t *free_blocks, const int32_t *free_count, int32_t *free_count_out,
                            int32_t *copy_src, int32_t *copy_dst, int32_t *copy_rows, int F, int B,
                            int block_size, int max_blocks, int num_blocks, int32_t *fork_err, void *stream);

/* ---------------------------------------------------------------------------
 * Blocks given back by reference: sequence b keeps the blocks of its first keep_lens[b] tokens (0: it has
 * ended; its length or more: only surplus blocks go).  Each entry ceil(keep / bs) .. blocks_held[b] - 1 takes
 * one from its block's shares; a block with no reference left goes onto the stack free_blocks, in
 * ascending order of ids after all entries of the batch are counted.  blocks_held_out[b] = entries kept; the
 * table keeps its values.
 * seq_err[b], overwritten: TSV_DERR_CAPACITY (keep_lens[b] < 0, blocks_held[b] outside [0, max_blocks]) and
 * TSV_DERR_POOL for *free_count outside [0, num_blocks]: nothing is given back.  TSV_DERR_BLOCK (a block id
 * outside [0, num_blocks)): that entry is dropped.  TSV_DERR_POOL also where more references of a block
 * come back than there were, or more blocks than the pool has places for (the rest is lost): the others are served.
 * ------------------------------------------------------------------------- */
tsv_status tsv_kv_release_seqs(const int32_t *keep_lens, const int32_t *block_table, const int32_t *blocks_held,
                               int32_t *blocks_held_out, const int32_t *shares, int32_t *shares_out,
                               int32_t *free_blocks, const int32_t *free_count, int32_t *free_count_out, int B,
                               int block_size, int max_blocks, int num_blocks, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * The blocks in use put together at the low end of the cache.  The n distinct blocks of the held
 * table entries are live -- so every block in use must be in this table --; the k-th live block with an id of
 * n or more moves to the k-th free id below n: copy_src[k] -> copy_dst[k] for k < *copy_count, and -1 from there
 * to num_blocks / 2, the places of both lists.  block_table_out and shares_out follow the moves (shares_out is 0
 * for free blocks); free_blocks[0 .. num_blocks - n) = num_blocks - 1 .. n, *free_count_out = num_blocks - n, so the
 * lowest free id is taken first.  tsv_kv_copy_blocks(..., copy_count) moves the rows, in each layer's cache; no
 * block is both source and destination.
 * seq_err[b], overwritten: TSV_DERR_CAPACITY (blocks_held[b] outside [0, max_blocks]: the row is copied as it is and
 * its blocks do not count as live), TSV_DERR_BLOCK (a block id outside [0, num_blocks): the entry stays).
 * `workspace` holds tsv_kv_compact_workspace_size(num_blocks) bytes, 4-byte aligned; calls that may overlap on the
 * GPU need one each.  max_blocks up to 2^27.
 * ------------------------------------------------------------------------- */
size_t tsv_kv_compact_workspace_size(int num_blocks);

tsv_status tsv_kv_compact_blocks(const int32_t *block_table, int32_t *block_table_out, const int32_t *blocks_held,
                                 const int32_t *shares, int32_t *shares_out, int32_t *free_blocks,
                                 int32_t *free_count_out, int32_t *copy_src, int32_t *copy_dst,
                                 int32_t *copy_count, int B, int max_blocks, int num_blocks, void *workspace,
                                 size_t workspace_bytes, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * Block contents copied within a cache: the first copy_rows[i] slots (NULL: all; held to [0, block_size]) of
 * block copy_src[i] of k_cache and v_cache go to block copy_dst[i], for i < n, or i < *copy_count if that
 * is not NULL (held to [0, n]).  copy_src[i] < 0: nothing.  Destinations must differ, and no
 * destination may be a source of another copy.  copy_err[i], overwritten: TSV_DERR_BLOCK for a source
 * >= num_blocks or a destination outside [0, num_blocks) (nothing is copied).  D in {64, 128}; caches
 * 16-byte aligned.
 * ------------------------------------------------------------------------- */
tsv_status tsv_kv_copy_blocks(void *k_cache, void *v_cache, const int32_t *copy_src, const int32_t *copy_dst,
                              const int32_t *copy_rows, const int32_t *copy_count, int n, int Hkv, int D,
                              int block_size, int num_blocks, tsv_dtype dtype, int32_t *copy_err, void *stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per sequence where groups of sequences share the first keys.
 *
 * Group g is the sequences group_offsets[g] .. group_offsets[g+1] - 1 (group_offsets[0] = 0, ascending,
 * group_offsets[G] = B; a group may be empty).  Its sequences attend to the same first P_g = prefix_lens[g]
 * keys, 0 <= P_g <= seq_lens[b], which are read from the table row of the group's first sequence, once for all
 * of them; keys P_g .. L_b - 1 come from each sequence's own row.  P_g need not be a multiple of the block size.  The
 * first sequence's row has to name the blocks of the P_g keys whatever its own length is: it may have ended (it is
 * flagged then, the others are not) while others of its group go on, as long as the shared blocks are held.
 * out and lse are those of tsv_decode_attn for tables with these keys, with the same precision: fp32 sums and weights (a bf16 call's
 * weights within 2^-15 of themselves), out rounded once.  A repeated call gives the same bits.
 * L_b = 0: out is zero and lse -infinity.  Slots outside a sequence's keys are never read into the result.
 * `workspace` as in tsv_tree_verify_attn, with tsv_prefix_decode_attn_workspace_size(...) bytes, 16-byte aligned; calls
 * that may overlap on the GPU need one each.  out and lse must not overlap the inputs.
 * seq_err[b]: TSV_DERR_SEQ (all sequences: the offsets are not as above), TSV_DERR_CAPACITY (L_b < 0 or
 * > max_blocks * block_size, P_g < 0 or > L_b), TSV_DERR_BLOCK (a block id that covers one of the sequence's keys,
 * the shared ones included, outside [0, num_blocks)), TSV_DERR_TIMEOUT (bf16: a wait gave up; a group's sequences
 * are told together, and those of other groups with them); rows of a flagged sequence are NaN.
 * D in {64, 128}; Hq % Hkv == 0; block_size a power of two in [8, 128]; B and G up to 8192;
 * max_blocks * block_size and num_blocks * block_size up to 2^30, B * Hq up to 2^24; scale > 0, scale * log2(e)
 * finite.
 * ------------------------------------------------------------------------- */
size_t tsv_prefix_decode_attn_workspace_size(int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks,
                                             tsv_dtype dtype);

tsv_status tsv_prefix_decode_attn(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_table, const int32_t *seq_lens,
                                  const int32_t *group_offsets, const int32_t *prefix_lens, void *out, float *lse,
                                  int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks,
                                  int num_blocks, float scale, tsv_dtype dtype, void *workspace,
                                  size_t workspace_bytes, int32_t *seq_err, void *stream);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens, with entropy and top alternatives.
 *
 * Row t of logits (row_stride elements after the one before, its V elements contiguous) gives
 * p = softmax(logits[t] / temperature):  logprobs[t] = ln p(tokens[t]);  entropy[t] = -sum p ln p (entropy may be
 * NULL);  top_ids, top_logprobs [T, top]: the `top` entries of largest logit, ties to the lower index, and
 * their ln p (both may be NULL if top = 0).  A logit of -infinity is an entry of probability 0.  Sums are fp32.
 * tokens[t] < 0 (padding): the row is not read; logprobs, entropy and top_logprobs are 0, top_ids -1.
 * tok_err[t], overwritten: TSV_DERR_TOKEN (tokens[t] >= V), TSV_DERR_NONFINITE (a NaN or +infinity, or no finite logit):
 * the row's floats are NaN and its ids -1.
 * logits fp32 or bf16, aligned to their elements; 0 <= top <= min(32, V); T up to 2^27, V up to 2^30;
 * temperature > 0, it and its inverse finite.
 * ------------------------------------------------------------------------- */
tsv_status tsv_token_logprobs(const void *logits, int64_t row_stride, const int32_t *tokens, int T, int V,
                              float temperature, int top, tsv_dtype logits_dtype, float *logprobs,
                              float *entropy, int32_t *top_ids, float *top_logprobs, int32_t *tok_err, void *stream);

/* ---------------------------------------------------------------------------
 * Tree construction (host side).  Sequoia summary, sections "Scalable Speculative
 * Decoding" and "Dynamic Programming": the tree of speculated tokens is built by
 * dynamic programming to an optimal shape; the figure of forward-pass time against
 * input length: the tree size trades the draft model's time against the target's
 * verification time (hardware-aware).  The pages state neither the objective nor the
 * recurrence; this library reads them as follows.
 *
 * accept[k], k = 0 .. K-1: probability that the (k+1)-th drafted sibling is the one
 * the walk accepts at a node it has reached (positional acceptance, the same at every
 * node; accept[k] >= 0, sum <= 1 + 1e-9); siblings of rank > K are never accepted.
 * A node is reached with the product of accept[rank - 1] over the edges of its root
 * path (rank = 1 + the number of earlier siblings), so the expected number of tokens
 * a verification step generates -- accepted drafts plus the bonus -- is
 *     E(tree) = sum over the tree's nodes of that product   (the root counts 1).
 *
 * These calls read and write HOST memory, run synchronously on the calling thread,
 * need no GPU, and use O(min(d_max, n_max) * min(K, n_max) * n_max) bytes of
 * temporary host memory.  Argument errors return TSV_ERR_ARG.
 * ------------------------------------------------------------------------- */

/* values[n * (d_max + 1) + d] = the largest E over trees of n nodes (root included)
 * and depth <= d (root at depth 0), for 1 <= n <= n_max, 0 <= d <= d_max; row n = 0
 * is 0, and -INFINITY where no tree exists (n > 1 with d = 0).
 * 1 <= n_max <= 128, d_max >= 0, K >= 1; values holds (n_max + 1) * (d_max + 1). */
tsv_status tsv_sequoia_values(const double *accept, int K, int n_max, int d_max, double *values);

/* One tree of n nodes and depth <= max_depth attaining the largest E: parent[0..n-1]
 * in breadth-first order with siblings by rank (parent[0] = -1, parent[i] < i, a
 * node's children have increasing indices in draft order, the order in which the walk
 * tries them); *expected = its E.  1 <= n <= 128; max_depth >= 1 unless n == 1. */
tsv_status tsv_sequoia_tree(const double *accept, int K, int n, int max_depth, int32_t *parent,
                            double *expected);

/* Hardware-aware size and depth: the (n, d) with 1 <= n <= n_max, 0 <= d <= d_max that
 * maximises  speedup(n, d) = E_best(n, d) * t_verify[1] / (t_verify[n] + d * t_draft),
 * where t_verify[n] > 0 is the time of one target forward over n tree tokens
 * (t_verify[1]: one incremental decoding step; t_verify[0] is not read) and
 * t_draft >= 0 the time of one draft forward, run once per tree level.  Ties go to
 * the smaller n, then the smaller d. */
tsv_status tsv_sequoia_plan(const double *accept, int K, int n_max, int d_max, const double *t_verify,
                            double t_draft, int *n_best, int *d_best, double *speedup);

/* Acceptance statistics for the planner, accumulated from verification outputs (HOST
 * copies of parent, accepted_nodes and accept_len, layouts as above).  For every
 * sequence with accept_len[b] >= 0 and every node on its accepted path
 * accepted_nodes[b, 0 .. accept_len[b]] -- the nodes the walk reached -- with c
 * children: reached[k] += 1 for every rank k + 1 <= min(c, K), and accepted[r - 1] += 1
 * when the path goes on to the child of rank r <= K.  Under the positional model above,
 * accepted[k] / reached[k] estimates accept[k].  The counts are added to the arrays
 * (int64 [K]), so steps can be accumulated; sequences with accept_len < 0 are skipped.
 * TSV_ERR_ARG for a parent array that is not a tree or a path that does not follow it. */
tsv_status tsv_sequoia_accept_counts(const int32_t *parent, const int32_t *accepted_nodes,
                                     const int32_t *accept_len, int B, int N, int K, int64_t *reached,
                                     int64_t *accepted);

#ifdef __cplusplus
}
#endif

#endif /* TSV_H */
