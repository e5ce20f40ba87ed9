// continue_api.cu -- the C entries of the operators for several continuations of one prompt (cache
// blocks by reference, attention over shared prefixes, token log probabilities): host-side argument
// checks, launch planning and dispatch.  No allocation, no host synchronisation.
#include <cmath>

#include "../common.cuh"
#include "continue_args.cuh"
#include "serving_checks.cuh"

namespace {

tsv_status check_table(int B, int block_size, int max_blocks, int num_blocks) {
    if (B < 0 || max_blocks < 1 || num_blocks < 1)
        return report_error(TSV_ERR_ARG, "bad sizes B=%d max_blocks=%d num_blocks=%d", B, max_blocks, num_blocks);
    if (B > tsv::kPagesMaxSeqs) return report_error(TSV_ERR_UNSUPPORTED, "B=%d exceeds %d sequences", B, tsv::kPagesMaxSeqs);
    if (!pow2_in(block_size, 8, 128)) return report_error(TSV_ERR_UNSUPPORTED, "block_size %d not a power of two in [8,128]", block_size);
    if ((long long)max_blocks * block_size > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "a table row covers more than 2^30 slots");
    if (num_blocks > (1 << 30)) return report_error(TSV_ERR_UNSUPPORTED, "num_blocks=%d exceeds 2^30", num_blocks);
    return TSV_OK;
}

tsv_status check_prefix_shapes(int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks, int num_blocks, tsv_dtype dtype) {
    if (B < 0 || G < 0 || Hq < 1 || max_blocks < 1) return report_error(TSV_ERR_ARG, "bad sizes B=%d G=%d Hq=%d max_blocks=%d", B, G, Hq, max_blocks);
    tsv_status st = check_cache_shape(Hkv, D, block_size, num_blocks, dtype);
    if (st != TSV_OK) return st;
    if (Hq % Hkv) return report_error(TSV_ERR_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
    if (B > tsv::kPagesMaxSeqs || G > tsv::kPagesMaxSeqs)
        return report_error(TSV_ERR_UNSUPPORTED, "B=%d or G=%d exceeds %d", B, G, tsv::kPagesMaxSeqs);
    if (B > 0 && G == 0) return report_error(TSV_ERR_ARG, "%d sequences in no group", B);
    if ((long long)max_blocks * block_size > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "a table row covers more than 2^30 slots");
    // (rows of the cache are 32-bit coordinates of its tensor map)
    if ((long long)num_blocks * block_size > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "the cache has more than 2^30 slots");
    if ((long long)B * Hq > (1LL << 24)) return report_error(TSV_ERR_UNSUPPORTED, "B * Hq exceeds 2^24 query rows");
    return check_row(Hq, D);
}

}  // namespace

extern "C" {

tsv_status tsv_kv_fork_seqs(const int32_t* fork_src, const int32_t* fork_dst, const int32_t* seq_lens, int32_t* seq_lens_out,
                            int32_t* block_table, const int32_t* blocks_held, int32_t* blocks_held_out, const int32_t* shares,
                            int32_t* shares_out, const int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
                            int32_t* copy_src, int32_t* copy_dst, int32_t* copy_rows, int F, int B, int block_size, int max_blocks,
                            int num_blocks, int32_t* fork_err, void* stream) {
    if (F < 0) return report_error(TSV_ERR_ARG, "bad size F=%d", F);
    const tsv_status st = check_table(B, block_size, max_blocks, num_blocks);
    if (st != TSV_OK) return st;
    if (F > tsv::kPagesMaxForks) return report_error(TSV_ERR_UNSUPPORTED, "F=%d exceeds %d forks", F, tsv::kPagesMaxForks);
    if ((F > 0 && (!fork_src || !fork_dst || !copy_src || !copy_dst || !copy_rows || !fork_err)) ||
        (B > 0 && (!seq_lens || !seq_lens_out || !block_table || !blocks_held || !blocks_held_out)) || !shares || !shares_out ||
        !free_blocks || !free_count || !free_count_out)
        return report_error(TSV_ERR_ARG, "null array argument");
    tsv::ForkArgs a{};
    a.fork_src = fork_src;
    a.fork_dst = fork_dst;
    a.seq_lens = seq_lens;
    a.seq_lens_out = seq_lens_out;
    a.block_table = block_table;
    a.held = blocks_held;
    a.held_out = blocks_held_out;
    a.shares = shares;
    a.shares_out = shares_out;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.copy_rows = copy_rows;
    a.fork_err = fork_err;
    a.F = F;
    a.B = B;
    a.bs_log2 = log2i(block_size);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    return launch_status(tsv::launch_kv_fork(a, device_sms(), static_cast<cudaStream_t>(stream)), "kv_fork_seqs");
}

tsv_status tsv_kv_release_seqs(const int32_t* keep_lens, const int32_t* block_table, const int32_t* blocks_held,
                               int32_t* blocks_held_out, const int32_t* shares, int32_t* shares_out, int32_t* free_blocks,
                               const int32_t* free_count, int32_t* free_count_out, int B, int block_size, int max_blocks,
                               int num_blocks, int32_t* seq_err, void* stream) {
    const tsv_status st = check_table(B, block_size, max_blocks, num_blocks);
    if (st != TSV_OK) return st;
    if ((B > 0 && (!keep_lens || !block_table || !blocks_held || !blocks_held_out || !seq_err)) || !shares || !shares_out || !free_blocks ||
        !free_count || !free_count_out)
        return report_error(TSV_ERR_ARG, "null array argument");
    tsv::ReleaseArgs a{};
    a.keep_lens = keep_lens;
    a.block_table = block_table;
    a.held = blocks_held;
    a.held_out = blocks_held_out;
    a.shares = shares;
    a.shares_out = shares_out;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.seq_err = seq_err;
    a.B = B;
    a.bs_log2 = log2i(block_size);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    return launch_status(tsv::launch_kv_release(a, device_sms(), static_cast<cudaStream_t>(stream)), "kv_release_seqs");
}

size_t tsv_kv_compact_workspace_size(int num_blocks) { return num_blocks < 1 ? 0 : (size_t)num_blocks * sizeof(int32_t); }

tsv_status tsv_kv_compact_blocks(const int32_t* block_table, int32_t* block_table_out, const int32_t* blocks_held, const int32_t* shares,
                                 int32_t* shares_out, int32_t* free_blocks, int32_t* free_count_out, int32_t* copy_src,
                                 int32_t* copy_dst, int32_t* copy_count, int B, int max_blocks, int num_blocks, void* workspace,
                                 size_t workspace_bytes, int32_t* seq_err, void* stream) {
    const tsv_status st = check_table(B, 8, max_blocks, num_blocks);
    if (st != TSV_OK) return st;
    if ((B > 0 && (!block_table || !block_table_out || !blocks_held || !seq_err)) || !shares || !shares_out || !free_blocks ||
        !free_count_out || !copy_count || (num_blocks > 1 && (!copy_src || !copy_dst)))
        return report_error(TSV_ERR_ARG, "null array argument");
    const size_t need = tsv_kv_compact_workspace_size(num_blocks);
    if (workspace == nullptr || workspace_bytes < need)
        return report_error(TSV_ERR_ARG, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 3) return report_error(TSV_ERR_ARG, "workspace must be 4-byte aligned");
    tsv::CompactBlocksArgs a{};
    a.block_table = block_table;
    a.block_table_out = block_table_out;
    a.held = blocks_held;
    a.shares = shares;
    a.shares_out = shares_out;
    a.free_blocks = free_blocks;
    a.free_count_out = free_count_out;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.copy_count = copy_count;
    a.remap = static_cast<int32_t*>(workspace);
    a.seq_err = seq_err;
    a.B = B;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    return launch_status(tsv::launch_kv_compact_blocks(a, device_sms(), static_cast<cudaStream_t>(stream)), "kv_compact_blocks");
}

tsv_status tsv_kv_copy_blocks(void* k_cache, void* v_cache, const int32_t* copy_src, const int32_t* copy_dst, const int32_t* copy_rows,
                              const int32_t* copy_count, int n, int Hkv, int D, int block_size, int num_blocks, tsv_dtype dtype,
                              int32_t* copy_err, void* stream) {
    if (n < 0) return report_error(TSV_ERR_ARG, "bad size n=%d", n);
    tsv_status st = check_cache_shape(Hkv, D, block_size, num_blocks, dtype);
    if (st == TSV_OK) st = check_row(Hkv, D);
    if (st != TSV_OK) return st;
    if (n > (1 << 30)) return report_error(TSV_ERR_UNSUPPORTED, "n=%d exceeds 2^30", n);
    if (n == 0) return TSV_OK;
    if (!k_cache || !v_cache || !copy_src || !copy_dst || !copy_err) return report_error(TSV_ERR_ARG, "null array argument");
    if (!aligned16(k_cache) || !aligned16(v_cache)) return report_error(TSV_ERR_ARG, "the caches must be 16-byte aligned");
    tsv::CopyArgs a{};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.copy_rows = copy_rows;
    a.copy_count = copy_count;
    a.copy_err = copy_err;
    a.n = n;
    a.bs = block_size;
    a.row_vecs = static_cast<int>((long long)Hkv * D * (dtype == TSV_F32 ? 4 : 2) / 16);
    a.num_blocks = num_blocks;
    return launch_status(tsv::launch_kv_copy(a, device_sms(), static_cast<cudaStream_t>(stream)), "kv_copy_blocks");
}

size_t tsv_prefix_decode_attn_workspace_size(int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks, tsv_dtype dtype) {
    if (check_prefix_shapes(B, G, Hq, Hkv, D, block_size, max_blocks, 1, dtype) != TSV_OK || B == 0) return 0;
    return tsv::make_prefix_plan(B, G, Hq, Hkv, D, block_size, max_blocks, dtype == TSV_BF16, device_sms()).ws_bytes;
}

tsv_status tsv_prefix_decode_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* group_offsets, const int32_t* prefix_lens, void* out,
                                  float* lse, int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks, int num_blocks,
                                  float scale, tsv_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* seq_err,
                                  void* stream) {
    const tsv_status st = check_prefix_shapes(B, G, Hq, Hkv, D, block_size, max_blocks, num_blocks, dtype);
    if (st != TSV_OK) return st;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!(scale > 0.0f) || !std::isfinite(scale_log2)) return report_error(TSV_ERR_ARG, "scale must be positive, and finite times log2(e)");
    if (B == 0) return TSV_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !group_offsets || !prefix_lens || !out || !seq_err)
        return report_error(TSV_ERR_ARG, "null array argument");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return report_error(TSV_ERR_ARG, "q, caches and out must be 16-byte aligned");
    const tsv::PrefixPlan p = tsv::make_prefix_plan(B, G, Hq, Hkv, D, block_size, max_blocks, dtype == TSV_BF16, device_sms());
    if (workspace == nullptr || workspace_bytes < p.ws_bytes)
        return report_error(TSV_ERR_ARG, "workspace of %zu bytes needed, %zu given", p.ws_bytes, workspace_bytes);
    if (!aligned16(workspace)) return report_error(TSV_ERR_ARG, "workspace must be 16-byte aligned");
    char* ws = static_cast<char*>(workspace);
    tsv::PrefixArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.group_offsets = group_offsets;
    a.prefix_lens = prefix_lens;
    a.out = out;
    a.lse = lse;
    a.seq_err = seq_err;
    a.start = reinterpret_cast<long long*>(ws);
    a.item = reinterpret_cast<int4*>(ws + p.item);
    a.group = reinterpret_cast<int*>(ws + p.group);
    a.part_o = reinterpret_cast<float*>(ws + p.part_o);
    a.part_m = reinterpret_cast<float*>(ws + p.part_m);
    a.part_l = reinterpret_cast<float*>(ws + p.part_l);
    a.whole_o = reinterpret_cast<float*>(ws + p.whole_o);
    a.whole_m = reinterpret_cast<float*>(ws + p.whole_m);
    a.whole_l = reinterpret_cast<float*>(ws + p.whole_l);
    a.used = reinterpret_cast<int2*>(ws + p.used);
    a.begin = reinterpret_cast<int4*>(ws + p.begin);
    a.tc_begin = reinterpret_cast<int4*>(ws + p.tc_begin);
    a.tc_start = reinterpret_cast<long long*>(ws + p.tc_start);
    a.tc_o = reinterpret_cast<float*>(ws + p.tc_o);
    a.tc_m = reinterpret_cast<float*>(ws + p.tc_m);
    a.tc_l = reinterpret_cast<float*>(ws + p.tc_l);
    a.tc_lanes = p.tc_lanes;
    a.B = B;
    a.G = G;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.gq = Hq / Hkv;
    a.rows = p.rows;
    a.team = p.team;
    a.lanes = p.lanes;
    a.bs_log2 = log2i(block_size);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale_log2;
    return launch_status(tsv::launch_prefix_attn(a, dtype == TSV_BF16, static_cast<cudaStream_t>(stream)), "prefix_decode_attn");
}

tsv_status tsv_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens, int T, int V, float temperature, int top,
                              tsv_dtype logits_dtype, float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                              int32_t* tok_err, void* stream) {
    if (T < 0 || V < 1 || top < 0) return report_error(TSV_ERR_ARG, "bad sizes T=%d V=%d top=%d", T, V, top);
    if (T > (1 << 27) || V > (1 << 30)) return report_error(TSV_ERR_UNSUPPORTED, "T=%d exceeds 2^27 or V=%d exceeds 2^30", T, V);
    if (top > tsv::kMaxTop) return report_error(TSV_ERR_UNSUPPORTED, "top=%d exceeds %d alternatives", top, tsv::kMaxTop);
    if (top > V) return report_error(TSV_ERR_ARG, "%d alternatives of %d entries", top, V);
    if (logits_dtype != TSV_BF16 && logits_dtype != TSV_F32) return report_error(TSV_ERR_ARG, "bad dtype %d", (int)logits_dtype);
    if (row_stride < V) return report_error(TSV_ERR_ARG, "the row stride is smaller than a row");
    const float inv_t = 1.0f / temperature;
    if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(inv_t * 1.4426950408889634f) || !(inv_t > 0.0f))
        return report_error(TSV_ERR_ARG, "temperature must be positive and finite, and its inverse too");
    if (T == 0) return TSV_OK;
    if (!logits || !tokens || !logprobs || !tok_err || (top > 0 && (!top_ids || !top_logprobs)))
        return report_error(TSV_ERR_ARG, "null array argument");
    if (reinterpret_cast<uintptr_t>(logits) % (logits_dtype == TSV_F32 ? 4 : 2))
        return report_error(TSV_ERR_ARG, "logits must be aligned to their elements");
    tsv::LogprobArgs a{};
    a.logits = logits;
    a.stride = row_stride;
    a.tokens = tokens;
    a.logprob = logprobs;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.tok_err = tok_err;
    a.T = T;
    a.V = V;
    a.top = top;
    a.inv_t = inv_t;
    return launch_status(tsv::launch_token_logprobs(a, logits_dtype == TSV_BF16, device_sms(), static_cast<cudaStream_t>(stream)), "token_logprobs");
}

}  // extern "C"
