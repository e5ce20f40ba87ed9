// serving_api.cu -- the C entries of the serving operators (slot plan, rotary K/V append,
// single-token attention): host-side argument checks, launch planning and dispatch.  No
// allocation, no host synchronisation.
#include <cmath>

#include "../common.cuh"
#include "serving_args.cuh"
#include "serving_checks.cuh"

namespace {
tsv_status check_decode_shapes(int B, int Hq, int Hkv, int D, int block_size, int max_blocks, int num_blocks, tsv_dtype dtype) {
    if (B < 0 || Hq < 1 || max_blocks < 1) return report_error(TSV_ERR_ARG, "bad sizes B=%d Hq=%d max_blocks=%d", B, Hq, max_blocks);
    const tsv_status st = check_cache_shape(Hkv, D, block_size, num_blocks, dtype);
    if (st != TSV_OK) return st;
    if (Hq % Hkv) return report_error(TSV_ERR_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
    if ((long long)max_blocks * block_size > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "a table row covers more than 2^30 slots");
    if ((long long)B * Hq > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "B * Hq exceeds 2^30 query rows");
    return check_row(Hq, D);
}
}  // namespace

extern "C" {

tsv_status tsv_kv_plan_slots(const int32_t* seq_lens, const int32_t* new_lens, const int32_t* parent,
                             int32_t* block_table, const int32_t* blocks_held, int32_t* blocks_held_out,
                             int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
                             int32_t* total_lens, int32_t* token_offsets, int64_t* slot_map, int32_t* positions,
                             int B, int N, int block_size, int max_blocks, int num_blocks, int max_tokens,
                             int32_t* seq_err, void* stream) {
    if (B < 0 || max_blocks < 1 || num_blocks < 1 || max_tokens < 0)
        return report_error(TSV_ERR_ARG, "bad sizes B=%d max_blocks=%d num_blocks=%d max_tokens=%d", B, max_blocks, num_blocks, max_tokens);
    if (B > tsv::kPlanMaxSeqs) return report_error(TSV_ERR_UNSUPPORTED, "B=%d exceeds %d sequences", B, tsv::kPlanMaxSeqs);
    if (!pow2_in(block_size, 8, 128)) return report_error(TSV_ERR_UNSUPPORTED, "block_size %d not a power of two in [8,128]", block_size);
    if ((long long)max_blocks * block_size > (1LL << 30)) return report_error(TSV_ERR_UNSUPPORTED, "a table row covers more than 2^30 slots");
    if (max_tokens > (1 << 30) || num_blocks > (1 << 30))
        return report_error(TSV_ERR_UNSUPPORTED, "max_tokens=%d or num_blocks=%d exceeds 2^30", max_tokens, num_blocks);
    if (parent != nullptr && N < 1) return report_error(TSV_ERR_ARG, "bad size N=%d", N);
    if (parent != nullptr && N > tsv::kMaxNodes) return report_error(TSV_ERR_UNSUPPORTED, "N=%d exceeds %d tree nodes", N, tsv::kMaxNodes);
    // an empty batch has no per-sequence arrays; with none of the others either there is nothing to write
    if (B == 0 && !free_count && !free_count_out && !token_offsets && !slot_map && !positions) return TSV_OK;
    const bool per_seq = seq_lens && new_lens && block_table && blocks_held && blocks_held_out && free_blocks && total_lens && seq_err;
    if ((B > 0 && !per_seq) || !free_count || !free_count_out || !token_offsets || (max_tokens > 0 && (!slot_map || !positions)))
        return report_error(TSV_ERR_ARG, "null array argument");
    tsv::PlanArgs a{};
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.parent = parent;
    a.block_table = block_table;
    a.held = blocks_held;
    a.held_out = blocks_held_out;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.total_lens = total_lens;
    a.token_offsets = token_offsets;
    a.slot_map = slot_map;
    a.positions = positions;
    a.seq_err = seq_err;
    a.B = B;
    a.N = N;
    a.bs_log2 = log2i(block_size);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.max_tokens = max_tokens;
    const cudaError_t e = tsv::launch_kv_plan(a, static_cast<cudaStream_t>(stream));
    return launch_status(e, "kv_plan_slots");
}

tsv_status tsv_rope_kv_append(const void* q, const void* k, const void* v, const int32_t* positions,
                              const float* inv_freq, void* q_out, void* k_cache, void* v_cache,
                              const int64_t* slot_map, int T, int Hq, int Hkv, int D, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int64_t q_out_stride, int block_size, int num_blocks,
                              tsv_dtype dtype, const tsv_rope_options* opts, int32_t* tok_err, void* stream) {
    if (T < 0 || Hq < 1) return report_error(TSV_ERR_ARG, "bad sizes T=%d Hq=%d", T, Hq);
    tsv_status st = check_cache_shape(Hkv, D, block_size, num_blocks, dtype);
    if (st == TSV_OK) st = check_row(Hq > Hkv ? Hq : Hkv, D);
    if (st != TSV_OK) return st;
    if (T > (1 << 30)) return report_error(TSV_ERR_UNSUPPORTED, "T=%d exceeds 2^30", T);
    const tsv_rope_options o = opts ? *opts : tsv_rope_options{D, 0, 1, 0, {D / 2, 0, 0, 0}};
    if (o.rotary_dim < 16 || o.rotary_dim > D || o.rotary_dim % 16)
        return report_error(TSV_ERR_UNSUPPORTED, "rotary_dim %d not a multiple of 16 in [16, %d]", o.rotary_dim, D);
    if ((o.neighbours != 0 && o.neighbours != 1) || (o.rounds != 0 && o.rounds != 1))
        return report_error(TSV_ERR_ARG, "neighbours and rounds must be 0 or 1");
    if (o.axes < 1 || o.axes > 4) return report_error(TSV_ERR_ARG, "axes must be 1 to 4, not %d", o.axes);
    int left[4] = {0, 0, 0, 0};
    long long pairs = 0;
    for (int i = 0; i < o.axes; ++i) {
        if (o.sections[i] < 0) return report_error(TSV_ERR_ARG, "section %d is negative", i);
        left[i] = o.sections[i];
        pairs += o.sections[i];
    }
    if (pairs != o.rotary_dim / 2)
        return report_error(TSV_ERR_ARG, "the sections hold %lld pairs, rotary_dim has %d", pairs, o.rotary_dim / 2);
    const long long esz = dtype == TSV_F32 ? 4 : 2, vec = 16 / esz;
    if (q_stride < (long long)Hq * D || k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D || q_out_stride < (long long)Hq * D)
        return report_error(TSV_ERR_ARG, "a token stride is smaller than its row");
    if (q_stride % vec || k_stride % vec || v_stride % vec || q_out_stride % vec)
        return report_error(TSV_ERR_ARG, "token strides must be multiples of 16 bytes");
    if (T == 0) return TSV_OK;
    if (!q || !k || !v || !positions || !inv_freq || !q_out || !k_cache || !v_cache || !slot_map || !tok_err)
        return report_error(TSV_ERR_ARG, "null array argument");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache))
        return report_error(TSV_ERR_ARG, "q, k, v, q_out and the caches must be 16-byte aligned");
    if (q == q_out && q_stride != q_out_stride) return report_error(TSV_ERR_ARG, "in place, q and q_out need the same stride");
    tsv::RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.slot_map = slot_map;
    a.tok_err = tok_err;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.slots = (long long)num_blocks * block_size;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.R = o.rotary_dim;
    a.neighbours = o.neighbours;
    // axis of each pair: section after section, or in rounds over the axes that have pairs left
    for (int p = 0, ax = 0; p < o.rotary_dim / 2; ++p) {
        while (left[ax] == 0) ax = (ax + 1) % o.axes;
        a.axis[p] = static_cast<uint8_t>(ax);
        --left[ax];
        if (o.rounds) ax = (ax + 1) % o.axes;
    }
    const cudaError_t e = tsv::launch_rope_append(a, dtype == TSV_BF16, device_sms(), static_cast<cudaStream_t>(stream));
    return launch_status(e, "rope_kv_append");
}

size_t tsv_decode_attn_workspace_size(int B, int Hq, int Hkv, int D, int block_size, int max_blocks, tsv_dtype dtype) {
    if (check_decode_shapes(B, Hq, Hkv, D, block_size, max_blocks, 1, dtype) != TSV_OK || B == 0) return 0;
    return tsv::make_decode_plan(B, Hq, Hkv, D, block_size, max_blocks, dtype == TSV_BF16, device_sms()).ws_bytes;
}

tsv_status tsv_decode_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                           const int32_t* seq_lens, void* out, float* lse, int B, int Hq, int Hkv, int D,
                           int block_size, int max_blocks, int num_blocks, float scale, tsv_dtype dtype,
                           void* workspace, size_t workspace_bytes, int32_t* seq_err, void* stream) {
    const tsv_status st = check_decode_shapes(B, Hq, Hkv, D, block_size, max_blocks, num_blocks, dtype);
    if (st != TSV_OK) return st;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!(scale > 0.0f) || !std::isfinite(scale_log2)) return report_error(TSV_ERR_ARG, "scale must be positive, and finite times log2(e)");
    if (B == 0) return TSV_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !seq_err)
        return report_error(TSV_ERR_ARG, "null array argument");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return report_error(TSV_ERR_ARG, "q, caches and out must be 16-byte aligned");
    const tsv::DecodePlan p = tsv::make_decode_plan(B, Hq, Hkv, D, block_size, max_blocks, dtype == TSV_BF16, device_sms());
    if (p.ws_bytes > 0 && (workspace == nullptr || workspace_bytes < p.ws_bytes))
        return report_error(TSV_ERR_ARG, "workspace of %zu bytes needed, %zu given", p.ws_bytes, workspace_bytes);
    if (p.ws_bytes > 0 && !aligned16(workspace)) return report_error(TSV_ERR_ARG, "workspace must be 16-byte aligned");
    tsv::DecodeArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = out;
    a.lse = lse;
    a.seq_err = seq_err;
    const size_t warps = (size_t)p.lanes * p.team, rows = 2 * warps * p.rows;
    a.split = static_cast<int4*>(workspace);
    a.part_o = reinterpret_cast<float*>(a.split + warps);
    a.part_m = a.part_o + rows * D;
    a.part_l = a.part_m + rows;
    a.part_bad = reinterpret_cast<int*>(a.part_l + rows);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.G = Hq / Hkv;
    a.rows = p.rows;
    a.groups = p.groups;
    a.team = p.team;
    a.by_unit = p.by_unit;
    a.lanes = p.lanes;
    a.bs_log2 = log2i(block_size);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale_log2;
    const cudaError_t e = tsv::launch_decode_attn(a, dtype == TSV_BF16, static_cast<cudaStream_t>(stream));
    return launch_status(e, "decode_attn");
}

}  // extern "C"
