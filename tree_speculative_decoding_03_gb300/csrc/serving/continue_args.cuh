// continue_args.cuh -- arguments of the operators for several continuations of one prompt: cache
// blocks by reference, attention over a shared prefix, token log probabilities.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace tsv {

constexpr int kPagesMaxSeqs = 8192;   // sequences of a call (the forks' claims live in shared memory)
constexpr int kPagesMaxForks = 8192;  // forks of a call

struct ForkArgs {
    const int32_t* fork_src;  // [F]
    const int32_t* fork_dst;  // [F]
    const int32_t* seq_lens;
    int32_t* seq_lens_out;
    int32_t* block_table;
    const int32_t* held;
    int32_t* held_out;
    const int32_t* shares;  // [num_blocks]
    int32_t* shares_out;
    const int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* free_count_out;
    int32_t* copy_src;  // [F]
    int32_t* copy_dst;
    int32_t* copy_rows;
    int32_t* fork_err;  // [F]
    int F, B, bs_log2, max_blocks, num_blocks;
};
cudaError_t launch_kv_fork(const ForkArgs& a, int num_sms, cudaStream_t stream);

struct ReleaseArgs {
    const int32_t* keep_lens;
    const int32_t* block_table;
    const int32_t* held;
    int32_t* held_out;
    const int32_t* shares;
    int32_t* shares_out;
    int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* free_count_out;
    int32_t* seq_err;
    int B, bs_log2, max_blocks, num_blocks;
};
cudaError_t launch_kv_release(const ReleaseArgs& a, int num_sms, cudaStream_t stream);

struct CompactBlocksArgs {
    const int32_t* block_table;
    int32_t* block_table_out;
    const int32_t* held;
    const int32_t* shares;
    int32_t* shares_out;
    int32_t* free_blocks;
    int32_t* free_count_out;
    int32_t* copy_src;  // [num_blocks / 2]
    int32_t* copy_dst;
    int32_t* copy_count;
    int32_t* remap;  // workspace: [num_blocks]
    int32_t* seq_err;
    int B, max_blocks, num_blocks;
};
cudaError_t launch_kv_compact_blocks(const CompactBlocksArgs& a, int num_sms, cudaStream_t stream);

struct CopyArgs {
    void* k_cache;
    void* v_cache;
    const int32_t* copy_src;  // [n]
    const int32_t* copy_dst;
    const int32_t* copy_rows;   // [n] or nullptr: whole blocks
    const int32_t* copy_count;  // one int or nullptr: n
    int32_t* copy_err;
    int n, bs, row_vecs, num_blocks;  // row_vecs: 16-byte vectors of a slot (all heads)
};
cudaError_t launch_kv_copy(const CopyArgs& a, int num_sms, cudaStream_t stream);

constexpr int kPrefixTcKeys = 128;  // keys of a tile of the tensor-core kernel
constexpr int kPrefixTcRows = 256;  // query rows of a unit there

// Attention over shared prefixes.  Plan: a deterministic function of the shapes and the SM count.
struct PrefixPlan {
    int rows;   // query rows of a unit of the stream
    int team;   // warps that go through the same keys, each with a kv head of its own
    int lanes;  // teams the key tiles are divided between
    int tc_lanes;  // CTAs of the bf16 kernel (0: fp32), first those of the prefixes' tiles, then those of the stream
    // byte offsets of the workspace's parts, and its size
    size_t item, group, part_o, part_m, part_l, whole_o, whole_m, whole_l, used, begin, tc_begin, tc_start, tc_o, tc_m, tc_l, ws_bytes;
};
PrefixPlan make_prefix_plan(int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks, bool bf16, int num_sms);

struct PrefixArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* group_offsets;  // [G + 1]
    const int32_t* prefix_lens;    // [G]
    void* out;
    float* lse;  // [B, Hq] or nullptr
    int32_t* seq_err;
    // An item is a run of keys with the query rows that attend to it: the prefix of group i (i < G), or
    // what sequence i - G has of its own.
    long long* start;  // [G + B + 1]: running sums of the items' tiles, over all their units
    int4* item;        // [G + B]: first sequence (whose table holds the keys), first key, end, query rows
    int* group;        // [B]: the sequence's group
    float* part_o;     // [2 * warps][rows][D]: pieces of units, two slots a warp (warp = lane * team + member)
    float* part_m;
    float* part_l;
    float* whole_o;  // [3][B * Hq][D]: units in one piece: prefixes, the sequences' own keys, prefixes' odd tiles
    float* whole_m;
    float* whole_l;
    int2* used;           // lanes and tensor-core CTAs that have tiles
    int4* begin;          // [lanes][3]: where a lane's tiles begin: item, chunk, run of heads, tile; the item; their number
    int4* tc_begin;       // [tc_lanes][2]: group, unit, tile, number of tiles; the group's item.  No tiles: the first of its
                          // warps of the stream and their number, -, 0
    long long* tc_start;  // [G + 1]: running sums of the prefixes' tiles on the tensor cores
    float* tc_o;          // [4 * tc_lanes][128][D]: pieces there; a CTA's first and last unit, two streams each
    float* tc_m;
    float* tc_l;
    int B, G, Hq, Hkv, D, gq, rows, team, lanes, tc_lanes;  // gq = Hq / Hkv
    int bs_log2, max_blocks, num_blocks;
    float scale_log2;  // scale * log2(e)
};
cudaError_t launch_prefix_tc(const PrefixArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_attn(const PrefixArgs& a, bool bf16, cudaStream_t stream);

constexpr int kMaxTop = 32;  // alternatives of a row

struct LogprobArgs {
    const void* logits;
    long long stride;  // elements from one row to the next
    const int32_t* tokens;
    float* logprob;
    float* entropy;       // or nullptr
    int32_t* top_ids;     // [T, top]
    float* top_logprobs;  // [T, top]
    int32_t* tok_err;
    int T, V, top;
    float inv_t;  // 1 / temperature
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, bool bf16, int num_sms, cudaStream_t stream);

}  // namespace tsv
