// serving_args.cuh -- arguments of the serving operators around the paged cache: the
// slot plan, the rotary K/V append and single-token attention.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace tsv {

constexpr int kPlanMaxSeqs = 8192;  // sequences of one slot plan (their scans live in shared memory)

struct PlanArgs {
    const int32_t* seq_lens;
    const int32_t* new_lens;
    const int32_t* parent;  // [B, N] or nullptr
    int32_t* block_table;
    const int32_t* held;
    int32_t* held_out;
    int32_t* free_blocks;  // [num_blocks]
    const int32_t* free_count;
    int32_t* free_count_out;
    int32_t* total_lens;
    int32_t* token_offsets;  // [B + 1]
    int64_t* slot_map;       // [max_tokens]
    int32_t* positions;      // [max_tokens]
    int32_t* seq_err;
    int B, N, bs_log2, max_blocks, num_blocks, max_tokens;
};
cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream);

constexpr int kRopeMaxPairs = 64;  // rotary pairs of a head (D <= 128)

struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* positions;  // [axes, T]
    const float* inv_freq;     // [R / 2]
    void* q_out;
    void* k_cache;
    void* v_cache;
    const int64_t* slot_map;  // [T]
    int32_t* tok_err;         // [T]
    long long q_stride, k_stride, v_stride, q_out_stride;  // elements from one token to the next
    long long slots;          // num_blocks * block_size
    int T, Hq, Hkv, D, R;
    int neighbours;           // pairs (2i, 2i + 1); 0: pairs (i, i + R / 2)
    uint8_t axis[kRopeMaxPairs];  // axis whose position a pair takes
};
cudaError_t launch_rope_append(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream);

// Plan of a single-token attention call: a deterministic function of the shapes and the
// SM count (the workspace query and the call must agree).
struct DecodePlan {
    int rows;     // query rows one unit covers (of one kv head)
    int groups;   // row groups per kv head
    int team;     // warps that go through the same keys, each with a unit of its own
    int lanes;    // teams the key tiles are divided between
    bool by_unit; // the join has a record per unit (they are fewer than the warps), else per warp
    size_t ws_bytes;
};
DecodePlan make_decode_plan(int B, int Hq, int Hkv, int D, int block_size, int max_blocks, bool bf16, int num_sms);

struct DecodeArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    void* out;
    float* lse;  // [B, Hq] or nullptr
    int32_t* seq_err;
    // pieces of units, two slots a warp (warp = lane * team + member)
    float* part_o;  // [2 * warps][rows][D]
    float* part_m;  // [2 * warps][rows]
    float* part_l;  // [2 * warps][rows]
    int4* split;    // [warps]: sequence, unit, last lane (-1: in one piece) and first slot of a unit in pieces
    int* part_bad;  // [2 * warps]
    int B, Hq, Hkv, D, G, rows, groups, team, lanes, by_unit;
    int bs_log2, max_blocks, num_blocks;
    float scale_log2;  // scale * log2(e)
};
cudaError_t launch_decode_attn(const DecodeArgs& a, bool bf16, cudaStream_t stream);

}  // namespace tsv
