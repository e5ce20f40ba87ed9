// pages.cu -- cache blocks that several sequences share: sequences forked, blocks released by
// reference, the cache put together at its low end, block contents copied.
//
// shares[i] counts the table entries of block i beyond its first: 0 for a block of one sequence and
// for a free one.  (A count of all entries would have to be set where blocks are taken, in the
// slot plan too; this one is right for every block that the plan takes or gives back.)
//
// All but the copy are integers: chains of latencies (launch, lengths, scan, ids) over a few hundred
// KB of tables, not bytes.  Places in the pool and in the copy lists are prefix sums in an order that
// the arguments fix (forks in order, ids ascending), and the only atomics are counts and error
// bits, whose result does not depend on their order.
#include <cooperative_groups.h>

#include "../common.cuh"
#include "continue_args.cuh"

namespace tsv {
namespace {
namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kFatal = TSV_DERR_SEQ | TSV_DERR_CAPACITY | TSV_DERR_POOL;  // errors that leave a fork undone

__device__ __forceinline__ int cdiv_shift(int x, int s) { return (x >> s) + ((x & ((1 << s) - 1)) != 0); }

// The sum over the block's threads before this one; *total: over all.  1024 threads.
__device__ __forceinline__ int block_scan(int x, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // s_warp of the last scan has been read
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return incl - x + (warp ? before : 0);
}

// ------------------------------------------------------------------ fork

// Fork i, by the threads first, first + step, ...: the source's full blocks go into the destination's row, a
// reference each.
__device__ __forceinline__ void fork_row(const ForkArgs& a, int i, int first, int step) {
    const int src = a.fork_src[i];
    if (src < 0 || (__ldcg(a.fork_err + i) & kFatal)) return;
    const int dst = a.fork_dst[i], full = __ldcg(a.seq_lens_out + dst) >> a.bs_log2;
    const int32_t* from = a.block_table + (long long)src * a.max_blocks;
    int32_t* to = a.block_table + (long long)dst * a.max_blocks;
    constexpr int U = 4;
    bool bad = false;
    for (int j0 = first; j0 < full; j0 += U * step) {
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = j0 + u * step < full ? from[j0 + u * step] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * step;
            if (j >= full || !TSV_IN_BOUNDS(j, a.max_blocks, a.fork_err + i)) continue;
            to[j] = id[u];
            if (id[u] >= 0 && id[u] < a.num_blocks)
                atomicAdd(a.shares_out + id[u], 1);
            else
                bad = true;
        }
    }
    if (bad) atomicOr(a.fork_err + i, TSV_DERR_BLOCK);
}

// CTA 0 checks the forks, gives each its fresh block and writes the lists; the others copy the
// shares when the result is another array.  Small calls have one CTA for it all, the rows too (7 forks of
// 2053 tokens and their copy: 7.3 -> 6.2 us).
constexpr int kForkSmallIds = 16384, kForkSmallEntries = 32768;  // block ids, and table entries of all forks, up to which
__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(const __grid_constant__ ForkArgs a, int alone) {
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int step = (gridDim.x - 1) * kPlanThreads;
        for (int i = (blockIdx.x - 1) * kPlanThreads + tid; i < a.num_blocks; i += step) a.shares_out[i] = a.shares[i];
        return;
    }
    extern __shared__ int s_claims[];  // [B]: forks to the sequence
    __shared__ int s_warp[32];
    for (int b = tid; b < a.B; b += kPlanThreads) {
        s_claims[b] = 0;
        if (a.held_out != a.held) a.held_out[b] = a.held[b];
        if (a.seq_lens_out != a.seq_lens) a.seq_lens_out[b] = a.seq_lens[b];
    }
    if (alone && a.shares_out != a.shares)
        for (int i = tid; i < a.num_blocks; i += kPlanThreads) a.shares_out[i] = a.shares[i];
    const int count = *a.free_count;
    const bool count_ok = count >= 0 && count <= a.num_blocks;
    __syncthreads();
    for (int i = tid; i < a.F; i += kPlanThreads) {
        const int d = a.fork_dst[i];
        if (a.fork_src[i] >= 0 && d >= 0 && d < a.B) atomicAdd(&s_claims[d], 1);
    }
    __syncthreads();
    constexpr int kPer = kPagesMaxForks / kPlanThreads;
    const int per = (a.F + kPlanThreads - 1) / kPlanThreads;  // consecutive forks of a thread, at most kPer
    int src[kPer], dst[kPer], len[kPer], err[kPer], part[kPer];
    int needs = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        src[u] = -1;
        const int i = tid * per + u;
        if (u >= per || i >= a.F) continue;
        src[u] = a.fork_src[i];
        if (src[u] < 0) continue;
        dst[u] = a.fork_dst[i];
        err[u] = 0;
        part[u] = -1;
        len[u] = 0;
        if (src[u] >= a.B || dst[u] < 0 || dst[u] >= a.B || s_claims[dst[u]] > 1 || a.held[dst[u]] != 0) {
            err[u] = TSV_DERR_SEQ;
            continue;
        }
        const int L = a.seq_lens[src[u]], h = a.held[src[u]];
        if (L < 0 || h < 0 || h > a.max_blocks || cdiv_shift(L, a.bs_log2) > h) {
            err[u] = TSV_DERR_CAPACITY;
            continue;
        }
        if (!count_ok) {
            err[u] = TSV_DERR_POOL;
            continue;
        }
        len[u] = L;
        if (L & ((1 << a.bs_log2) - 1)) {
            part[u] = a.block_table[(long long)src[u] * a.max_blocks + (L >> a.bs_log2)];
            ++needs;
            err[u] = -1;  // takes a block
        }
    }
    int total;
    int taken = block_scan(needs, s_warp, &total);  // (its barriers: every input has been read by now)
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = tid * per + u;
        if (u >= per || i >= a.F) continue;
        int from = -1, to = -1, rows = 0, e = 0;
        if (src[u] >= 0) {
            e = err[u];
            const int full = len[u] >> a.bs_log2;
            if (e == -1) {
                e = 0;
                if (++taken > count) {
                    e = TSV_DERR_POOL;
                } else {
                    const int fresh = a.free_blocks[count - taken];
                    a.block_table[(long long)dst[u] * a.max_blocks + full] = fresh;
                    if (part[u] < 0 || part[u] >= a.num_blocks || fresh < 0 || fresh >= a.num_blocks) {
                        e = TSV_DERR_BLOCK;
                    } else {
                        from = part[u];
                        to = fresh;
                        rows = len[u] & ((1 << a.bs_log2) - 1);
                    }
                }
            }
            if (!(e & kFatal)) {
                a.held_out[dst[u]] = cdiv_shift(len[u], a.bs_log2);
                a.seq_lens_out[dst[u]] = len[u];
            }
        }
        a.copy_src[i] = from;
        a.copy_dst[i] = to;
        a.copy_rows[i] = rows;
        a.fork_err[i] = e;
    }
    if (tid == 0) *a.free_count_out = count_ok ? count - min(total, count) : count;
    if (!alone) return;
    __syncthreads();  // what the rows need is written, by this CTA
    for (int i = tid >> 5; i < a.F; i += kPlanThreads / 32) fork_row(a, i, tid & 31, 32);
}

// One fork a CTA; blockIdx.y divides long rows.
__global__ void __launch_bounds__(kRowThreads) kv_fork_rows_kernel(const __grid_constant__ ForkArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    fork_row(a, blockIdx.x, blockIdx.y * kRowThreads + threadIdx.x, gridDim.y * kRowThreads);
}


// ------------------------------------------------------------------ scans over the block ids

// CTA `rank` of `ctas` takes a run of ids, in tiles of 4096: a warp 128 neighbours, 32 at a time.
constexpr int kTileIds = 4 * kPlanThreads;
struct IdRun {
    int first, end;
    __device__ __forceinline__ IdRun(int num_blocks, int rank, int ctas) {
        const int chunk = (num_blocks + ctas - 1) / ctas;
        first = min(rank * chunk, num_blocks);
        end = min(first + chunk, num_blocks);
    }
    __device__ __forceinline__ static int id(int tile, int u) {
        return tile + (threadIdx.x >> 5) * 128 + u * 32 + (threadIdx.x & 31);
    }
};

// Ranks within a tile: rank[u] = marked ids of the tile before id(tile, u); returns their number.
__device__ __forceinline__ int tile_ranks(const bool (&mark)[4], int (&rank)[4], int* s_warp) {
    const int lane = threadIdx.x & 31;
    int sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const unsigned m = __ballot_sync(0xffffffffu, mark[u]);
        rank[u] = sum + __popc(m & ((1u << lane) - 1));
        sum += __popc(m);
    }
    int total;
    // every lane holds the warp's sum: one lane hands it to the scan, the others nothing
    const int before = block_scan(lane == 0 ? sum : 0, s_warp, &total);
    const int base = __shfl_sync(0xffffffffu, before, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u) rank[u] += base;
    return total;
}

// Sums over the cluster's CTAs before this one, *all: over all CTAs.  s_slot must not be written again before a
// barrier of the cluster.
template <int CLUSTER>
__device__ __forceinline__ int2 cluster_before(int2 mine, int2* s_slot, int2* all) {
    if (CLUSTER == 1) {
        *all = mine;
        return make_int2(0, 0);
    }
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) *s_slot = mine;
    cl.sync();
    int2 before = make_int2(0, 0), sum = make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) {
        const int2 x = *cl.map_shared_rank(s_slot, r);
        if (r < static_cast<int>(cl.block_rank())) {
            before.x += x.x;
            before.y += x.y;
        }
        sum.x += x.x;
        sum.y += x.y;
    }
    *all = sum;
    return before;
}
template <int CLUSTER>
__device__ __forceinline__ void cluster_barrier() {
    if (CLUSTER == 1)
        __syncthreads();
    else
        cg::this_cluster().sync();
}
template <int CLUSTER>
__device__ __forceinline__ int cluster_rank() {
    return CLUSTER == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
}

// ------------------------------------------------------------------ release

// Entries a sequence keeps; *err: what is wrong with it (then it keeps all).
__device__ __forceinline__ int kept_blocks(const ReleaseArgs& a, int held, int keep, bool count_ok, int* err) {
    *err = 0;
    if (held < 0 || held > a.max_blocks || keep < 0)
        *err = TSV_DERR_CAPACITY;
    else if (!count_ok)
        *err = TSV_DERR_POOL;
    return *err ? held : min(held, cdiv_shift(keep, a.bs_log2));
}

__global__ void __launch_bounds__(256) copy_ints_kernel(int32_t* to, const int32_t* from, int n) {
    pdl_wait();
    pdl_launch_dependents();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) to[i] = from[i];
}

// Sequence b, by the threads first, first + n, ...: each released entry takes one reference off its block; -1 is
// none left.  True if a block id is outside the cache.
__device__ __forceinline__ bool release_row(const ReleaseArgs& a, int b, int first, int n, int* err) {
    const int count = *a.free_count, held = a.held[b];
    const int stay = kept_blocks(a, held, a.keep_lens[b], count >= 0 && count <= a.num_blocks, err);
    const int32_t* row = a.block_table + (long long)b * a.max_blocks;
    bool bad = false;
    constexpr int U = 4;
    if (*err == 0)
        for (int j0 = stay + first; j0 < held; j0 += U * n) {
            int id[U];
#pragma unroll
            for (int u = 0; u < U; ++u) id[u] = j0 + u * n < held ? row[j0 + u * n] : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j0 + u * n >= held) continue;
                if (id[u] >= 0 && id[u] < a.num_blocks)
                    atomicSub(a.shares_out + id[u], 1);
                else
                    bad = true;
            }
        }
    return bad;
}

// One sequence a CTA.
__global__ void __launch_bounds__(kPlanThreads) kv_release_count_kernel(const __grid_constant__ ReleaseArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    int err;
    const bool bad = __syncthreads_or(release_row(a, blockIdx.x, threadIdx.x, blockDim.x, &err));
    if (threadIdx.x == 0) a.seq_err[blockIdx.x] = bad ? TSV_DERR_BLOCK : err;
}

// One cluster: blocks without a reference go onto the pool in order of their ids.
template <int CLUSTER>
__device__ __forceinline__ void release_push(const ReleaseArgs& a) {
    __shared__ int s_warp[32];
    __shared__ int2 s_slot;
    const int tid = threadIdx.x, rank = cluster_rank<CLUSTER>();
    const IdRun run(a.num_blocks, rank, CLUSTER);
    const int count = *a.free_count;
    const bool count_ok = count >= 0 && count <= a.num_blocks;
    int mine = 0;
    bool over = false;
    for (int id = run.first + tid; id < run.end; id += kPlanThreads) {
        const int s = __ldcg(a.shares_out + id);
        mine += s < 0;
        over |= s < -1;
    }
    int sum;
    block_scan(mine, s_warp, &sum);
    int2 all;  // blocks without a reference, whether any was given back too often
    const int before = cluster_before<CLUSTER>(make_int2(count_ok ? sum : 0, __syncthreads_or(over) ? 1 : 0), &s_slot, &all).x;
    const bool full = count_ok && all.x > a.num_blocks - count;
    if (all.y || full) {
        // more references given back than there were, or more blocks than the pool has places: the
        // sequences that took part are told
        for (int b = rank; b < a.B; b += CLUSTER) {
            const int held = a.held[b];
            int err;
            const int stay = kept_blocks(a, held, a.keep_lens[b], count_ok, &err);
            bool hit = full && err == 0 && stay < held;
            if (err == 0)
                for (int j = stay + tid; j < held; j += kPlanThreads) {
                    const int id = a.block_table[(long long)b * a.max_blocks + j];
                    hit |= id >= 0 && id < a.num_blocks && __ldcg(a.shares_out + id) < -1;
                }
            if (__syncthreads_or(hit) && tid == 0) a.seq_err[b] |= TSV_DERR_POOL;
        }
    }
    cluster_barrier<CLUSTER>();  // counts and shares have been read
    int place = count + before;
    for (int tile = run.first; tile < run.end; tile += kTileIds) {
        bool mark[4];
        int r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int id = IdRun::id(tile, u);
            mark[u] = count_ok && id < run.end && __ldcg(a.shares_out + id) < 0;
        }
        const int n = tile_ranks(mark, r, s_warp);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!mark[u]) continue;
            const int id = IdRun::id(tile, u);
            a.shares_out[id] = 0;
            if (place + r[u] < a.num_blocks) a.free_blocks[place + r[u]] = id;
        }
        place += n;
    }
    for (int b = rank * kPlanThreads + tid; b < a.B; b += CLUSTER * kPlanThreads) {
        int err;
        a.held_out[b] = kept_blocks(a, a.held[b], a.keep_lens[b], count_ok, &err);
    }
    if (rank == 0 && tid == 0) *a.free_count_out = count_ok ? min(count + all.x, a.num_blocks) : count;
}
template <int CLUSTER>
__global__ void __launch_bounds__(kPlanThreads) kv_release_push_kernel(const __grid_constant__ ReleaseArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    release_push<CLUSTER>(a);
}

// Small calls: one CTA for it all (8 sequences of 2053 tokens: 10 -> 4.2 us).
constexpr int kReleaseSmallIds = 8192, kReleaseSmallEntries = 32768;  // block ids, and table entries, up to which
__global__ void __launch_bounds__(kPlanThreads) kv_release_small_kernel(const __grid_constant__ ReleaseArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    if (a.shares_out != a.shares)
        for (int i = threadIdx.x; i < a.num_blocks; i += kPlanThreads) a.shares_out[i] = a.shares[i];
    __syncthreads();
    for (int b = threadIdx.x >> 5; b < a.B; b += kPlanThreads / 32) {
        int err;
        const bool bad = __any_sync(0xffffffffu, release_row(a, b, threadIdx.x & 31, 32, &err));
        if ((threadIdx.x & 31) == 0) a.seq_err[b] = bad ? TSV_DERR_BLOCK : err;
    }
    __syncthreads();
    release_push<1>(a);
}

// ------------------------------------------------------------------ compaction

__global__ void __launch_bounds__(256) kv_compact_clear_kernel(const __grid_constant__ CompactBlocksArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < a.num_blocks; i += gridDim.x * 256) {
        a.remap[i] = 0;
        if (i < a.num_blocks / 2) {
            a.copy_src[i] = -1;
            a.copy_dst[i] = -1;
        }
    }
}

// One sequence a CTA: its blocks are live.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_mark_kernel(const __grid_constant__ CompactBlocksArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x, held = a.held[b];
    const bool ok = held >= 0 && held <= a.max_blocks;
    const int32_t* row = a.block_table + (long long)b * a.max_blocks;
    bool bad = false;
    if (ok)
        for (int j = threadIdx.x; j < held; j += blockDim.x) {
            const int id = row[j];
            if (id >= 0 && id < a.num_blocks)
                a.remap[id] = 1;
            else
                bad = true;
        }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) a.seq_err[b] = !ok ? TSV_DERR_CAPACITY : bad ? TSV_DERR_BLOCK : 0;
}

// Small caches and tables, one CTA instead of the three kernels around it: the live ids are bits in shared
// memory, their ranks come from running sums of the words.
constexpr int kBitIds = 16384, kBitEntries = 65536;  // ids, and table entries, up to which it is taken
__global__ void __launch_bounds__(kPlanThreads) kv_compact_small_kernel(const __grid_constant__ CompactBlocksArgs a) {
    constexpr int kWords = kBitIds / 32;  // a thread has at most one
    static_assert(kWords <= kPlanThreads, "a word for each thread");
    __shared__ uint32_t s_live[kWords];
    __shared__ int s_before[kWords + 1];  // live ids before a word
    __shared__ uint16_t s_from[kBitIds / 2], s_to[kBitIds / 2];
    __shared__ int s_warp[32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, nb = a.num_blocks, words = (nb + 31) >> 5;
    for (int w = tid; w < words; w += kPlanThreads) s_live[w] = 0;
    __syncthreads();
    for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {  // a warp a sequence
        const int held = a.held[b];
        const bool ok = held >= 0 && held <= a.max_blocks;
        bool bad = false;
        constexpr int U = 4;
        if (ok)
            for (int j0 = lane; j0 < held; j0 += 32 * U) {
                int id[U];
#pragma unroll
                for (int u = 0; u < U; ++u) id[u] = j0 + 32 * u < held ? a.block_table[(long long)b * a.max_blocks + j0 + 32 * u] : -1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (id[u] >= 0 && id[u] < nb)
                        atomicOr(&s_live[id[u] >> 5], 1u << (id[u] & 31));
                    else
                        bad |= j0 + 32 * u < held;
                }
            }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) a.seq_err[b] = !ok ? TSV_DERR_CAPACITY : bad ? TSV_DERR_BLOCK : 0;
    }
    __syncthreads();
    int n;
    const int before = block_scan(tid < words ? __popc(s_live[tid]) : 0, s_warp, &n);
    if (tid < kWords) s_before[tid] = before;
    if (tid == 0) s_before[kWords] = n;
    __syncthreads();
    auto rank = [&](int id) { return s_before[id >> 5] + ((id & 31) ? __popc(s_live[id >> 5] & ((1u << (id & 31)) - 1)) : 0); };
    const int moves = n - rank(n);
    for (int id = tid; id < nb; id += kPlanThreads) {
        const bool live = (s_live[id >> 5] >> (id & 31)) & 1u;
        const int rk = rank(id);
        if (live && id >= n) {
            s_from[rk - (n - moves)] = static_cast<uint16_t>(id);  // its share moves with it, below
        } else if (live) {
            if (a.shares_out != a.shares) a.shares_out[id] = a.shares[id];
        } else {
            if (id < n) s_to[id - rk] = static_cast<uint16_t>(id);
            a.shares_out[id] = 0;
        }
        if (id < nb - n) a.free_blocks[id] = nb - 1 - id;
    }
    __syncthreads();
    for (int k = tid; k < nb / 2; k += kPlanThreads) {
        const int from = k < moves ? s_from[k] : -1, to = k < moves ? s_to[k] : -1;
        a.copy_src[k] = from;
        a.copy_dst[k] = to;
        if (from < 0) continue;
        const int s = a.shares[from];
        a.remap[from] = to;
        a.shares_out[to] = s;
        a.shares_out[from] = 0;
    }
    if (tid == 0) {
        *a.free_count_out = nb - n;
        *a.copy_count = moves;
    }
}

// One cluster: with n live blocks, the k-th live id from n on moves to the k-th free id below n.
template <int CLUSTER>
__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(const __grid_constant__ CompactBlocksArgs a) {
    __shared__ int s_warp[32];
    __shared__ int2 s_slot[2];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, rank = cluster_rank<CLUSTER>();
    const IdRun run(a.num_blocks, rank, CLUSTER);
    int mine = 0;
    for (int id = run.first + tid; id < run.end; id += kPlanThreads) mine += a.remap[id];
    int sum;
    block_scan(mine, s_warp, &sum);
    int2 all;
    const int before = cluster_before<CLUSTER>(make_int2(sum, 0), &s_slot[0], &all).x, n = all.x;
    mine = 0;
    for (int id = max(run.first, n) + tid; id < run.end; id += kPlanThreads) mine += a.remap[id];
    block_scan(mine, s_warp, &sum);
    cluster_before<CLUSTER>(make_int2(sum, 0), &s_slot[1], &all);
    const int moves = all.x;
    cluster_barrier<CLUSTER>();
    int place = before;  // live ids before the tile
    for (int tile = run.first; tile < run.end; tile += kTileIds) {
        bool mark[4];
        int r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int id = IdRun::id(tile, u);
            mark[u] = id < run.end && a.remap[id] != 0;
        }
        const int live = tile_ranks(mark, r, s_warp);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int id = IdRun::id(tile, u);
            if (id >= run.end) continue;
            const int rk = place + r[u];
            if (mark[u] && id < n) {
                if (a.shares_out != a.shares) a.shares_out[id] = a.shares[id];
            } else if (mark[u]) {
                // its share moves with it, below
                if (TSV_IN_BOUNDS(rk - (n - moves), a.num_blocks / 2, nullptr)) a.copy_src[rk - (n - moves)] = id;
            } else {
                if (id < n && TSV_IN_BOUNDS(id - rk, a.num_blocks / 2, nullptr)) a.copy_dst[id - rk] = id;
                a.shares_out[id] = 0;
            }
            if (id < a.num_blocks - n) a.free_blocks[id] = a.num_blocks - 1 - id;
        }
        place += live;
    }
    __threadfence();
    cluster_barrier<CLUSTER>();
    for (int k = rank * kPlanThreads + tid; k < moves; k += CLUSTER * kPlanThreads) {
        const int from = __ldcg(a.copy_src + k), to = __ldcg(a.copy_dst + k);
        a.remap[from] = to;
        const int s = __ldcg(a.shares + from);
        a.shares_out[to] = s;
        a.shares_out[from] = 0;
    }
    if (rank == 0 && tid == 0) {
        *a.free_count_out = a.num_blocks - n;
        *a.copy_count = moves;
    }
}

// One sequence a CTA: its row under the new ids; entries that are not held stay.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_rows_kernel(const __grid_constant__ CompactBlocksArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x, held = a.held[b], n = a.num_blocks - *a.free_count_out;  // ids below n stay
    const int mine = held <= a.max_blocks ? held : 0;
    const int end = a.block_table_out == a.block_table ? mine : a.max_blocks;
    const int32_t* row = a.block_table + (long long)b * a.max_blocks;
    int32_t* out = a.block_table_out + (long long)b * a.max_blocks;
    constexpr int U = 4;
    const int step = blockDim.x;
    for (int j0 = threadIdx.x; j0 < end; j0 += U * step) {
        int id[U], to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = j0 + u * step < end ? row[j0 + u * step] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) to[u] = j0 + u * step < mine && id[u] >= n && id[u] < a.num_blocks ? a.remap[id[u]] : id[u];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * step < end) out[j0 + u * step] = to[u];
    }
}

// ------------------------------------------------------------------ copy

// A piece is 16 KB of one block of one cache: 4 vectors a thread, all on their way before one is
// written.
constexpr int kCopyThreads = 256, kCopyVecs = 4, kPieceVecs = kCopyThreads * kCopyVecs;

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a, int pieces) {
    pdl_wait();
    pdl_launch_dependents();
    const int n = a.copy_count ? min(max(*a.copy_count, 0), a.n) : a.n;
    for (int i = blockIdx.x * kCopyThreads + threadIdx.x; i < a.n; i += gridDim.x * kCopyThreads) {
        int e = 0;
        if (i < n && a.copy_src[i] >= 0) {
            const int d = a.copy_dst[i];
            if (a.copy_src[i] >= a.num_blocks || d < 0 || d >= a.num_blocks) e = TSV_DERR_BLOCK;
        }
        a.copy_err[i] = e;
    }
    const long long all = (long long)n * 2 * pieces, block_vecs = (long long)a.bs * a.row_vecs;
    for (long long w = blockIdx.x; w < all; w += gridDim.x) {
        const int i = static_cast<int>(w / (2 * pieces)), rest = static_cast<int>(w % (2 * pieces));
        const int s = a.copy_src[i], d = a.copy_dst[i];
        if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks || s == d) continue;
        const int rows = a.copy_rows ? min(max(a.copy_rows[i], 0), a.bs) : a.bs;
        const long long vecs = (long long)rows * a.row_vecs, first = (long long)(rest >> 1) * kPieceVecs + threadIdx.x;
        uint4* cache = static_cast<uint4*>((rest & 1) ? a.v_cache : a.k_cache);
        const uint4* from = cache + s * block_vecs;
        uint4* to = cache + d * block_vecs;
        uint4 x[kCopyVecs];
#pragma unroll
        for (int u = 0; u < kCopyVecs; ++u)
            if (first + u * kCopyThreads < vecs) x[u] = from[first + u * kCopyThreads];
#pragma unroll
        for (int u = 0; u < kCopyVecs; ++u)
            if (first + u * kCopyThreads < vecs) to[first + u * kCopyThreads] = x[u];
    }
}

#ifdef TSV_TEST_HOOKS
bool g_test_pages_cluster = true;  // test build: whether the cluster counts as resident
#endif

// Whether a cluster of eight CTAs of the kernel can be resident (a partitioned GPU may not have as
// many SMs in one group); looked up once per device and host thread.
template <typename K>
bool cluster8_fits(K kernel, int& of_dev, bool& fits) {
#ifdef TSV_TEST_HOOKS
    if (!g_test_pages_cluster) return false;
#endif
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev != of_dev) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 8;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(8);
        cfg.blockDim = dim3(kPlanThreads);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        fits = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
        of_dev = dev;
    }
    return fits;
}

// Threads for a row of the table, a CTA a row.
unsigned row_threads(int max_blocks) {
    unsigned t = 128;
    while (t < kPlanThreads && static_cast<int>(4 * t) < max_blocks) t *= 2;
    return t;
}
unsigned int_ctas(int n, int num_sms) {
    const int c = (n + 1023) / 1024;
    return static_cast<unsigned>(c < 1 ? 1 : c < num_sms ? c : num_sms);
}

// Block ids up to which one CTA scans them; beyond, a cluster of eight.
constexpr int kOneCtaIds = 8192;

}  // namespace

#ifdef TSV_TEST_HOOKS
// test build only: 0 = the cluster counts as not resident
extern "C" void tsv_test_set_pages_cluster(int on) { g_test_pages_cluster = on != 0; }
#endif

cudaError_t launch_kv_fork(const ForkArgs& a, int num_sms, cudaStream_t stream) {
    const bool alone = (a.shares_out == a.shares || a.num_blocks <= kForkSmallIds) && (long long)a.F * a.max_blocks <= kForkSmallEntries;
    const unsigned copiers = alone || a.shares_out == a.shares ? 0u : int_ctas(a.num_blocks, num_sms);
    cudaError_t e = launch_pdl(kv_fork_plan_kernel, dim3(1 + copiers), dim3(kPlanThreads), a.B * sizeof(int), stream, 1u, a, alone ? 1 : 0);
    if (e != cudaSuccess || a.F == 0 || alone) return e;
    const int split = (a.max_blocks + 4 * kRowThreads - 1) / (4 * kRowThreads);
    return launch_pdl(kv_fork_rows_kernel, dim3(static_cast<unsigned>(a.F), static_cast<unsigned>(split < 16 ? split : 16)), dim3(kRowThreads),
                      0, stream, 1u, a);
}

cudaError_t launch_kv_release(const ReleaseArgs& a, int num_sms, cudaStream_t stream) {
    thread_local int of_dev = -1;
    thread_local bool fits = false;
    if (a.num_blocks <= kReleaseSmallIds && (long long)a.B * a.max_blocks <= kReleaseSmallEntries)
        return launch_pdl(kv_release_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, 1u, a);
    cudaError_t e = cudaSuccess;
    if (a.shares_out != a.shares)
        e = launch_pdl(copy_ints_kernel, dim3(int_ctas(a.num_blocks, num_sms)), dim3(256), 0, stream, 1u, a.shares_out, a.shares, a.num_blocks);
    if (e == cudaSuccess && a.B > 0)
        e = launch_pdl(kv_release_count_kernel, dim3(static_cast<unsigned>(a.B)), dim3(row_threads(a.max_blocks)), 0, stream, 1u, a);
    if (e != cudaSuccess) return e;
    if (a.num_blocks > kOneCtaIds && cluster8_fits(kv_release_push_kernel<8>, of_dev, fits))
        return launch_pdl(kv_release_push_kernel<8>, dim3(8), dim3(kPlanThreads), 0, stream, 8u, a);
    return launch_pdl(kv_release_push_kernel<1>, dim3(1), dim3(kPlanThreads), 0, stream, 1u, a);
}

cudaError_t launch_kv_compact_blocks(const CompactBlocksArgs& a, int num_sms, cudaStream_t stream) {
    thread_local int of_dev = -1;
    thread_local bool fits = false;
    cudaError_t e;
    if (a.num_blocks <= kBitIds && (long long)a.B * a.max_blocks <= kBitEntries) {
        e = launch_pdl(kv_compact_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, 1u, a);
    } else {
        e = launch_pdl(kv_compact_clear_kernel, dim3(int_ctas(a.num_blocks, num_sms)), dim3(256), 0, stream, 1u, a);
        if (e == cudaSuccess && a.B > 0)
            e = launch_pdl(kv_compact_mark_kernel, dim3(static_cast<unsigned>(a.B)), dim3(row_threads(a.max_blocks)), 0, stream, 1u, a);
        if (e != cudaSuccess) return e;
        if (a.num_blocks > kOneCtaIds && cluster8_fits(kv_compact_plan_kernel<8>, of_dev, fits))
            e = launch_pdl(kv_compact_plan_kernel<8>, dim3(8), dim3(kPlanThreads), 0, stream, 8u, a);
        else
            e = launch_pdl(kv_compact_plan_kernel<1>, dim3(1), dim3(kPlanThreads), 0, stream, 1u, a);
    }
    if (e != cudaSuccess || a.B == 0) return e;
    return launch_pdl(kv_compact_rows_kernel, dim3(static_cast<unsigned>(a.B)), dim3(row_threads(a.max_blocks)), 0, stream, 1u, a);
}

cudaError_t launch_kv_copy(const CopyArgs& a, int num_sms, cudaStream_t stream) {
    const long long block_vecs = (long long)a.bs * a.row_vecs;
    const int pieces = static_cast<int>((block_vecs + kPieceVecs - 1) / kPieceVecs);
    const long long all = (long long)a.n * 2 * pieces, most = 8LL * num_sms;
    return launch_pdl(kv_copy_kernel, dim3(static_cast<unsigned>(all < most ? all : most)), dim3(kCopyThreads), 0, stream, 1u, a, pieces);
}

}  // namespace tsv
