// kv_plan.cu -- block tables, slot maps and positions from request lengths.
//
// Per sequence b with L cached and n new tokens and `held` blocks:
//   want = ceil((L + n) / bs), grow = max(0, want - held), back = max(0, held - want).
// The pool is a stack of free block ids.  The surplus blocks (table entries want .. held-1)
// are pushed in order of (b, index), then the fresh ones are popped in order of (b, index).
// Both are prefix sums over the sequences: place count + i of the stack is the i-th surplus
// block, and the k-th fresh block is at place top - 1 - k with top = count + sum(back).  So
// no thread waits for another's push or pop, and the result does not depend on timing.
//
// One cluster (one CTA for small batches): every CTA loads all lengths and scans them -- they are
// a few KB, and reading them is cheaper than passing the scans on.  After a cluster barrier, from
// which on outputs that share memory with inputs may be written, the tokens, the fresh table
// entries and the returned blocks are one list of items, divided between all threads; each
// item finds its sequence by bisection of the scans in shared memory.  The work is a chain of
// latencies (launch, lengths, scan, ids, stores), not bytes.  Large slot maps are filled by a
// second kernel over all SMs instead, from the outputs of the first.
#include <climits>
#include <cooperative_groups.h>

#include "../common.cuh"
#include "serving_args.cuh"

namespace tsv {
namespace {
namespace cg = cooperative_groups;

// Launches by size, us in a stream (one CTA / a cluster of 16 / the cluster and a fill kernel): 8 trees
// of 6 nodes 3.7 / 4.7 / 6.7; 32 of 16 4.2 / 4.6 / 8.2; 16 of 64 6.6 / 5.7 / 14.2; 512 of 64 - / 9.5 / 15.7; 1000
// prompts of 60 tokens - / 8.3 / 10.0; 1000 trees of 64 - / 15.6 / 15.9; 1000 prompts of 255 tokens with a
// cluster of 8 36.6, with the fill kernel 9.4.  Against 16 CTAs a cluster of 8 takes 15.2 for 512 x 64.
constexpr int kPlanCluster = 16;
constexpr int kPlanSmallSeqs = 64, kPlanSmallTokens = 512;  // one CTA up to here
constexpr int kPlanClusterTokens = 65536;                  // tokens by the cluster up to here
constexpr int kFillThreads = 256, kFillTokens = 4;  // the second kernel: threads, tokens of a thread

// First i in [0, n) with end[i] > x (n when there is none): the sequence item x falls in.
__device__ __forceinline__ int first_above(const int* end, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Sums of counts stay at INT_MAX once they reach it (associative, so a scan may use it).
__device__ __forceinline__ int sat_add(int a, int b) {
    const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
    return s > static_cast<unsigned>(INT_MAX) ? INT_MAX : static_cast<int>(s);
}

// Three running sums: tokens, fresh blocks, returned blocks.
struct Three {
    int a, b, c;
    __device__ __forceinline__ void add(const Three& o) {
        a = sat_add(a, o.a);
        b = sat_add(b, o.b);
        c = sat_add(c, o.c);
    }
};
__device__ __forceinline__ Three warp_scan(Three v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Three y{__shfl_up_sync(0xffffffffu, v.a, o), __shfl_up_sync(0xffffffffu, v.b, o), __shfl_up_sync(0xffffffffu, v.c, o)};
        if (lane >= o) v.add(y);
    }
    return v;
}
// Inclusive scan over the block; `carry` (the same in every thread) holds the sums of the passes
// before.
template <int THREADS>
__device__ __forceinline__ Three block_scan(Three v, Three* s_warp, Three* carry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v);
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    // every warp scans the warps' sums for itself
    const Three w = warp_scan(lane < THREADS / 32 ? s_warp[lane] : Three{0, 0, 0});
    const int from = warp > 0 ? warp - 1 : 0;
    Three before{__shfl_sync(0xffffffffu, w.a, from), __shfl_sync(0xffffffffu, w.b, from), __shfl_sync(0xffffffffu, w.c, from)};
    if (warp > 0) v.add(before);
    v.add(*carry);
    carry->add(Three{__shfl_sync(0xffffffffu, w.a, 31), __shfl_sync(0xffffffffu, w.b, 31), __shfl_sync(0xffffffffu, w.c, 31)});
    __syncthreads();
    return v;
}

// Distance of node j from the root, or -1 where the path leaves the rules of a tree.  Every node
// is checked by its own first step.
__device__ __forceinline__ int depth_of(const int32_t* par, int j) {
    int depth = 0, x = j;
    while (x > 0) {
        const int p = par[x];
        if (p < 0 || p >= x) return -1;
        x = p;
        ++depth;
    }
    return par[0] == -1 ? depth : -1;
}

template <int THREADS, int CLUSTER, bool TOKENS>
__global__ void __launch_bounds__(THREADS, 1) kv_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int s_dyn[];
    int* s_len = s_dyn;              // cached length (0 for a negative one)
    int* s_held = s_len + a.B;       // blocks held
    int* s_tok = s_held + a.B;       // end of the sequence's tokens
    int* s_grow = s_tok + a.B;       // end of its fresh blocks
    int* s_back = s_grow + a.B;      // end of its returned blocks
    uint8_t* s_err = reinterpret_cast<uint8_t*>(s_back + a.B);
    __shared__ Three s_warp[32];
    __shared__ int s_top, s_grown;
    const int tid = threadIdx.x, bs = 1 << a.bs_log2;
    const int rank = CLUSTER > 1 ? static_cast<int>(blockIdx.x) : 0;  // the grid is one cluster
    const long long cap = (long long)a.max_blocks << a.bs_log2;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) {
        s_top = 0;
        s_grown = 0;
    }
    const int count = *a.free_count;
    const bool pool_ok = count >= 0 && count <= a.num_blocks;
    // The running sums of all three counts.  A sequence whose tokens pass the map's end takes and
    // returns nothing, which the token sums decide: where that happens the scan is repeated
    // without those sequences' blocks.
    int total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        Three carry{0, 0, 0};
        bool past = false;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            const int b = b0 + tid;
            int L = 0, n = 0, held = 0, err = 0, grow = 0, back = 0;
            if (b < a.B) {
                L = a.seq_lens[b];
                n = a.new_lens[b];
                held = a.held[b];
                if (L < 0 || n < 0 || (long long)L + n > cap || held < 0 || held > a.max_blocks) err |= TSV_DERR_CAPACITY;
                if (a.parent != nullptr && n > a.N) err |= TSV_DERR_PARENT;
                if (!pool_ok) err |= TSV_DERR_POOL;
                n = max(n, 0);
                L = max(L, 0);
                if (pass == 1 && n > 0 && s_tok[b] > a.max_tokens) err |= TSV_DERR_CAPACITY;
                if (err == 0) {
                    const int want = static_cast<int>(((long long)L + n + bs - 1) >> a.bs_log2);
                    grow = max(want - held, 0);
                    back = max(held - want, 0);
                }
            }
            const Three e = block_scan<THREADS>(Three{n, grow, back}, s_warp, &carry);
            if (b < a.B) {
                past |= n > 0 && e.a > a.max_tokens;
                // more blocks come back than the pool has places for: the caller's counts are wrong
                if (back > 0 && (long long)count + e.c > a.num_blocks) err |= TSV_DERR_POOL;
                s_len[b] = L;
                s_held[b] = held;
                s_tok[b] = e.a;
                s_grow[b] = e.b;
                s_back[b] = e.c;
                s_err[b] = static_cast<uint8_t>(err);
                // the last sequence that gives back decides the stack's height
                if (back > 0 && err == 0) atomicMax(&s_top, e.c);
            }
        }
        total = carry.a;
        if (!__syncthreads_or(past) || pass == 1) break;
        if (tid == 0) s_top = 0;
        __syncthreads();
    }
    const int top = (pool_ok ? count : 0) + s_top;
    for (int b = tid; b < a.B; b += THREADS) {
        const int before = b > 0 ? s_grow[b - 1] : 0;
        int err = s_err[b];
        if (s_grow[b] > before && err == 0) {
            if (s_grow[b] > top)
                err |= TSV_DERR_POOL;
            else
                atomicMax(&s_grown, s_grow[b]);
            s_err[b] = static_cast<uint8_t>(err);
        }
        if (b % CLUSTER == rank) a.seq_err[b] = err;
    }
    // every CTA of the cluster has read the inputs: from here on their memory may be written.  The
    // error words are in place too; bits are added to them below.
    if (CLUSTER > 1)
        cg::this_cluster().sync();
    else
        __syncthreads();
    const int grown = s_grown, left = top - grown;

    auto begin = [&](const int* end, int b) { return b > 0 ? end[b - 1] : 0; };
    auto want_of = [&](int b) {
        return static_cast<int>(((long long)s_len[b] + s_tok[b] - begin(s_tok, b) + bs - 1) >> a.bs_log2);
    };
    // block id at place p of the stack
    auto stack_at = [&](int p) {
        if (p < count) return TSV_IN_BOUNDS(p, a.num_blocks, a.seq_err) ? a.free_blocks[p] : -1;
        const int i = p - count, b = first_above(s_back, a.B, i);
        if (b >= a.B) return -1;
        const long long at = (long long)b * a.max_blocks + want_of(b) + (i - begin(s_back, b));
        return TSV_IN_BOUNDS(at, (long long)a.B * a.max_blocks, a.seq_err + b) ? a.block_table[at] : -1;
    };

    const int t0 = rank * THREADS + tid;
    constexpr int kAll = CLUSTER * THREADS;
    const int tokens = TOKENS ? a.max_tokens : 0, pushed = pool_ok ? max(left - count, 0) : 0;
    const int seqs = max(a.B, 1);  // an empty batch has the first item's single words too
    const long long items = (long long)tokens + seqs + grown + pushed;
    for (long long item = t0; item < items; item += kAll) {
        if (item < tokens) {
            const int t = static_cast<int>(item);
            long long slot = -1;
            int pos = -1;
            const int b = t < total ? first_above(s_tok, a.B, t) : a.B;
            if (b < a.B && s_err[b] == 0) {
                const int j = t - begin(s_tok, b), at = s_len[b] + j, blk = at >> a.bs_log2, held = s_held[b];
                const int id = blk < held ? (TSV_IN_BOUNDS(blk, a.max_blocks, a.seq_err + b) ? a.block_table[(long long)b * a.max_blocks + blk] : -1)
                                          : stack_at(top - 1 - (begin(s_grow, b) + blk - held));
                const int depth = a.parent != nullptr ? depth_of(a.parent + (long long)b * a.N, j) : j;
                int err = 0;
                if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
                    slot = ((long long)id << a.bs_log2) + (at & (bs - 1));
                else
                    err |= TSV_DERR_BLOCK;
                if (depth >= 0)
                    pos = s_len[b] + depth;
                else
                    err |= TSV_DERR_PARENT;
                if (err) atomicOr(&a.seq_err[b], err);
            }
            a.slot_map[t] = slot;
            a.positions[t] = pos;
            continue;
        }
        int k = static_cast<int>(item - tokens);
        if (k < seqs) {
            if (k == 0) {
                a.token_offsets[0] = 0;
                *a.free_count_out = pool_ok ? left : count;
            }
            if (k >= a.B) continue;
            const bool ok = s_err[k] == 0;
            const int end = s_tok[k];
            a.token_offsets[k + 1] = end;
            a.held_out[k] = ok ? want_of(k) : s_held[k];
            a.total_lens[k] = s_len[k] + (ok ? end - begin(s_tok, k) : 0);
            continue;
        }
        k -= seqs;
        if (k < grown) {
            const int b = first_above(s_grow, a.B, k);
            const int j = s_held[b] + (k - begin(s_grow, b));
            if (TSV_IN_BOUNDS(j, a.max_blocks, a.seq_err + b)) a.block_table[(long long)b * a.max_blocks + j] = stack_at(top - 1 - k);
            continue;
        }
        k -= grown;  // a returned block that stays on the stack
        const int id = stack_at(count + k);
        if (TSV_IN_BOUNDS(count + k, a.num_blocks, a.seq_err)) a.free_blocks[count + k] = id;
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
            const int b = first_above(s_back, a.B, k);
            if (b < a.B) atomicOr(&a.seq_err[b], TSV_DERR_BLOCK);
        }
    }
}

// The slots and positions of a large map, from the first kernel's outputs: a CTA's tokens lie in
// the sequences between two places of token_offsets, which it copies to shared memory.
__global__ void __launch_bounds__(kFillThreads) kv_plan_fill_kernel(const __grid_constant__ PlanArgs a) {
    constexpr int kTok = kFillThreads * kFillTokens;
    __shared__ int s_end[kTok + 1];
    __shared__ int s_b[2];
    const int tid = threadIdx.x, bs = 1 << a.bs_log2;
    const int t0 = blockIdx.x * kTok, t1 = min(t0 + kTok, a.max_tokens);
    pdl_wait();
    pdl_launch_dependents();
    const int* end = a.token_offsets + 1;
    const int total = min(end[a.B - 1], a.max_tokens);  // (an empty batch: token_offsets[0], 0)
    if (tid < 64) {
        // warp 0: the sequence of the CTA's first token, warp 1: of its last; 32 probes a step
        const int lane = tid & 31, x = tid < 32 ? t0 : min(t1, total) - 1;
        int lo = 0, n = a.B;  // the first i with end[i] > x lies in [lo, lo + n)
        while (n > 0) {
            const int step = (n + 31) >> 5, i = lo + min(lane * step + step, n) - 1;
            const unsigned above = __ballot_sync(0xffffffffu, end[i] > x);
            if (above == 0) {
                lo += n;
                break;
            }
            const int f = __ffs(above) - 1;
            const int next = lo + f * step;
            n = min(step, n - f * step) - 1;  // the probe itself is above: what is left lies before it
            lo = next;
        }
        if (lane == 0) s_b[tid >> 5] = lo;
    }
    __syncthreads();
    const int b0 = s_b[0], nb = t0 < total ? s_b[1] - b0 + 1 : 0;
    // a sequence without tokens holds no token, so at most kTok of them do; the others in between
    // would not fit: those CTAs bisect in global memory
    const bool local = nb <= kTok;
    if (local)
        for (int i = tid; i < nb; i += kFillThreads) s_end[i] = end[b0 + i];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kFillTokens; ++u) {
        const int t = t0 + u * kFillThreads + tid;
        if (t >= a.max_tokens) break;
        long long slot = -1;
        int pos = -1;
        if (t < total) {
            const int b = b0 + (local ? first_above(s_end, nb, t) : first_above(end + b0, nb, t));
            const int first = a.token_offsets[b], j = t - first, n = end[b] - first;
            const int tot = a.total_lens[b], e = a.seq_err[b];
            // a sequence that was not served keeps its length, so these hold its tokens back
            const bool held_back = (e & (TSV_DERR_CAPACITY | TSV_DERR_POOL)) != 0 || (a.parent != nullptr && n > a.N);
            if (!held_back) {
                const int at = tot - n + j;
                const int blk = at >> a.bs_log2;
                const int id = TSV_IN_BOUNDS(blk, a.max_blocks, a.seq_err + b) ? a.block_table[(long long)b * a.max_blocks + blk] : -1;
                const int depth = a.parent != nullptr ? depth_of(a.parent + (long long)b * a.N, j) : j;
                int err = 0;
                if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
                    slot = ((long long)id << a.bs_log2) + (at & (bs - 1));
                else
                    err |= TSV_DERR_BLOCK;
                if (depth >= 0)
                    pos = tot - n + depth;
                else
                    err |= TSV_DERR_PARENT;
                if (err) atomicOr(&a.seq_err[b], err);
            }
        }
        a.slot_map[t] = slot;
        a.positions[t] = pos;
    }
}

constexpr size_t plan_smem(int B) { return (size_t)B * (5 * sizeof(int) + 1) + 16; }

// The kernel's limits, raised once per device and host thread.
template <int THREADS, int CLUSTER, bool TOKENS>
cudaError_t raise_limits(int dev) {
    thread_local int set_dev = -1;
    if (dev == set_dev) return cudaSuccess;
    const auto kernel = kv_plan_kernel<THREADS, CLUSTER, TOKENS>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(plan_smem(kPlanMaxSeqs)));
    if (e == cudaSuccess && CLUSTER > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) set_dev = dev;
    return e;
}

#ifdef TSV_TEST_HOOKS
int g_test_plan_cluster = kPlanCluster;  // test build: the largest cluster that counts as resident
#endif

// Whether a cluster of this size, with the largest batch's shared memory, can be resident.
template <int CLUSTER>
bool cluster_fits(int dev) {
#ifdef TSV_TEST_HOOKS
    if (CLUSTER > g_test_plan_cluster) return false;
#endif
    if (raise_limits<1024, CLUSTER, true>(dev) != cudaSuccess) return false;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CLUSTER;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(CLUSTER);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = plan_smem(kPlanMaxSeqs);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kv_plan_kernel<1024, CLUSTER, true>, &cfg) == cudaSuccess && n > 0;
}

template <int THREADS, int CLUSTER, bool TOKENS>
cudaError_t launch_plan(const PlanArgs& a, int dev, cudaStream_t stream) {
    const size_t smem = plan_smem(a.B);
    const cudaError_t e = raise_limits<THREADS, CLUSTER, TOKENS>(dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_plan_kernel<THREADS, CLUSTER, TOKENS>, dim3(CLUSTER), dim3(THREADS), smem, stream, CLUSTER, a);
}

// The cluster's size: a cluster of 16 needs as many SMs of one GPC, which a partitioned GPU may not
// have; then 8, or one CTA.  Looked up once per device and host thread.
template <bool TOKENS>
cudaError_t launch_clustered(const PlanArgs& a, int dev, cudaStream_t stream) {
    thread_local int of_dev = -1, size = 0;
#ifdef TSV_TEST_HOOKS
    of_dev = -1;
#endif
    if (dev != of_dev) {
        size = cluster_fits<kPlanCluster>(dev) ? kPlanCluster : cluster_fits<8>(dev) ? 8 : 1;
        of_dev = dev;
    }
    if (size == kPlanCluster) return launch_plan<1024, kPlanCluster, TOKENS>(a, dev, stream);
    return size == 8 ? launch_plan<1024, 8, TOKENS>(a, dev, stream) : launch_plan<1024, 1, TOKENS>(a, dev, stream);
}

}  // namespace

#ifdef TSV_TEST_HOOKS
// test build only: clusters of more CTAs count as not resident
extern "C" int tsv_test_set_plan_cluster(int most) {
    const int before = g_test_plan_cluster;
    g_test_plan_cluster = most;
    return before;
}
#endif

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (a.B <= kPlanSmallSeqs && a.max_tokens <= kPlanSmallTokens) return launch_plan<512, 1, true>(a, dev, stream);
    if (a.max_tokens <= kPlanClusterTokens) return launch_clustered<true>(a, dev, stream);
    e = launch_clustered<false>(a, dev, stream);
    if (e != cudaSuccess) return e;
    constexpr int kTok = kFillThreads * kFillTokens;
    return launch_pdl(kv_plan_fill_kernel, dim3(static_cast<unsigned>((a.max_tokens + kTok - 1) / kTok)), dim3(kFillThreads), 0,
                      stream, 1u, a);
}

}  // namespace tsv
