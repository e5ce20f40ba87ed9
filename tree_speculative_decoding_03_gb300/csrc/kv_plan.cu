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
// One cluster: every CTA loads all lengths and scans them (they are a few KB, and reading
// them is cheaper than passing the scans on); after a cluster barrier, from which on outputs
// that share memory with inputs may be written, the tokens, the fresh table entries and the
// returned blocks are divided between all threads, each finding its sequence by bisection of
// the scans in shared memory.
#include <climits>
#include <cooperative_groups.h>

#include "common.cuh"
#include "serving_args.cuh"

namespace tsv {
namespace {
namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

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

__device__ __forceinline__ int sat_int(long long x) { return x > INT_MAX ? INT_MAX : static_cast<int>(x); }

// Inclusive block-wide scan of three sums at once; *carry holds the totals of the passes before.
struct Three {
    long long a, b, c;
};
__device__ __forceinline__ Three block_scan(Three v, Three* s_warp, Three* carry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o),
                        c = __shfl_up_sync(0xffffffffu, v.c, o);
        if (lane >= o) {
            v.a += a;
            v.b += b;
            v.c += c;
        }
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        Three w = lane < kPlanThreads / 32 ? s_warp[lane] : Three{0, 0, 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o),
                            c = __shfl_up_sync(0xffffffffu, w.c, o);
            if (lane >= o) {
                w.a += a;
                w.b += b;
                w.c += c;
            }
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        v.a += s_warp[warp - 1].a;
        v.b += s_warp[warp - 1].b;
        v.c += s_warp[warp - 1].c;
    }
    v.a += carry->a;
    v.b += carry->b;
    v.c += carry->c;
    carry->a += s_warp[31].a;
    carry->b += s_warp[31].b;
    carry->c += s_warp[31].c;
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kPlanThreads, 1) kv_plan_kernel(const PlanArgs a) {
    extern __shared__ int s_dyn[];
    int* s_len = s_dyn;              // cached length (0 for a sequence whose lengths are bad)
    int* s_held = s_len + a.B;       // blocks held
    int* s_tok = s_held + a.B;       // end of the sequence's tokens
    int* s_grow = s_tok + a.B;       // end of its fresh blocks
    int* s_back = s_grow + a.B;      // end of its returned blocks
    uint8_t* s_err = reinterpret_cast<uint8_t*>(s_back + a.B);
    __shared__ Three s_warp[32];
    __shared__ int s_top, s_grown;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, bs = 1 << a.bs_log2;
    const long long cap = (long long)a.max_blocks << a.bs_log2;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) {
        s_top = 0;
        s_grown = 0;
    }
    const int count = *a.free_count;
    const bool pool_ok = count >= 0 && count <= a.num_blocks;
    Three carry{0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int L = 0, n = 0, held = 0, err = 0;
        long long want = 0, grow = 0, back = 0;
        if (b < a.B) {
            L = a.seq_lens[b];
            n = a.new_lens[b];
            held = a.held[b];
            if (L < 0 || n < 0 || (long long)L + n > cap || held < 0 || held > a.max_blocks) err |= TSV_DERR_CAPACITY;
            if (a.parent != nullptr && n > a.N) err |= TSV_DERR_PARENT;
            if (!pool_ok) err |= TSV_DERR_POOL;
            if (n < 0) n = 0;
            if (L < 0) L = 0;
            if (err == 0) {
                want = ((long long)L + n + bs - 1) >> a.bs_log2;
                grow = want > held ? want - held : 0;
                back = held > want ? held - want : 0;
            }
        }
        // tokens first: a sequence whose tokens do not all fit the map takes and returns nothing
        Three v{n, grow, back};
        Three e = block_scan(v, s_warp, &carry);
        if (b < a.B) {
            if (e.a > a.max_tokens && n > 0) err |= TSV_DERR_CAPACITY;
            s_len[b] = L;
            s_held[b] = held;
            s_tok[b] = sat_int(e.a);
            s_grow[b] = static_cast<int>(grow);
            s_back[b] = static_cast<int>(back);
            s_err[b] = static_cast<uint8_t>(err);
        }
    }
    __syncthreads();
    const long long total = carry.a;
    carry = Three{0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        const bool live = b < a.B && s_err[b] == 0;
        const long long grow = live ? s_grow[b] : 0, back = live ? s_back[b] : 0;
        const Three e = block_scan(Three{0, grow, back}, s_warp, &carry);
        if (b < a.B) {
            int err = s_err[b];
            // more blocks come back than the pool has places for: the caller's counts are wrong
            if (back > 0 && count + e.c > a.num_blocks) err |= TSV_DERR_POOL;
            if (back > 0 && err == 0) atomicMax(&s_top, static_cast<int>(e.c));
            s_err[b] = static_cast<uint8_t>(err);
            s_grow[b] = sat_int(e.b);
            s_back[b] = sat_int(e.c);
        }
    }
    __syncthreads();
    const int top = (pool_ok ? count : 0) + s_top;
    for (int b = tid; b < a.B; b += kPlanThreads) {
        const int before = b > 0 ? s_grow[b - 1] : 0;
        if (s_grow[b] > before) {
            if (s_grow[b] > top)
                s_err[b] |= static_cast<uint8_t>(TSV_DERR_POOL);
            else
                atomicMax(&s_grown, s_grow[b]);
        }
    }
    // every CTA of the cluster has read the inputs: from here on outputs may be written
    cluster.sync();
    const int grown = s_grown;
    const int left = top - grown;
    const int t0 = static_cast<int>(cluster.block_rank()) * kPlanThreads + tid;
    const int nthreads = kPlanCluster * kPlanThreads;

    auto want_of = [&](int b) {
        const int n = s_tok[b] - (b > 0 ? s_tok[b - 1] : 0);
        return static_cast<int>(((long long)s_len[b] + n + bs - 1) >> a.bs_log2);
    };
    // block id at place p of the stack
    auto stack_at = [&](int p) {
        if (p < count) return a.free_blocks[p];
        const int i = p - count;
        const int b = first_above(s_back, a.B, i);
        if (b >= a.B) return -1;
        return a.block_table[(long long)b * a.max_blocks + want_of(b) + (i - (b > 0 ? s_back[b - 1] : 0))];
    };

    for (int b = t0; b < a.B; b += nthreads) {
        const int err = s_err[b];
        const int n = s_tok[b] - (b > 0 ? s_tok[b - 1] : 0);
        a.seq_err[b] = err;
        a.token_offsets[b + 1] = s_tok[b];
        if (err == 0) {
            a.held_out[b] = want_of(b);
            a.total_lens[b] = s_len[b] + n;
        } else {
            a.held_out[b] = s_held[b];
            a.total_lens[b] = s_len[b];
        }
    }
    if (t0 == 0) {
        a.token_offsets[0] = 0;
        *a.free_count_out = pool_ok ? left : count;
    }
    // errors found below are added to words that another CTA may be writing above
    cluster.sync();

    for (int t = t0; t < a.max_tokens; t += nthreads) {
        long long slot = -1;
        int pos = -1;
        if (t < total) {
            const int b = first_above(s_tok, a.B, t);
            if (s_err[b] == 0) {
                const int j = t - (b > 0 ? s_tok[b - 1] : 0);
                const int at = s_len[b] + j, blk = at >> a.bs_log2, held = s_held[b];
                const int id = blk < held ? a.block_table[(long long)b * a.max_blocks + blk]
                                          : stack_at(top - 1 - ((b > 0 ? s_grow[b - 1] : 0) + blk - held));
                if (id >= 0 && id < a.num_blocks)
                    slot = ((long long)id << a.bs_log2) + (at & (bs - 1));
                else
                    atomicOr(&a.seq_err[b], TSV_DERR_BLOCK);
                int depth = j;
                if (a.parent != nullptr) {
                    // distance to the root; every node is checked by its own first step
                    const int32_t* par = a.parent + (long long)b * a.N;
                    depth = 0;
                    int x = j;
                    while (x > 0) {
                        const int p = __ldg(par + x);
                        if (p < 0 || p >= x) break;
                        x = p;
                        ++depth;
                    }
                    if (x != 0 || __ldg(par) != -1) {
                        depth = -1 - s_len[b];  // position -1
                        atomicOr(&a.seq_err[b], TSV_DERR_PARENT);
                    }
                }
                pos = s_len[b] + depth;
            }
        }
        a.slot_map[t] = slot;
        a.positions[t] = pos;
    }
    for (int k = t0; k < grown; k += nthreads) {
        const int b = first_above(s_grow, a.B, k);
        const int j = s_held[b] + (k - (b > 0 ? s_grow[b - 1] : 0));
        a.block_table[(long long)b * a.max_blocks + j] = stack_at(top - 1 - k);
    }
    for (int p = (pool_ok ? count : left) + t0; p < left; p += nthreads) {
        const int id = stack_at(p);
        a.free_blocks[p] = id;
        if (id < 0 || id >= a.num_blocks) {
            const int b = first_above(s_back, a.B, p - count);
            if (b < a.B) atomicOr(&a.seq_err[b], TSV_DERR_BLOCK);
        }
    }
}

}  // namespace

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
    const size_t smem = (size_t)a.B * (5 * sizeof(int) + 1) + 16;
    thread_local int smem_dev = -1;
    thread_local size_t smem_set = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != smem_dev || smem > smem_set) {
        e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        smem_dev = dev;
        smem_set = smem;
    }
    return launch_pdl(kv_plan_kernel, dim3(kPlanCluster), dim3(kPlanThreads), smem, stream, kPlanCluster, a);
}

}  // namespace tsv
