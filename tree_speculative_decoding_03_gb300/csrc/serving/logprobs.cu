// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives of logits rows.
//
// With z = x / T, m = max z, s = sum e^{z - m}, w = sum e^{z - m} (z - m):
//   log p(t) = z_t - m - ln s,   H = -sum p ln p = ln s - w / s.
// One pass: every thread keeps a running m, s and w of its slice in fp32 and rescales them when m
// grows (s' = f s, w' = f (w + s (m_old - m)), f = e^{m_old - m}).  Bound by the logits' bytes.
//
// The alternatives come from the same pass: a thread's running maximum is the largest of its
// slice.  Of 64 groups of threads the n-th largest group maximum is a bound that at least n
// entries reach, so only slices whose maximum reaches it hold alternatives -- some n of 256, or
// of 512 in a cluster --
// and those few are read again by all threads.  The entries that reach the bound, hardly more than n, are
// ranked among themselves; where they are many, warps keep lists in order.  Nothing depends on the values but
// the time: a row of equal logits is read three times.  (Lists for every row, a slice at a time: 2000 rows of
// 128256 bf16 with 5 / 20 / 32 alternatives 106 / 131 / 153 us, without any 91.)
// Order: value descending (-0 and 0 are equal), then index ascending, as one 64-bit key.
//
// A row is taken by one CTA, by a cluster of up to eight where there are too few rows to fill the GPU, or, where it is
// short, by a warp.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "../common.cuh"
#include "continue_args.cuh"

namespace tsv {
namespace {
namespace cg = cooperative_groups;

constexpr int kGroups = 64;
// vectors of a tile: neighbours, so that a thread's slice is read again in 64-byte pieces (16-byte pieces
// spread over the row cost four times their bytes: 2000 rows of 128256 bf16, 20 alternatives, 126 us; these 115)
constexpr int kAhead = 2;
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;
// z - m in units of log2 is held above this, where e^{z - m} is 0 in fp32: a logit of -inf then adds
// 0 * -200 to w and not 0 * -inf
constexpr float kFloor = -200.0f;
static_assert(kGroups >= kMaxTop && kMaxTop <= 32, "a group for each alternative, a lane for each");

typedef unsigned long long Key;  // 0: none

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// larger value, then lower index, is the larger key; finite and -inf values give keys above 0
__device__ __forceinline__ Key make_key(float x, uint32_t index) {
    const uint32_t u = __float_as_uint(x + 0.0f), ord = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (static_cast<Key>(ord) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(Key k) {
    const uint32_t o = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int key_index(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

// pairs of fp32, an instruction a pair
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float first(Pair p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float second(Pair p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A 32-byte vector of logits as floats.
template <typename Elem>
struct Vec;
struct Raw {
    uint32_t r[8];
    __device__ __forceinline__ void load(const void* p) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    }
};
template <>
struct Vec<float> : Raw {
    static constexpr int N = 8;
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = 0xff800000u;
    }
    __device__ __forceinline__ void set(int i, const float* p) { r[i] = __float_as_uint(*p); }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(r[i]); }
    __device__ __forceinline__ float top() const {
        return max_nan(max_nan(max_nan(get(0), get(1)), max_nan(get(2), get(3))), max_nan(max_nan(get(4), get(5)), max_nan(get(6), get(7))));
    }
};
template <>
struct Vec<__nv_bfloat16> : Raw {
    static constexpr int N = 16;
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = 0xff80ff80u;
    }
    __device__ __forceinline__ void set(int i, const __nv_bfloat16* p) {
        const uint32_t u = *reinterpret_cast<const unsigned short*>(p);
        r[i >> 1] = i & 1 ? (r[i >> 1] & 0x0000ffffu) | (u << 16) : (r[i >> 1] & 0xffff0000u) | u;
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16); }
    __device__ __forceinline__ float top() const {
        const uint32_t u = max_nan2(max_nan2(max_nan2(r[0], r[1]), max_nan2(r[2], r[3])), max_nan2(max_nan2(r[4], r[5]), max_nan2(r[6], r[7])));
        return max_nan(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};

// A row as aligned vectors: the first may begin before the row and the last end behind it, and of
// those only the row's own elements are read.
template <typename Elem>
struct Row {
    static constexpr int N = Vec<Elem>::N;
    const Elem* x;
    int head, V, vecs;  // elements of the first vector before the row
    __device__ __forceinline__ Row(const Elem* row, int V_)
        : x(row), head(static_cast<int>((reinterpret_cast<uintptr_t>(row) & 31) / sizeof(Elem))), V(V_) {
        vecs = static_cast<int>(((long long)head + V + N - 1) / N);
    }
    __device__ __forceinline__ int index(int v) const { return v * N - head; }  // of the vector's first element
    // vectors between the first and the last
    __device__ __forceinline__ int inner() const { return max(vecs - 2, 0); }
    // the first or last vector of the row if it is thread t's (-1: it is not)
    __device__ __forceinline__ int edge(int t, bool first_cta, bool last_cta) const {
        return t == 0 && first_cta ? 0 : t == 1 && last_cta && vecs > 1 ? vecs - 1 : -1;
    }
    // a vector that may reach over the row's ends
    __device__ __forceinline__ Vec<Elem> load_some(int v) const {
        Vec<Elem> y;
        const int i0 = index(v);
        y.none();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i0 + i >= 0 && i0 + i < V) y.set(i, x + i0 + i);
        return y;
    }
    // vectors v, v + 1, ... below `end`, which lie inside the row
    template <int COUNT>
    __device__ __forceinline__ void load_tile(Vec<Elem> (&y)[COUNT], int v, int end) const {
        const Elem* p = x + index(v);
        if (v + COUNT <= end) {
#pragma unroll
            for (int u = 0; u < COUNT; ++u) y[u].load(p + u * N);
        } else {
#pragma unroll
            for (int u = 0; u < COUNT; ++u) {
                y[u].none();
                if (v + u < end) y[u].load(p + u * N);
            }
        }
    }
};

// Running sums of a slice, m in units of x.
struct Stats {
    float m, s, w;
    // c = log2(e) / T
    __device__ __forceinline__ void rise(float to, float c) {
        const float d = fmaxf((m - to) * c, kFloor), f = ex2(d);
        w = f * fmaf(s, d, w);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(float m2, float s2, float w2, float c) {
        Stats o{m2, s2, w2};
        if (o.m > m) rise(o.m, c);
        if (m > o.m) o.rise(m, c);
        s += o.s;
        w += o.w;
    }
};

// sum = sum of e^{z - m}, w = sum of e^{z - m} (z - m) log2(e) over a thread's vectors.  MASKED: the exponent is
// held above kFloor, an instruction more for an entry.
template <bool ENTROPY, bool MASKED, typename V>
__device__ __forceinline__ void add_tile(const V (&y)[kAhead], Pair less, Pair by, float* sum, float* w) {
    Pair s2[2] = {0, 0}, w2[2] = {0, 0};  // (0.0f, 0.0f)
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < V::N; i += 2) {
            Pair d = mul2(add2(pair(y[u].get(i), y[u].get(i + 1)), less), by);
            if (ENTROPY && MASKED) d = pair(fmaxf(first(d), kFloor), fmaxf(second(d), kFloor));
            const Pair p = pair(ex2(first(d)), ex2(second(d)));
            s2[(i >> 1) & 1] = add2(s2[(i >> 1) & 1], p);
            if (ENTROPY) w2[(i >> 1) & 1] = fma2(p, d, w2[(i >> 1) & 1]);
        }
    const Pair ss = add2(s2[0], s2[1]), ww = add2(w2[0], w2[1]);
    *sum = first(ss) + second(ss);
    *w = first(ww) + second(ww);
}

// The best keys of a warp, in order: lane i holds the i-th (0: none).
struct Best {
    Key key = 0;
    // the lanes' candidates (0: none); `top` are kept
    __device__ __forceinline__ void add(Key k, int top) {
        const int lane = threadIdx.x & 31;
        Key least = __shfl_sync(0xffffffffu, key, top - 1);
        unsigned todo = __ballot_sync(0xffffffffu, k > least);
        while (todo) {
            const Key n = __shfl_sync(0xffffffffu, k, __ffs(todo) - 1);
            const int pos = __popc(__ballot_sync(0xffffffffu, key > n));
            const Key up = __shfl_up_sync(0xffffffffu, key, 1);
            if (lane == pos) key = n;
            if (lane > pos) key = up;
            least = __shfl_sync(0xffffffffu, key, top - 1);
            todo &= todo - 1;
            todo &= __ballot_sync(0xffffffffu, k > least);
        }
    }
};

__host__ __device__ constexpr int threads_of(int cluster) { return cluster == 1 ? 256 : 512; }

// Appends a key; beyond kKeys they are counted alone.  The order in the list does not matter: keys are
// distinct and ranked later.
constexpr int kKeys = 512;  // at least 32 a warp
__device__ __forceinline__ void keep(Key* keys, int* n, Key k) {
    const int at = atomicAdd(n, 1);
    if (at < kKeys) keys[at] = k;
}

// Ranks the `n` keys of `keys` (distinct): the thread of rank r < top gives out[r].
__device__ __forceinline__ void rank_keys(const Key* keys, int n, int top, Key* out) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const Key k = keys[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += keys[j] > k;
        if (r < top) out[r] = k;
    }
}

// Row t has no token: padding, or a wrong one.
__device__ __forceinline__ void no_row(const LogprobArgs& a, int t, int token, int tid) {
    const float x = token < 0 ? 0.0f : __int_as_float(0x7fc00000);
    if (tid == 0) {
        a.logprob[t] = x;
        if (a.entropy) a.entropy[t] = x;
        a.tok_err[t] = token < 0 ? 0 : TSV_DERR_TOKEN;
    }
    if (tid < a.top) {
        a.top_ids[(long long)t * a.top + tid] = -1;
        a.top_logprobs[(long long)t * a.top + tid] = x;
    }
}

// Short rows, a warp a row, PER entries of it in a lane's registers; the bound comes from 64 groups of every
// 64th entry.  (A CTA a row has too few threads with a slice for 64 groups and waits through its barriers: 4000
// rows of 400 bf16 with 20 alternatives 141 us there, 10.7 here; 100 rows 13 and 6.)
constexpr int kShortWarps = 4, kShortKeys = 128;
constexpr int kShortRow = 1024;  // entries up to which a row is short: 32 a lane
template <typename Elem, int PER>
__global__ void __launch_bounds__(32 * kShortWarps) token_logprobs_short_kernel(const __grid_constant__ LogprobArgs a) {
    __shared__ __align__(16) float s_group[kShortWarps][kGroups];
    __shared__ Key s_keys[kShortWarps][kShortKeys], s_best[kShortWarps][32];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = static_cast<int>(blockIdx.x) * kShortWarps + warp;
    if (t >= a.T) return;
    const int token = a.tokens[t];
    if (token < 0 || token >= a.V) {
        no_row(a, t, token, lane);
        return;
    }
    const Elem* x = static_cast<const Elem*>(a.logits) + (long long)t * a.stride;
    const float xt = static_cast<float>(x[token]), c = a.inv_t * kLog2e;
    float z[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] = 32 * i + lane < a.V ? static_cast<float>(x[32 * i + lane]) : -INFINITY;
    float mine[2] = {z[0], z[1]};  // the lane's two groups
#pragma unroll
    for (int i = 2; i < PER; ++i) mine[i & 1] = max_nan(mine[i & 1], z[i]);
    float m = max_nan(mine[0], mine[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float nan = __int_as_float(0x7fc00000);
    if (!(m < INFINITY && m > -INFINITY)) {  // a NaN or +inf, or no finite logit: no distribution
        if (lane == 0) {
            a.logprob[t] = nan;
            if (a.entropy) a.entropy[t] = nan;
            a.tok_err[t] = TSV_DERR_NONFINITE;
        }
        if (lane < a.top) {
            a.top_ids[(long long)t * a.top + lane] = -1;
            a.top_logprobs[(long long)t * a.top + lane] = nan;
        }
        return;
    }
    float s = 0.0f, w = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float d = fmaxf((z[i] - m) * c, kFloor), p = ex2(d);
        s += p;
        w = fmaf(p, d, w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    const float log_s = logf(s);
    if (lane == 0) {
        a.logprob[t] = (xt - m) * a.inv_t - log_s;
        if (a.entropy) a.entropy[t] = log_s - kLn2 * (w / s);
        a.tok_err[t] = 0;
    }
    if (a.top == 0) return;
    // the bound: the top-th largest of the group maxima
    s_group[warp][lane] = mine[0];
    s_group[warp][32 + lane] = mine[1];
    __syncwarp();
    int r0 = 0, r1 = 0;
#pragma unroll 4
    for (int j = 0; j < kGroups; ++j) {
        const float o = s_group[warp][j];
        r0 += o > mine[0] || (o == mine[0] && j < lane);
        r1 += o > mine[1] || (o == mine[1] && j < 32 + lane);
    }
    const unsigned at0 = __ballot_sync(0xffffffffu, r0 == a.top - 1), at1 = __ballot_sync(0xffffffffu, r1 == a.top - 1);
    const float bound = __shfl_sync(0xffffffffu, at0 ? mine[0] : mine[1], __ffs(at0 ? at0 : at1) - 1);
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = 32 * i + lane < a.V && z[i] >= bound;
        const unsigned all = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(all & ((1u << lane) - 1));
        if (in && at < kShortKeys) s_keys[warp][at] = make_key(z[i], static_cast<uint32_t>(32 * i + lane));
        n += __popc(all);
    }
    __syncwarp();
    if (n <= kShortKeys) {
        for (int i = lane; i < n; i += 32) {
            const Key k = s_keys[warp][i];
            int r = 0;
            for (int j = 0; j < n; ++j) r += s_keys[warp][j] > k;
            if (r < a.top) s_best[warp][r] = k;
        }
    } else {  // ties: the best in order, one a lane
        Best best;
#pragma unroll 1
        for (int i = 0; i < PER; ++i) {
            const int at = 32 * i + lane;
            const float y = at < a.V ? static_cast<float>(x[at]) : -INFINITY;
            best.add(at < a.V && y >= bound ? make_key(y, static_cast<uint32_t>(at)) : 0, a.top);
        }
        s_best[warp][lane] = best.key;
    }
    __syncwarp();
    if (lane < a.top) {
        const Key k = s_best[warp][lane];
        a.top_ids[(long long)t * a.top + lane] = key_index(k);
        a.top_logprobs[(long long)t * a.top + lane] = (key_value(k) - m) * a.inv_t - log_s;
    }
}

// THREADS: 256, four CTAs an SM, where there is a row for each CTA, so that a row's end overlaps other rows' loads
// (2000 rows of 128256 bf16 logits); 512 in a cluster.
template <typename Elem, int CLUSTER, bool ENTROPY>
__global__ void __launch_bounds__(threads_of(CLUSTER), 1024 / threads_of(CLUSTER)) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    constexpr int N = Vec<Elem>::N, kThreads = threads_of(CLUSTER), kWarps = kThreads / 32;
    __shared__ float s_m[kWarps], s_s[kWarps], s_w[kWarps];
    __shared__ __align__(16) float s_group[kGroups];
    __shared__ Stats s_stats;   // of the CTA
    __shared__ int s_bad, s_n, s_count, s_slices[kThreads];
    __shared__ float s_bound;
    __shared__ Key s_keys[kKeys], s_best[32];
    __shared__ Key s_all[CLUSTER > 1 ? CLUSTER * 32 : 1];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CLUSTER == 1 ? 0 : static_cast<int>(blockIdx.x % CLUSTER);
    const int t = static_cast<int>(blockIdx.x / CLUSTER);
    const int token = a.tokens[t];
    if (token < 0 || token >= a.V) {  // padding, or a wrong token: the same in every CTA of the cluster
        if (rank == 0) no_row(a, t, token, tid);
        return;
    }
    const Elem* x = static_cast<const Elem*>(a.logits) + (long long)t * a.stride;
    const Row<Elem> row(x, a.V);
    // the CTA's vectors, but for the row's first and last
    const int begin = 1 + static_cast<int>((long long)row.inner() * rank / CLUSTER), end = 1 + static_cast<int>((long long)row.inner() * (rank + 1) / CLUSTER);
    const float c = a.inv_t * kLog2e;
    Stats st{-INFINITY, 0.0f, 0.0f};
    bool bad = false, masked = false;
    // The row's first and last vector, which may hold other elements too: the first two threads'.
    const int edge = row.edge(tid, rank == 0, rank == CLUSTER - 1);
    if (edge >= 0) {
        const Vec<Elem> y = row.load_some(edge);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float z = y.get(i);
            if (!(z <= st.m)) {
                bad |= !(z < INFINITY);
                st.rise(z, c);
            }
            const float d = st.m == -INFINITY ? kFloor : fmaxf((z - st.m) * c, kFloor), p = ex2(d);
            st.s += p;
            if (ENTROPY) st.w = fmaf(p, d, st.w);
        }
    }
    // the others, the next ones on their way while a tile is added
    Vec<Elem> next[kAhead];
    row.load_tile(next, begin + kAhead * tid, end);
    for (int v = begin + kAhead * tid; v < end; v += kAhead * kThreads) {
        Vec<Elem> y[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) y[u] = next[u];
        row.load_tile(next, v + kAhead * kThreads, end);
        float top = y[0].top();
#pragma unroll
        for (int u = 1; u < kAhead; ++u) top = max_nan(top, y[u].top());
        if (!(top <= st.m)) {
            bad |= !(top < INFINITY);  // +inf or NaN
            st.rise(top, c);
        }
        if (st.m == -INFINITY) continue;
        const Pair less = pair(-st.m, -st.m), by = pair(c, c);
        float sum, w;
        if (!masked) {
            add_tile<ENTROPY, false>(y, less, by, &sum, &w);
            masked = ENTROPY && w != w;  // entries of -inf among them, 0 * -inf: once more and from now on without
        }
        if (masked) add_tile<ENTROPY, true>(y, less, by, &sum, &w);
        st.s += sum;
        if (ENTROPY) st.w += w;
    }
    const float slice_max = st.m;
    if (tid == 0) {
        s_n = 0;
        s_count = 0;
        s_bound = -INFINITY;
    }
    // the CTA's sums, in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        st.join(__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o), __shfl_xor_sync(0xffffffffu, st.w, o), c);
    if (lane == 0) {
        s_m[warp] = st.m;
        s_s[warp] = st.s;
        s_w[warp] = st.w;
    }
    if (a.top > 0) {
        // groups of neighbours, as few as make 64 groups of the threads that have a slice: then half of the groups
        // hold entries wherever 32 threads do (4000 rows of 3000 bf16 with 32 alternatives and four threads a
        // group, most groups empty and the bound -inf: 462 us; 52)
        const int threads = min((end - begin + kAhead - 1) / kAhead, kThreads);
        int log2 = 0;
        while (threads > kGroups << log2) ++log2;
        float g = slice_max;
        for (int o = 1; o < 1 << log2; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if ((tid & ((1 << log2) - 1)) == 0 && tid >> log2 < kGroups) s_group[tid >> log2] = g;
    }
    bad = __syncthreads_or(bad);
    if (warp == 0) {
        Stats all{lane < kWarps ? s_m[lane] : -INFINITY, lane < kWarps ? s_s[lane] : 0.0f, lane < kWarps ? s_w[lane] : 0.0f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            all.join(__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.s, o), __shfl_xor_sync(0xffffffffu, all.w, o), c);
        if (lane == 0) {
            s_stats = all;
            s_bad = bad;
        }
    }
    if (a.top > 0) {
        // the bound: the top-th largest of the group maxima (in a bad row, none may be found)
        if (tid < kGroups) {
            const float g = s_group[tid];
            int r = 0;
#pragma unroll
            for (int j = 0; j < kGroups; j += 4) {
                const float4 o = *reinterpret_cast<const float4*>(s_group + j);
                r += (o.x > g || (o.x == g && j < tid)) + (o.y > g || (o.y == g && j + 1 < tid)) + (o.z > g || (o.z == g && j + 2 < tid)) +
                     (o.w > g || (o.w == g && j + 3 < tid));
            }
            if (r == a.top - 1) s_bound = g;
        }
        __syncthreads();
        const float bound = s_bound;
        // slices that hold alternatives: some `top` of them
        if (!bad && slice_max >= bound) s_slices[atomicAdd(&s_count, 1)] = tid;
        if (tid < 32) s_best[tid] = 0;
        __syncthreads();
        const int slices = s_count, per_slice = (end - begin + kAhead * kThreads - 1) / (kAhead * kThreads) * kAhead;
        // vector q of thread t's slice
        auto slice_vec = [&](int t, int q) { return begin + kAhead * t + q % kAhead + q / kAhead * (kAhead * kThreads); };
        // all their vectors, spread over the threads
        for (int i0 = tid; i0 < slices * per_slice; i0 += 2 * kThreads) {
            Vec<Elem> y[2];
            int v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = i0 + u * kThreads, sl = i / per_slice;
                v[u] = i < slices * per_slice ? slice_vec(s_slices[sl], i - sl * per_slice) : end;
                y[u].none();
                if (v[u] < end) y[u].load(x + row.index(v[u]));
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!(v[u] < end && y[u].top() >= bound)) continue;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (y[u].get(i) >= bound) keep(s_keys, &s_n, make_key(y[u].get(i), static_cast<uint32_t>(row.index(v[u]) + i)));
            }
        }
        if (edge >= 0 && !bad) {
            const Vec<Elem> y = row.load_some(edge);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = row.index(edge) + i;
                if (at >= 0 && at < a.V && y.get(i) >= bound) keep(s_keys, &s_n, make_key(y.get(i), static_cast<uint32_t>(at)));
            }
        }
        __syncthreads();
        if (s_n > kKeys) {
            // more entries reach the bound than there is room for (rows of equal or few distinct values, of
            // rising ones): every warp keeps its best in order, one a lane, from whole slices
            __syncthreads();
            if (tid == 0) s_n = 0;
            Best best;
            for (int sl = warp; sl < slices; sl += kWarps) {
                const int owner = s_slices[sl];
                auto offer = [&](const Vec<Elem>& y, int v, bool have) {
                    if (!__any_sync(0xffffffffu, have && y.top() >= bound)) return;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int at = row.index(v) + i;
                        const float z = y.get(i);
                        const bool in = have && at >= 0 && at < a.V && z >= bound;
                        if (__any_sync(0xffffffffu, in)) best.add(in ? make_key(z, static_cast<uint32_t>(at)) : 0, a.top);
                    }
                };
                const int some = row.edge(owner, rank == 0, rank == CLUSTER - 1);
                if (some >= 0) offer(row.load_some(some), some, lane == 0);
                for (int q0 = 0; q0 < per_slice; q0 += 32) {
                    const int v = q0 + lane < per_slice ? slice_vec(owner, q0 + lane) : end;
                    Vec<Elem> y;
                    y.none();
                    if (v < end) y.load(x + row.index(v));
                    offer(y, v, v < end);
                }
            }
            __syncthreads();
            if (best.key != 0 && lane < a.top) keep(s_keys, &s_n, best.key);
            __syncthreads();
        }
        rank_keys(s_keys, s_n, a.top, s_best);
    }
    __syncthreads();
    Stats all = s_stats;
    bad = s_bad != 0;
    if (CLUSTER > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        if (rank == 0) {
            all = Stats{-INFINITY, 0.0f, 0.0f};
            bad = false;
            Key least = 0;  // the largest of the CTAs' last keys: at least `top` keys reach it
            for (int r = 0; r < CLUSTER; ++r) {
                const Stats o = *cl.map_shared_rank(&s_stats, r);
                all.join(o.m, o.s, o.w, c);
                bad |= *cl.map_shared_rank(&s_bad, r) != 0;
                if (a.top > 0) least = max(least, cl.map_shared_rank(s_best, r)[a.top - 1]);
            }
            if (a.top > 0) {
                if (tid == 0) s_n = 0;
                __syncthreads();
                for (int i = tid; i < CLUSTER * a.top; i += kThreads) {
                    const Key k = cl.map_shared_rank(s_best, i / a.top)[i % a.top];
                    if (k != 0 && k >= least) s_all[atomicAdd(&s_n, 1)] = k;
                }
                __syncthreads();
                rank_keys(s_all, s_n, a.top, s_keys);  // (s_keys is this CTA's own, no longer read)
                __syncthreads();
                if (tid < a.top) s_best[tid] = s_keys[tid];
            }
        }
        cl.sync();  // no CTA leaves while its sums and keys are read
        if (rank != 0) return;
    }
    // a row without a finite logit has no distribution
    bad |= !(all.m > -INFINITY);
    const float nan = __int_as_float(0x7fc00000), log_s = logf(all.s);
    if (tid == 0) {
        const float xt = static_cast<float>(x[token]);
        a.logprob[t] = bad ? nan : (xt - all.m) * a.inv_t - log_s;
        if (ENTROPY) a.entropy[t] = bad ? nan : log_s - kLn2 * (all.w / all.s);
        a.tok_err[t] = bad ? TSV_DERR_NONFINITE : 0;
    }
    if (tid < a.top) {
        const Key k = s_best[tid];
        a.top_ids[(long long)t * a.top + tid] = bad ? -1 : key_index(k);
        a.top_logprobs[(long long)t * a.top + tid] = bad ? nan : (key_value(k) - all.m) * a.inv_t - log_s;
    }
}

#ifdef TSV_TEST_HOOKS
int g_test_logprobs_cluster = 8;  // test build: the largest cluster that counts as resident
#endif

// Whether a cluster of this size can be resident (a partitioned GPU may not have as many SMs in one
// group); looked up once per device and host thread.
template <typename Elem, int CLUSTER>
bool cluster_fits() {
#ifdef TSV_TEST_HOOKS
    if (CLUSTER > g_test_logprobs_cluster) return false;
#endif
    thread_local int of_dev = -1;
    thread_local bool fits = false;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev != of_dev) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CLUSTER;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(CLUSTER);
        cfg.blockDim = dim3(threads_of(CLUSTER));
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0, n_entropy = 0;
        fits = cudaOccupancyMaxActiveClusters(&n, token_logprobs_kernel<Elem, CLUSTER, false>, &cfg) == cudaSuccess && n > 0 &&
               cudaOccupancyMaxActiveClusters(&n_entropy, token_logprobs_kernel<Elem, CLUSTER, true>, &cfg) == cudaSuccess && n_entropy > 0;
        of_dev = dev;
    }
    return fits;
}

template <typename Elem, int CLUSTER>
cudaError_t launch_rows(const LogprobArgs& a, cudaStream_t stream) {
    const auto kernel = a.entropy ? token_logprobs_kernel<Elem, CLUSTER, true> : token_logprobs_kernel<Elem, CLUSTER, false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(a.T) * CLUSTER), dim3(threads_of(CLUSTER)), 0, stream, static_cast<unsigned>(CLUSTER), a);
}

template <typename Elem, int PER>
cudaError_t launch_short(const LogprobArgs& a, cudaStream_t stream) {
    return launch_pdl(token_logprobs_short_kernel<Elem, PER>, dim3(static_cast<unsigned>((a.T + kShortWarps - 1) / kShortWarps)),
                      dim3(32 * kShortWarps), 0, stream, 1u, a);
}

template <typename Elem>
cudaError_t launch_type(const LogprobArgs& a, int num_sms, cudaStream_t stream) {
    if (a.V <= 64) return launch_short<Elem, 2>(a, stream);
    if (a.V <= 256) return launch_short<Elem, 8>(a, stream);
    if (a.V <= kShortRow) return launch_short<Elem, kShortRow / 32>(a, stream);
    // CTAs a row: as many as still find a place (two an SM) and have a vector for each thread
    const long long vecs = ((long long)a.V + Vec<Elem>::N - 1) / Vec<Elem>::N;
    int n = 1;
    while (n < 8 && 2LL * n * a.T <= 2LL * num_sms && vecs >= 2LL * n * threads_of(2)) n *= 2;
    // (a smaller cluster, or one CTA, where one cannot be resident)
    if (n >= 8 && cluster_fits<Elem, 8>()) return launch_rows<Elem, 8>(a, stream);
    if (n >= 4 && cluster_fits<Elem, 4>()) return launch_rows<Elem, 4>(a, stream);
    if (n >= 2 && cluster_fits<Elem, 2>()) return launch_rows<Elem, 2>(a, stream);
    return launch_rows<Elem, 1>(a, stream);
}

}  // namespace

#ifdef TSV_TEST_HOOKS
// test build only: clusters above this size count as not resident
extern "C" void tsv_test_set_logprobs_cluster(int most) { g_test_logprobs_cluster = most; }
#endif

cudaError_t launch_token_logprobs(const LogprobArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    return bf16 ? launch_type<__nv_bfloat16>(a, num_sms, stream) : launch_type<float>(a, num_sms, stream);
}

}  // namespace tsv
