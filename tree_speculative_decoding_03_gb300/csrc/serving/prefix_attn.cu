// prefix_attn.cu -- attention of one new token per sequence where groups of sequences share the first
// keys of their caches: the shared keys are read once for all rows of the group.
//
//   s_t = scale * q . k_t over t in [0, P) of the group's first sequence and t in [P, L) of the
//   sequence itself;  out = sum_t e^{s_t - m} v_t / l,  m = max s,  l = sum_t e^{s_t - m},  lse = m + ln l.
//
// A softmax over two runs of keys is the join of the two runs' (m, l, O): M = max m_i, O = sum e^{m_i - M}
// O_i, l likewise.  So the prefix of a group, with the rows of all its sequences, and each sequence's own
// keys, with its own rows, are items of one schedule, and the last kernel joins what the pieces of
// both leave.
//
// Kernels: a plan (one CTA: checks, items, running sums of their tiles), the tiles, the join.  For bf16 the kernel of
// the tiles (prefix_tc.cu) has CTAs that take the prefixes to the tensor cores and CTAs for the stream of the sequences' own
// keys; for fp32 it is the stream alone, the prefixes' tiles among the others.  Lengths stay on the device.  An item's units in the stream
// are (group of query rows, kv head); `team` warps take neighbouring kv heads of the same rows and keys
// together.  The tiles of all units, item after item, form one row that is divided evenly between `lanes` teams.  A
// segment that is a whole unit leaves its (m, l, O) at its rows' places, a piece in one of its warp's two slots.
#include <cuda_bf16.h>

#include "../common.cuh"
#include "continue_args.cuh"
#include "prefix_stream.cuh"

namespace tsv {
namespace {

constexpr int kWarps = kStreamWarps / 2;  // of a CTA of the fp32 stream, two on an SM
constexpr int kThreads = 32 * kWarps;
constexpr size_t kSmem = (size_t)kWarps * (kRingBytes + kScratch * sizeof(float));
constexpr int kMaxTeam = kStreamWarps;
constexpr int kPlanThreads = 1024;

// ------------------------------------------------------------------ plan

// Tiles of a prefix on the tensor cores, over all its units.
__device__ __forceinline__ long long tc_tiles(const PrefixArgs& a, const int4& it) {
    return (long long)((it.z + kPrefixTcKeys - 1) / kPrefixTcKeys) * ((it.w + kPrefixTcRows - 1) / kPrefixTcRows) * a.Hkv;
}

// The sum over the block's threads before this one.
__device__ __forceinline__ long long block_before(long long mine, long long* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return incl - mine + (warp ? before : 0);
}

// Lanes that share T tiles: one tile each while there are lanes.
__device__ __forceinline__ int lanes_for(long long T, int lanes) { return T < lanes ? static_cast<int>(T) : lanes; }

// SMs left to the stream while the tensor-core CTAs have the others: both have work that lasts about as
// long.  Times at full load, in us of an SM: a tile of 128 keys and up to 256 rows 2.5 (heads of 128) or 2 (64)
// and a unit 3 more; a tile of the stream 1.4 on one of eight warps and a unit 9 more.  (Two kernels one after the other, each on
// all SMs, and with the division: 64 samples of a 32k prompt 114 and 103 us, 24 ragged groups 154 and 130, 8 samples 23 and 20; 300
// groups of 4 sequences, where the division is off, 356 and 411.  Units at 11 and 13, tiles at 1.2, units of the
// tensor cores at 2 and 4 gain 10 % on one of ten shapes and lose it on another.)
__device__ __forceinline__ int stream_sms(const PrefixArgs& a, long long T, long long tc_T) {
    if (T == 0 || tc_T == 0) return a.tc_lanes;
    const float units = static_cast<float>(a.B) * (a.Hkv / a.team) * ((a.gq + a.rows - 1) / a.rows);
    const float st = (9.0f * units + 1.4f * static_cast<float>(T)) * a.team / kStreamWarps;
    const float tc = (a.D == 128 ? 2.5f : 2.0f) * static_cast<float>(tc_T) + 3.0f * (static_cast<float>(a.G) * a.Hkv + a.tc_lanes);
    const int k = static_cast<int>(a.tc_lanes * st / (st + tc) + 0.5f), idle = tc_T < a.tc_lanes ? a.tc_lanes - static_cast<int>(tc_T) : 0;
    return min(max(max(k, idle), 1), a.tc_lanes - 1);
}

// The last i in [0, n) with start[i] <= x.
__device__ __forceinline__ int last_not_above(const long long* start, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int TILE>
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(16) uint8_t s_plan[];
    const int n = a.G + a.B, per = (n + kPlanThreads - 1) / kPlanThreads;
    int4* s_item = reinterpret_cast<int4*>(s_plan);  // [n] where a thread has one item
    long long* s_start = reinterpret_cast<long long*>(s_item + (per == 1 ? n : 0));  // [n + 1]
    long long* s_tc_start = s_start + n + 1;                                         // [G + 1]
    int* s_off = reinterpret_cast<int*>(s_tc_start + a.G + 1);                       // [G + 1]
    int* s_prefix = reinterpret_cast<int*>(s_tc_start);  // [G], until the sums are written there
    __shared__ long long s_warp[32], s_tc_warp[32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    // (with one item a thread, its length is on its way beside the offsets)
    const int len = per == 1 && tid >= a.G && tid < n ? a.seq_lens[tid - a.G] : 0;
    bool wrong = false;
    for (int g = tid; g <= a.G; g += kPlanThreads) {
        const int x = a.group_offsets[g];
        s_off[g] = x;
        if (g < a.G) s_prefix[g] = a.prefix_lens[g];
        wrong |= x < 0 || x > a.B || (g == 0 && x != 0) || (g == a.G && x != a.B);
    }
    __syncthreads();
    for (int g = tid; g < a.G; g += kPlanThreads) wrong |= s_off[g] > s_off[g + 1];
    wrong = __syncthreads_or(wrong);
    const long long cap = (long long)a.max_blocks << a.bs_log2;
    long long mine = 0, tc_mine = 0;
    int4 last = make_int4(0, 0, 0, 0);
    for (int u = 0; u < per; ++u) {
        const int i = tid * per + u;
        if (i >= n) break;
        int4 it = make_int4(0, 0, 0, 0);
        if (i < a.G) {
            const int P = s_prefix[i];
            if (!wrong && s_off[i + 1] > s_off[i])
                it = make_int4(s_off[i], 0, P > 0 && P <= cap ? P : 0, (s_off[i + 1] - s_off[i]) * a.gq);
        } else {
            const int b = i - a.G, L = per == 1 ? len : a.seq_lens[b];
            int g = 0, e = 0, P = 0;
            if (wrong) {
                e = TSV_DERR_SEQ;
            } else {
                // the last group that begins at or before b and is not empty
                int lo = 0, hi = a.G;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_off[mid] <= b)
                        lo = mid;
                    else
                        hi = mid;
                }
                g = lo;
                P = s_prefix[g];
                if (L < 0 || L > cap || P < 0 || P > L) e = TSV_DERR_CAPACITY;
            }
            it = make_int4(b, e ? 0 : P, e ? 0 : L, a.gq);
            a.group[b] = g;
            a.seq_err[b] = e;
        }
        a.item[i] = it;
        if (per == 1) s_item[i] = it;
        last = it;
        mine += (long long)item_tiles<TILE>(it) * item_units(a, i, it);
        if (i < a.G) tc_mine += tc_tiles(a, it);
    }
    __syncthreads();  // the prefix lengths have been read
    long long at = block_before(mine, s_warp), tc_at = block_before(tc_mine, s_tc_warp);
    for (int u = 0; u < per; ++u) {
        const int i = tid * per + u;
        if (i >= n) break;
        const int4 it = per == 1 ? last : a.item[i];  // (this thread's own)
        const long long end = at + (long long)item_tiles<TILE>(it) * item_units(a, i, it);
        s_start[i] = a.start[i] = at;
        at = end;
        if (i == n - 1) s_start[n] = a.start[n] = at;
        if (i <= a.G) s_tc_start[i] = a.tc_start[i] = tc_at;
        if (i < a.G) tc_at += tc_tiles(a, it);
    }
    __syncthreads();
    // where each lane begins
    const long long T = s_start[n], tc_T = a.tc_lanes > 0 ? s_tc_start[a.G] : 0;
    const int sms = a.tc_lanes > 0 ? stream_sms(a, T, tc_T) : 0;
    const int lanes = lanes_for(T, sms > 0 ? min(a.lanes, kStreamWarps * sms / a.team) : a.lanes);
    const int tc_lanes = lanes_for(tc_T, sms > 0 && T > 0 ? a.tc_lanes - sms : a.tc_lanes);
    if (tid == 0) *a.used = make_int2(lanes, tc_lanes);
    for (int k = tid; k < a.lanes + a.tc_lanes; k += kPlanThreads) {
        const bool tc = k >= a.lanes;
        const int c = tc ? k - a.lanes : k, of = tc ? tc_lanes : lanes;
        const long long all = tc ? tc_T : T;
        int4 p = make_int4(0, 0, 0, 0), it = p;
        int count = 0;
        if (tc && c >= tc_lanes) {  // the stream's: its warps, evenly on the CTAs that have it
            const int warps = (lanes * a.team + a.tc_lanes - tc_lanes - 1) / (a.tc_lanes - tc_lanes);
            p = make_int4((c - tc_lanes) * warps, warps, 0, 0);
        } else if (c < of) {
            const long long x = lane_start(c, all, of);
            count = static_cast<int>(lane_start(c + 1, all, of) - x);
            const int i = last_not_above(tc ? s_tc_start : s_start, tc ? a.G : n, x);
            it = per == 1 ? s_item[i] : a.item[i];
            const long long off = x - (tc ? s_tc_start : s_start)[i];
            const int tiles = tc ? (it.z + kPrefixTcKeys - 1) / kPrefixTcKeys : item_tiles<TILE>(it);
            const int unit = static_cast<int>(off / tiles), t = static_cast<int>(off - (long long)unit * tiles), runs = a.Hkv / a.team;
            p = tc ? make_int4(i, unit, t, count) : make_int4(i, unit / runs, unit % runs, t);
        }
        if (tc) {
            a.tc_begin[2 * c] = p;
            a.tc_begin[2 * c + 1] = it;
        } else {
            a.begin[3 * c] = p;
            a.begin[3 * c + 1] = it;
            a.begin[3 * c + 2] = make_int4(count, 0, 0, 0);
        }
    }
}

// ------------------------------------------------------------------ the stream of tiles, fp32

template <typename Core>
__global__ void __launch_bounds__(kThreads, 2) prefix_stream_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    float* scratch = reinterpret_cast<float*>(smem + kWarps * kRingBytes) + warp * kScratch;
    pdl_wait();
    pdl_launch_dependents();
    stream_tiles<Core>(a, blockIdx.x * kWarps + warp, smem_u32(smem) + warp * kRingBytes, scratch);
}

// ------------------------------------------------------------------ join

// Where the pieces of one row of an item lie.
struct Pieces {
    int n = 0;          // pieces
    long long at = 0;   // row of the first piece, in the whole units' places or in the slots
    long long next = 0; // row of the second piece; the others follow at `step`
    long long step = 0;
    const float *o = nullptr, *m = nullptr, *l = nullptr;  // the array they lie in, and its rows
    long long rows = 0;
};
__device__ __forceinline__ void in_places(const PrefixArgs& a, Pieces& p) {
    p.o = a.whole_o;
    p.m = a.whole_m;
    p.l = a.whole_l;
    p.rows = 3LL * a.B * a.Hq;
}
template <int TILE>
__device__ __forceinline__ Pieces find_pieces(const PrefixArgs& a, int i, int b, int kvh, int j, long long T, int lanes) {
    Pieces p;
    const int4 it = a.item[i];
    const int tiles = item_tiles<TILE>(it);
    if (tiles == 0 || it.w == 0) return p;
    const int x = (b - it.x) * a.gq + j, chunk = x / a.rows, member = kvh % a.team;
    const long long first = a.start[i] + ((long long)chunk * (a.Hkv / a.team) + kvh / a.team) * tiles;
    const int c0 = lane_of_tile(first, T, lanes), c1 = lane_of_tile(first + tiles - 1, T, lanes);
    p.n = c1 - c0 + 1;
    if (c0 == c1) {
        in_places(a, p);
        p.at = (i < a.G ? 0 : (long long)a.B * a.Hq) + (long long)b * a.Hq + kvh * a.gq + j;
    } else {
        const int r = x - chunk * a.rows;
        p.step = 2LL * a.team * a.rows;
        // the piece is the lane's first segment if the lane starts with the unit
        p.at = (2LL * (c0 * a.team + member) + (lane_start(c0, T, lanes) == first ? 0 : 1)) * a.rows + r;
        p.next = 2LL * ((c0 + 1) * a.team + member) * a.rows + r;
        p.o = a.part_o;
        p.m = a.part_m;
        p.l = a.part_l;
        p.rows = 2LL * a.lanes * a.team * a.rows;
    }
    return p;
}
__device__ __forceinline__ const float* of_ptr(const float* p, int lane) {
    return reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}
__device__ __forceinline__ void load_lane(const float* p, float (&x)[4]) {
    const float4 y = *reinterpret_cast<const float4*>(p);
    x[0] = y.x;
    x[1] = y.y;
    x[2] = y.z;
    x[3] = y.w;
}
__device__ __forceinline__ void load_lane(const float* p, float (&x)[2]) {
    const float2 y = *reinterpret_cast<const float2*>(p);
    x[0] = y.x;
    x[1] = y.y;
}
// The pieces of a prefix's row that the tensor-core kernel leaves.  Units of up to 128 rows have two from
// each CTA, one of every other tile; the odd ones are a search of their own (`odd`).
__device__ __forceinline__ Pieces find_tc_pieces(const PrefixArgs& a, int g, int b, int kvh, int j, int lanes, bool odd) {
    Pieces p;
    const int4 it = a.item[g];
    const int tiles = (it.z + kPrefixTcKeys - 1) / kPrefixTcKeys, groups = (it.w + kPrefixTcRows - 1) / kPrefixTcRows;
    if (tiles == 0 || it.w == 0) return p;
    const long long T = a.tc_start[a.G];
    const int x = (b - it.x) * a.gq + j, grp = x / kPrefixTcRows, r = x - grp * kPrefixTcRows;
    const bool by_tile = it.w - grp * kPrefixTcRows <= 128;
    if (odd && !by_tile) return p;
    const long long first = a.tc_start[g] + ((long long)kvh * groups + grp) * tiles;
    const int c0 = lane_of_tile(first, T, lanes), c1 = lane_of_tile(first + tiles - 1, T, lanes);
    p.n = c1 - c0 + 1;
    if (c0 == c1) {
        in_places(a, p);
        p.at = (odd ? 2LL * a.B * a.Hq : 0LL) + (long long)b * a.Hq + kvh * a.gq + j;
    } else {
        const int half = by_tile ? (odd ? 1 : 0) : r >> 7, rl = r & 127;
        p.step = 4 * 128;
        p.at = (4LL * c0 + (lane_start(c0, T, lanes) == first ? 0 : 2) + half) * 128 + rl;
        p.next = (4LL * (c0 + 1) + half) * 128 + rl;
        p.o = a.tc_o;
        p.m = a.tc_m;
        p.l = a.tc_l;
        p.rows = 512LL * a.tc_lanes;
    }
    return p;
}

// `wpr` warps to a query row, eight warps a CTA.  A lane holds the place, m and l of one piece at a time, a warp
// takes up to 32 pieces and then their O together, kJoinAhead rows on their way.  Warps of the same row take
// turns at the pieces and are joined in order, so the result does not depend on timing.  (A thread for
// each output element that looks up and weighs every piece for itself took 49 us where this takes 10: 4096 rows of 12
// pieces.)
constexpr int kJoinThreads = 256, kJoinAhead = 8;

template <typename Elem, int D, int TILE>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ PrefixArgs a, int wpr) {
    constexpr int C = D / 32;  // elements of a lane
    __shared__ float s_part[kJoinThreads / 32][D + 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % wpr;
    const int h = blockIdx.x * (kJoinThreads / 32 / wpr) + warp / wpr;  // query row of all
    const bool in = h < a.B * a.Hq;
    const int b = in ? h / a.Hq : 0, j = in ? (h % a.Hq) % a.gq : 0, kvh = in ? (h % a.Hq) / a.gq : 0;
    pdl_wait();
    pdl_launch_dependents();
    const int err = a.seq_err[b];
    // lane 0 looks up the pieces of the sequence's own keys, 1 those of the prefix, 2 its odd ones
    Pieces mine;
    if (in) {
        const long long T = a.start[a.G + a.B];
        const int2 used = *a.used;
        const int g = a.group[b];
        const bool tc = a.tc_lanes > 0;
        if (lane == 0 || (lane == 1 && !tc))
            mine = find_pieces<TILE>(a, lane == 0 ? a.G + b : g, b, kvh, j, T, used.x);
        else if (lane < 3 && tc)
            mine = find_tc_pieces(a, g, b, kvh, j, used.y, lane == 2);
    }
    float M = -INFINITY, sum = 0.0f, acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.0f;
    if (in && err == 0) {
        const int n0 = __shfl_sync(0xffffffffu, mine.n, 0), n1 = n0 + __shfl_sync(0xffffffffu, mine.n, 1),
                  n = n1 + __shfl_sync(0xffffffffu, mine.n, 2);
        const int run = min(32, (n + wpr - 1) / wpr);  // pieces of a warp's turn
        for (int c0 = run * sub; c0 < n; c0 += run * wpr) {
            const int i = lane < run ? c0 + lane : n, part = i < n0 ? 0 : i < n1 ? 1 : 2, k = i - (part == 0 ? 0 : part == 1 ? n0 : n1);
            auto of = [&](auto x) { return __shfl_sync(0xffffffffu, x, part); };
            const long long at = of(mine.at), next = of(mine.next), step = of(mine.step), rows = of(mine.rows);
            const float *pm = of_ptr(mine.m, part), *pl = of_ptr(mine.l, part), *po = of_ptr(mine.o, part);
            const long long row = k == 0 ? at : next + (k - 1) * step;
            float m = -INFINITY, l = 0.0f;
            if (i < n && TSV_IN_BOUNDS(row, rows, a.seq_err + b)) {
                m = pm[row];
                l = pl[row];
            }
            float m_new = fmaxf(M, m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, o));
            const float ms = safe_max(m_new), f0 = ex2(M - ms), f = ex2(m - ms);
            float add = f * l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
            M = m_new;
            sum = fmaf(sum, f0, add);
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] *= f0;
            // (a piece without tiles, l = 0, leaves no O)
            const float* o = l != 0.0f ? po + row * D : nullptr;
            const int most = min(run, n - c0);
            for (int q = 0; q < most; q += kJoinAhead) {
                float x[kJoinAhead][C], w[kJoinAhead];
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u) {
                    const float* from = of_ptr(o, (q + u) & 31);
                    w[u] = __shfl_sync(0xffffffffu, f, (q + u) & 31);
#pragma unroll
                    for (int c = 0; c < C; ++c) x[u][c] = 0.0f;
                    if (q + u < most && from != nullptr) load_lane(from + lane * C, x[u]);
                }
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u)
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[c] = fmaf(w[u], x[u][c], acc[c]);
            }
        }
    }
    if (wpr > 1) {
#pragma unroll
        for (int c = 0; c < C; ++c) s_part[warp][lane * C + c] = acc[c];
        if (lane == 0) {
            s_part[warp][D] = M;
            s_part[warp][D + 1] = sum;
        }
        __syncthreads();
        if (sub > 0) return;
        for (int w = warp + 1; w < warp + wpr; ++w) {
            const float* s = s_part[w];
            const float m_new = fmaxf(M, s[D]), ms = safe_max(m_new), f0 = ex2(M - ms), f1 = ex2(s[D] - ms);
            M = m_new;
            sum = sum * f0 + s[D + 1] * f1;
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = acc[c] * f0 + s[lane * C + c] * f1;
        }
    }
    if (!in) return;
    const ToResult<Elem, D> to{static_cast<Elem*>(a.out) + (long long)h * D, a.lse ? a.lse + h : nullptr, err != 0};
    // no keys at all: zeros (and an lse of -infinity)
    const float inv = err == 0 && a.seq_lens[b] == 0 ? 0.0f : to.factor(sum);
#pragma unroll
    for (int c = 0; c < C; c += 2) store2(to.base(0) + lane * C + c, acc[c] * inv, acc[c + 1] * inv);
    if (lane == 0) to.row(0, M, sum);
}

constexpr size_t plan_smem(int B, int G) {
    return (G + B <= kPlanThreads ? ((size_t)G + B) * sizeof(int4) : 0) + ((size_t)G + B + 1 + G + 1) * sizeof(long long) + ((size_t)G + 1) * sizeof(int);
}
static_assert(plan_smem(kPagesMaxSeqs, kPagesMaxSeqs) <= 232448 - 1024, "the plan's sums fit an SM's shared memory");

// Sets a kernel's dynamic shared memory once per device and host thread.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, int& of_dev) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev == of_dev) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) of_dev = dev;
    return e;
}

template <typename Core>
cudaError_t launch_stream(const PrefixArgs& a, cudaStream_t stream) {
    thread_local int smem_dev = -1;
    const cudaError_t e = allow_smem(prefix_stream_kernel<Core>, kSmem, smem_dev);
    if (e != cudaSuccess) return e;
    const int warps = a.lanes * a.team;
    return launch_pdl(prefix_stream_kernel<Core>, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), dim3(kThreads), kSmem, stream, 1u, a);
}

template <typename Elem, int D>
cudaError_t launch_kernels(const PrefixArgs& a, cudaStream_t stream) {
    constexpr bool bf16 = sizeof(Elem) == 2;
    constexpr int TILE = tile_keys(bf16, D);
    thread_local int smem_dev = -1;
    cudaError_t e = allow_smem(prefix_plan_kernel<TILE>, plan_smem(kPagesMaxSeqs, kPagesMaxSeqs), smem_dev);
    if (e == cudaSuccess) e = launch_pdl(prefix_plan_kernel<TILE>, dim3(1), dim3(kPlanThreads), plan_smem(a.B, a.G), stream, 1u, a);
    if (e != cudaSuccess) return e;
    if constexpr (bf16)
        e = launch_prefix_tc(a, stream);
    else
        e = a.rows <= 4 ? launch_stream<F32Core<D, 4>>(a, stream) : launch_stream<F32Core<D, 8>>(a, stream);
    if (e != cudaSuccess) return e;
    // warps to a row of the join: more where there are few rows, whose keys then lie in many pieces
    const int rows = a.B * a.Hq, wpr = rows <= 256 ? 8 : rows <= 1024 ? 2 : 1, per = kJoinThreads / 32 / wpr;
    return launch_pdl(prefix_join_kernel<Elem, D, TILE>, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kJoinThreads), 0, stream, 1u,
                      a, wpr);
}

template <int D>
cudaError_t launch_dim(const PrefixArgs& a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_kernels<__nv_bfloat16, D>(a, stream) : launch_kernels<float, D>(a, stream);
}

size_t aligned(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

PrefixPlan make_prefix_plan(int B, int G, int Hq, int Hkv, int D, int block_size, int max_blocks, bool bf16, int num_sms) {
    PrefixPlan p{};
    const int gq = Hq / Hkv;
    // a unit's rows: one or two 16-row fragments (bf16), 4 or 8 (fp32)
    const long long rows = (long long)B * gq;
    // bf16 prefixes go to the tensor cores at any number of rows.  In the stream, whose warp-level products
    // take 32 rows at a time, they are behind from some 16 rows on and ahead by little below: one prefix of
    // 16384 keys, 8 / 16 / 32 / 128 rows of 128: 36 / 36 / 43 / 49 us there, 29 / 38 / 95 / 256 in the stream; 12 of 4096
    // keys: 70 / 71 / 72 / 108 against 168 / 248 / 246 / 878.
    // (one CTA an SM, at least one for the prefixes and one for the stream)
    p.tc_lanes = bf16 ? (num_sms > 1 ? num_sms : 2) : 0;
    p.rows = bf16 ? (gq <= 16 ? 16 : 32) : (rows <= 4 ? 4 : 8);
    p.team = 1;
    for (int t = 2; t <= kMaxTeam; ++t)
        if (Hkv % t == 0) p.team = t;
    // eight warps an SM, as many as the shared memory takes; never more than share the most tiles
    // that the tables can hold
    const int tile = tile_keys(bf16, D);
    const long long cap_tiles = ((long long)max_blocks * block_size + tile - 1) / tile + 1;
    const long long units = (rows / p.rows + G) + (long long)B * ((gq + p.rows - 1) / p.rows);
    long long lanes = (long long)kStreamWarps * num_sms / p.team;
    const long long most = units * (Hkv / p.team) * cap_tiles;
    p.lanes = static_cast<int>(lanes < 1 ? 1 : lanes < most ? lanes : most);
    const size_t slots = 2 * (size_t)p.lanes * p.team * p.rows, whole = 3 * (size_t)B * Hq;
    size_t at = aligned(((size_t)G + B + 1) * sizeof(long long));
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += aligned(bytes);
        return o;
    };
    p.item = take(((size_t)G + B) * sizeof(int4));
    p.group = take((size_t)B * sizeof(int));
    p.part_o = take(slots * D * sizeof(float));
    p.part_m = take(slots * sizeof(float));
    p.part_l = take(slots * sizeof(float));
    p.whole_o = take(whole * D * sizeof(float));
    p.whole_m = take(whole * sizeof(float));
    p.whole_l = take(whole * sizeof(float));
    p.used = take(sizeof(int2));
    p.begin = take((size_t)p.lanes * 3 * sizeof(int4));
    p.tc_begin = take((size_t)p.tc_lanes * 2 * sizeof(int4));
    p.tc_start = take(((size_t)G + 1) * sizeof(long long));
    p.tc_o = take((size_t)p.tc_lanes * 512 * D * sizeof(float));
    p.tc_m = take((size_t)p.tc_lanes * 512 * sizeof(float));
    p.tc_l = take((size_t)p.tc_lanes * 512 * sizeof(float));
    p.ws_bytes = at;
    return p;
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, bool bf16, cudaStream_t stream) {
    return a.D == 64 ? launch_dim<64>(a, bf16, stream) : launch_dim<128>(a, bf16, stream);
}

}  // namespace tsv
