// decode_attn.cu -- attention of one new token per sequence over the paged KV cache, split
// over the cache's length and joined.
//
//   s_t = scale * q . k_t (t < L),  out = sum_t e^{s_t - m} v_t / l,  m = max s,  l = sum_t e^{s_t - m},
//   lse = m + ln l.
// Each K/V row is read once; the Hq / Hkv query rows of a kv head share it (about that many
// multiply-adds per element), so the call is bound by the cache's bytes: 64 sequences of 64/8 heads,
// 1.06 M keys, 4.36 GB in 622 us (7.0 TB/s, 1.03 of the measured copy rate); 13 fp32 sequences, 480 MB in
// 78 us (6.1 TB/s).  Calls of tens of MB spend as long on launch, schedule, first loads and the
// join: 8 sequences of 2048 keys, 67 MB, 20 us.
//
// Work split: a unit is (sequence, kv head, group of query rows).  Its keys are cut into tiles
// of 8 KB (bf16, D = 128: 16 keys).  `team` warps take as many units of one sequence together, each
// warp one unit and all of them the same keys, so neighbouring heads of a cache row, which are
// neighbours in memory, are read at about the same time (4.36 GB: 625 us, 660 without).  The tiles of all teams' units,
// sequence-major, form one row that is divided evenly between `lanes` teams, so every warp
// streams the same bytes whatever the mix of lengths.  A warp goes through its tiles as
// segments, one per unit it touches.  A segment that is a whole unit writes the result; the
// others leave (m, l, O) in a slot of the workspace (a warp has at most two such segments, its
// first and its last), and a second kernel joins them: O = sum_k 2^{m_k - M} O_k, l likewise, in
// the order of the lanes, so a result does not depend on timing.
//
// A warp works for itself: its own ring of tiles in shared memory, filled with asynchronous
// copies that run ahead across segment boundaries, its own running (m, l, O) in registers, and
// no block barrier anywhere.
//
// Joining inside the launch, through the shared memory of a cluster that owns a sequence's units,
// does not pay: 8 sequences of 2048 keys 30.5 us (16 CTAs a cluster) against 20.1, one of 100 keys 9.8
// against 8.3, one of 4096 18.2 against 10.4; it gained only where a sequence is short and there are
// several (16 of 512 keys: 12.8 against 13.8).
#include <cuda_bf16.h>

#include "../common.cuh"
#include "serving_args.cuh"

namespace tsv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRingBytes = 24576;  // of a warp: eight rings and the block's share fill an SM's shared memory
constexpr int kMaxTeam = 8;        // warps of a team
// tiles of a lane, at least: fewer pieces to join when there is little work, more latencies in a
// row (one sequence of 4096 keys with 2 / 3 / 4 / 6 tiles: 11.4 / 12.5 / 10.4 / 14.7 us)
constexpr int kMinTiles = 4;
constexpr int kFewLanes = 64;  // up to here two tiles do (one sequence of 256 fp32 keys 7.9 -> 6.9 us, 16 of 1 to 60 11.6 -> 8.3)
constexpr int kScratch = 136;      // floats of a warp beside its ring

// Keys of a tile: its K and V rows are 8 KB.
__host__ __device__ constexpr int tile_keys(bool bf16, int D) { return 4096 / (D * (bf16 ? 2 : 4)); }

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes to shared memory; `take` false writes zeros and reads nothing
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c (16 x 8, fp32) += a (16 x 16, bf16) * b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// Two weights (0 or normal numbers) as the sum of two bf16 each.  hi is the next bf16 below the
// weight, so lo = w - hi is exact in fp32 and positive, and rounded to at most 2^-8 of itself; a
// positive weight has two positive parts, which keep an infinite value infinite (0 or a sign change
// would make it NaN).
__device__ __forceinline__ void split_bf16(float w0, float w1, uint32_t* hi, uint32_t* lo) {
    const uint32_t h0 = max(__float_as_uint(w0), 1u) - 1u, h1 = max(__float_as_uint(w1), 1u) - 1u;
    *hi = __byte_perm(h0, h1, 0x7632);
    *lo = pack_bf16(w0 - __uint_as_float(h0 & 0xffff0000u), w1 - __uint_as_float(h1 & 0xffff0000u));
}
// the reference point of the exponentials; a row that has seen only -inf scores keeps P = 0
__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.0f : m; }

// ------------------------------------------------------------------ the two element types
// A warp's part of a tile, and the running state of its query rows.

// bf16: products on the tensor cores, 16 rows a fragment (MT fragments).  With at most 16 rows
// per K/V row the tensor rate is far from a limit (about 280 multiply-adds a clock and SM at
// full memory speed), so the warp-level product serves.  The second product takes each weight as
// two bf16 parts, hi + lo, so a weight is off by at most 2^-15 of itself and the result by little
// but its own rounding.  (One part alone is off by up to 2^-8, an error as large as the result's
// rounding at any number of keys.  The second part's products take: 64 sequences of 64/8 heads 620 -> 622
// us, 8 of 32/8 heads 19.9 -> 20.3, 32 of 64/1 heads 43.9 -> 48.4.)
template <int D_, int MT>
struct Bf16Core {
    static constexpr int D = D_, KEYS = tile_keys(true, D_), ROWB = D * 2, CH = ROWB / 16, NF = KEYS / 8;
    using Elem = __nv_bfloat16;
    uint32_t qf[MT][D / 16][4];
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];

    // chunk c (16 bytes) of a row sits at c ^ (row & 7): the 8 rows of a fragment load use
    // different banks
    static __device__ __forceinline__ uint32_t place(int row, int c) { return row * ROWB + ((c ^ (row & 7)) << 4); }

    // loads a unit's query rows (the running state is untouched: this runs ahead of reset)
    __device__ __forceinline__ void load_q(const Elem* q, int nrows) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r0 = 16 * t + (lane >> 2), r1 = r0 + 8, c = (lane & 3) * 2;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const Elem* p = q + kk * 16 + c;
                qf[t][kk][0] = r0 < nrows ? *reinterpret_cast<const uint32_t*>(p + r0 * D) : 0u;
                qf[t][kk][1] = r1 < nrows ? *reinterpret_cast<const uint32_t*>(p + r1 * D) : 0u;
                qf[t][kk][2] = r0 < nrows ? *reinterpret_cast<const uint32_t*>(p + r0 * D + 8) : 0u;
                qf[t][kk][3] = r1 < nrows ? *reinterpret_cast<const uint32_t*>(p + r1 * D + 8) : 0u;
            }
        }
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
        }
    }

    // `live` of the tile's keys exist
    __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, int live, float sl2, float*) {
        const int lane = threadIdx.x & 31;
        float s[MT][NF][4];  // 8 keys a fragment
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NF; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.0f;
        {
            const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
                for (int n = 0; n < NF; n += 2) {
                    uint32_t b[4];
                    ldsm4(b, ks + place(8 * n + row, 2 * kk + ((lane >> 3) & 1)));
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma16816(s[t][n], qf[t][kk], b[0], b[1]);
                        mma16816(s[t][n + 1], qf[t][kk], b[2], b[3]);
                    }
                }
            }
        }
        const int k0 = (lane & 3) * 2;
        uint32_t p[MT][NF / 2][4], p_lo[MT][NF / 2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (live < KEYS) {
#pragma unroll
                for (int n = 0; n < NF; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * n + k0 + (e & 1) >= live) s[t][n][e] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(s[t][0][2 * r], s[t][0][2 * r + 1]);
#pragma unroll
                for (int n = 1; n < NF; ++n) mx = fmaxf(mx, fmaxf(s[t][n][2 * r], s[t][n][2 * r + 1]));
                mx *= sl2;
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m[t][r], mx);
                const float ms = safe_max(m_new);
                if (__any_sync(0xffffffffu, m_new > m[t][r])) {
                    const float f = ex2(m[t][r] - ms);
                    l[t][r] *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[t][i][2 * r] *= f;
                        o[t][i][2 * r + 1] *= f;
                    }
                }
                m[t][r] = m_new;
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < NF; ++n) {
                    const float w0 = ex2(fmaf(s[t][n][2 * r], sl2, -ms)), w1 = ex2(fmaf(s[t][n][2 * r + 1], sl2, -ms));
                    sum += w0 + w1;
                    split_bf16(w0, w1, &p[t][n / 2][2 * (n & 1) + r], &p_lo[t][n / 2][2 * (n & 1) + r]);
                }
                l[t][r] += sum;
            }
        }
        {
            const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
            for (int n = 0; n < NF / 2; ++n) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];
                    ldsm4_t(b, vs + place(16 * n + row, 2 * i + (lane >> 4)));
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma16816(o[t][2 * i], p_lo[t][n], b[0], b[1]);
                        mma16816(o[t][2 * i + 1], p_lo[t][n], b[2], b[3]);
                        mma16816(o[t][2 * i], p[t][n], b[0], b[1]);
                        mma16816(o[t][2 * i + 1], p[t][n], b[2], b[3]);
                    }
                }
            }
        }
    }

    // hands each row's (row, m, l) and pieces of its O to the sink
    template <typename Sink>
    __device__ __forceinline__ void finish(int nrows, Sink sink, float*) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[t][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int row = 16 * t + 8 * r + (lane >> 2);
                if (row >= nrows) continue;
                if ((lane & 3) == 0) sink.row(row, m[t][r], sum);
                const float inv = sink.factor(sum);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) sink.two(row, 8 * i + (lane & 3) * 2, o[t][i][2 * r] * inv, o[t][i][2 * r + 1] * inv);
            }
    }
};

// fp32: multiply-adds on the FMA pipe.  Up to 8 rows a unit it follows memory (1 row 94 % of the
// copy rate, 4 rows 91 %, 8 rows 79 %); 16 rows are two units that read the keys twice.  Pairs of
// multiply-adds to an instruction, and 16 rows to a unit, took as long (16 rows: 201 us against
// 198; 8 rows: 52 against 51).  For the scores 8 dimensions of each row sit in a lane,
// D / 8 lanes a key, and the lanes' sums are exchanged so that each ends with one row's score;
// for the second product a lane owns D / 32 dimensions of all rows and the weights come from
// shared memory.
template <int D_, int RR>
struct F32Core {
    static constexpr int D = D_, KEYS = tile_keys(false, D_), ROWB = D * 4, CH = ROWB / 16;
    static constexpr int LPK = D / 8, KPP = 32 / LPK, PASSES = KEYS / KPP, DV = D / 32;
    using Elem = float;
    float qr[RR][8];
    float o[RR][DV];
    float m, l;  // of the row this lane ends with, l over the keys this lane saw

    static __device__ __forceinline__ uint32_t place(int row, int c) { return row * ROWB + (c << 4); }
    // the row whose score a lane ends with: the lane bits, from the highest of the key's lanes down
    static __device__ __forceinline__ int my_row() {
        const int i = (threadIdx.x & 31) % LPK;
        int row = 0;
#pragma unroll
        for (int n = RR, x = LPK / 2; n > 1; n >>= 1, x >>= 1) row = row * 2 + ((i & x) ? 1 : 0);
        return row;
    }

    __device__ __forceinline__ void load_q(const Elem* q, int nrows) {
        const int i = (threadIdx.x & 31) % LPK;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = r < nrows ? *reinterpret_cast<const float4*>(q + r * D + (i + h * LPK) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                qr[r][4 * h] = x.x;
                qr[r][4 * h + 1] = x.y;
                qr[r][4 * h + 2] = x.z;
                qr[r][4 * h + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int d = 0; d < DV; ++d) o[r][d] = 0.0f;
        m = -INFINITY;
        l = 0.0f;
    }

    __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, int live, float sl2, float* scratch) {
        const int lane = threadIdx.x & 31, i = lane % LPK;
        float sc[PASSES];
#pragma unroll
        for (int ps = 0; ps < PASSES; ++ps) {
            const int key = ps * KPP + lane / LPK;
            float k[8];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(k[0]), "=f"(k[1]), "=f"(k[2]), "=f"(k[3]) : "r"(ks + place(key, i)) : "memory");
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(k[4]), "=f"(k[5]), "=f"(k[6]), "=f"(k[7]) : "r"(ks + place(key, i + LPK)) : "memory");
            float v[RR];
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                float x = 0.0f;
#pragma unroll
                for (int d = 0; d < 8; ++d) x = fmaf(qr[r][d], k[d], x);
                v[r] = x;
            }
            // half of the rows go to the partner lane, half stay, until one is left
            int x = LPK / 2;
#pragma unroll
            for (int n = RR; n > 1; n >>= 1, x >>= 1) {
                const bool up = (i & x) != 0;
#pragma unroll
                for (int r = 0; r < n / 2; ++r) {
                    const float give = up ? v[r] : v[r + n / 2];
                    const float keep = up ? v[r + n / 2] : v[r];
                    v[r] = keep + __shfl_xor_sync(0xffffffffu, give, x);
                }
            }
#pragma unroll
            for (int y = LPK / (2 * RR); y > 0; y >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], y);
            sc[ps] = key < live ? v[0] * sl2 : -INFINITY;
        }
        float mx = sc[0];
#pragma unroll
        for (int ps = 1; ps < PASSES; ++ps) mx = fmaxf(mx, sc[ps]);
#pragma unroll
        for (int y = LPK; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float m_new = fmaxf(m, mx), ms = safe_max(m_new);
        const float f = ex2(m - ms);
        const bool moved = __any_sync(0xffffffffu, m_new > m);
        m = m_new;
        l *= f;
        const int row = my_row();
        float* sw = scratch;               // [KEYS][RR]
        float* sf = scratch + KEYS * RR;   // [RR]
        if (i % (LPK / RR) == 0) {
#pragma unroll
            for (int ps = 0; ps < PASSES; ++ps) {
                const float w = ex2(sc[ps] - ms);
                l += w;
                sw[(ps * KPP + lane / LPK) * RR + row] = w;
            }
            if (lane < LPK) sf[row] = f;
        }
        __syncwarp();
        if (moved) {
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const float g = sf[r];
#pragma unroll
                for (int d = 0; d < DV; ++d) o[r][d] *= g;
            }
        }
#pragma unroll
        for (int key = 0; key < KEYS; ++key) {
            float v[DV];
            if (DV == 4)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[DV - 2]), "=f"(v[DV - 1]) : "r"(vs + key * ROWB + lane * 16) : "memory");
            else
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(vs + key * ROWB + lane * 8) : "memory");
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const float w = sw[key * RR + r];
#pragma unroll
                for (int d = 0; d < DV; ++d) o[r][d] = fmaf(w, v[d], o[r][d]);
            }
        }
        __syncwarp();
    }

    template <typename Sink>
    __device__ __forceinline__ void finish(int nrows, Sink sink, float* scratch) {
        const int lane = threadIdx.x & 31, i = lane % LPK;
        float sum = l;
#pragma unroll
        for (int y = LPK; y < 32; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        if (lane < LPK && i % (LPK / RR) == 0) {
            const int row = my_row();
            scratch[row] = sum;
            if (row < nrows) sink.row(row, m, sum);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            if (r >= nrows) continue;
            const float inv = sink.factor(scratch[r]);
#pragma unroll
            for (int d = 0; d < DV; d += 2) sink.two(r, lane * DV + d, o[r][d] * inv, o[r][d + 1] * inv);
        }
        __syncwarp();
    }
};

// ------------------------------------------------------------------ the schedule

// Keys of sequence b that are attended to: 0 when its length does not fit the block table.
// (AHEAD: read before the wait for the kernel before, past the L1 cache.)  Lengths and block ids are
// read with ordinary loads, here and below: an earlier kernel may write them while this one is
// already resident, which the read-only path does not allow.
template <bool AHEAD = false>
__device__ __forceinline__ int seq_keys(const DecodeArgs& a, int b) {
    const int L = AHEAD ? __ldcg(a.seq_lens + b) : a.seq_lens[b];
    return (L < 0 || (long long)L > ((long long)a.max_blocks << a.bs_log2)) ? 0 : L;
}

__device__ __forceinline__ long long lane_start(int k, long long T, int lanes) { return (long long)k * T / lanes; }
__device__ __forceinline__ int lane_of_tile(long long x, long long T, int lanes) {
    return static_cast<int>(((x + 1) * lanes - 1) / T);
}

// Lanes that share T tiles.
__host__ __device__ __forceinline__ int lanes_of(long long T, int lanes) {
    const long long few = T / 2 < kFewLanes ? T / 2 : kFewLanes, n = T / kMinTiles > few ? T / kMinTiles : few;
    return n < 1 ? 1 : n < lanes ? static_cast<int>(n) : lanes;
}

// A position in the row of tiles: tile t of the `tiles` of unit `unit` of sequence b, which has
// `keys` keys.  A team's warps differ in the unit alone.
struct Place {
    int b, unit, t, tiles, keys;
    template <int TILE>
    __device__ __forceinline__ void next(const DecodeArgs& a) {
        if (++t < tiles) return;
        t = 0;
        unit += a.team;
        const int units = a.Hkv * a.groups;
        if (unit < units) return;
        unit -= units;
        do {
            ++b;
            keys = b < a.B ? seq_keys(a, b) : 1;
        } while (keys == 0);
        tiles = (keys + TILE - 1) / TILE;
    }
};

// One warp: the tiles [x, x_end) of lane `which` and where x lies, for the team's warp `member`;
// T = all tiles.
template <int TILE>
__device__ __forceinline__ Place locate(const DecodeArgs& a, int which, int member, long long* x_, long long* x_end, long long* T_) {
    const int lane = threadIdx.x & 31, units = a.Hkv * a.groups / a.team;
    // a run of sequences to each lane: their tiles, then a scan over the lanes
    const int run = (a.B + 31) >> 5;
    long long mine = 0;
    int keys0 = 0;
    for (int j = 0; j < run; ++j) {
        const int b = lane * run + j;
        const int keys = b < a.B ? seq_keys(a, b) : 0;
        if (j == 0) keys0 = keys;
        mine += (keys + TILE - 1) / TILE;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const long long T = __shfl_sync(0xffffffffu, incl, 31) * units;
    const int lanes = lanes_of(T, a.lanes);
    const long long x = which < lanes ? lane_start(which, T, lanes) : T;
    *x_ = x;
    *x_end = which < lanes ? lane_start(which + 1, T, lanes) : T;
    *T_ = T;
    Place p{0, 0, 0, 1, 0};
    if (x >= T) return p;
    const unsigned holds = __ballot_sync(0xffffffffu, (incl - mine) * units <= x && x < incl * units);
    const int owner = __ffs(holds) - 1;
    long long base = __shfl_sync(0xffffffffu, incl - mine, owner) * units;
    for (int j0 = 0; j0 < run; j0 += 32) {
        const int b = owner * run + j0 + lane;
        const bool in = j0 + lane < run && b < a.B;
        const int keys = run == 1 ? __shfl_sync(0xffffffffu, keys0, owner) : (in ? seq_keys(a, b) : 0);
        const int tiles = in ? (keys + TILE - 1) / TILE : 0;
        const long long w = (long long)tiles * units;
        long long end = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        end += base;
        const unsigned hit = __ballot_sync(0xffffffffu, end - w <= x && x < end);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const long long off = x - __shfl_sync(0xffffffffu, end - w, src);
            p.b = owner * run + j0 + src;
            p.tiles = __shfl_sync(0xffffffffu, tiles, src);
            p.keys = __shfl_sync(0xffffffffu, keys, src);
            p.unit = static_cast<int>(off / p.tiles);
            p.t = static_cast<int>(off - (long long)p.unit * p.tiles);
            p.unit = p.unit * a.team + member;
            break;
        }
        base = __shfl_sync(0xffffffffu, end, 31);
    }
    return p;
}

// One warp: where the pieces of unit `record` (of all units) lie, as the main kernel leaves them:
// sequence, unit, last lane (-1: in one piece, or no keys) and first slot.
template <int TILE>
__device__ __forceinline__ int4 unit_pieces(const DecodeArgs& a, int record) {
    const int lane = threadIdx.x & 31, units = a.Hkv * a.groups, b = record / units, unit = record % units;
    long long T = 0, first = 0;
    for (int i = lane; i < a.B; i += 32) {
        const int tiles = (seq_keys<true>(a, i) + TILE - 1) / TILE;
        T += tiles;
        first += i < b ? tiles : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        T += __shfl_xor_sync(0xffffffffu, T, o);
        first += __shfl_xor_sync(0xffffffffu, first, o);
    }
    const int tiles = (seq_keys<true>(a, b) + TILE - 1) / TILE, per_seq = units / a.team;
    T *= per_seq;
    first = first * per_seq + (long long)(unit / a.team) * tiles;
    if (tiles == 0) return make_int4(b, unit, -1, 0);
    const int lanes = lanes_of(T, a.lanes);
    const int c0 = lane_of_tile(first, T, lanes), c1 = lane_of_tile(first + tiles - 1, T, lanes);
    if (c0 == c1) return make_int4(b, unit, -1, 0);
    // the piece is the lane's first segment if the lane starts with the unit
    return make_int4(b, unit, c1, 2 * (c0 * a.team + unit % a.team) + (lane_start(c0, T, lanes) == first ? 0 : 1));
}

template <typename T>
__device__ __forceinline__ T to_elem(float x);
template <>
__device__ __forceinline__ float to_elem<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr float kLn2 = 0.69314718055994530942f;

// Where a segment's rows go: the result (a whole unit), or a slot of the workspace.
template <typename Elem, int D>
struct ToResult {
    Elem* out;   // the unit's first row
    float* lse;  // or nullptr
    bool bad;    // a block id outside the cache: NaN
    __device__ __forceinline__ void row(int r, float m, float l) const {
        if (lse != nullptr) lse[r] = bad ? __int_as_float(0x7fc00000) : (m + log2f(l)) * kLn2;
    }
    __device__ __forceinline__ float factor(float l) const { return bad ? __int_as_float(0x7fc00000) : 1.0f / l; }
    __device__ __forceinline__ void two(int r, int d, float x, float y) const { store2(out + r * D + d, x, y); }
    // the one rounding of the result
    static __device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
    static __device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16(x, y);
    }
};
template <int D>
struct ToSlot {
    float *o, *m, *l;  // of the slot
    __device__ __forceinline__ void row(int r, float m_, float l_) const {
        m[r] = m_;
        l[r] = l_;
    }
    __device__ __forceinline__ float factor(float) const { return 1.0f; }
    __device__ __forceinline__ void two(int r, int d, float x, float y) const {
        *reinterpret_cast<float2*>(o + r * D + d) = make_float2(x, y);
    }
};

template <typename Core>
__host__ __device__ constexpr int stages_of() { return kRingBytes / (2 * Core::KEYS * Core::ROWB); }
constexpr size_t kDecodeSmem = (size_t)kWarps * (kRingBytes + kScratch * sizeof(float));

// A warp's stream of tiles: the copies run STAGES - 1 tiles ahead and the block ids one more.
template <typename Core>
struct Stream {
    using Elem = typename Core::Elem;
    static constexpr int D = Core::D, KEYS = Core::KEYS, STAGES = stages_of<Core>(), RUNS = KEYS / 8;
    static constexpr uint32_t HALF = KEYS * Core::ROWB, STAGE = 2 * HALF;
    static constexpr int LANES_ROW = Core::CH < 32 ? Core::CH : 32, ROWS_IT = 32 / LANES_ROW;
    const DecodeArgs& a;
    const uint32_t ring;
    const int row_elems, lrow, lch, lane_elems;
    Place f;           // the tile whose ids were fetched last
    int ids[RUNS];     // its blocks (8 keys lie in one block); all lanes hold the same
    uint32_t bad = 0;  // stages holding a tile with a block id outside the cache
    int left;          // tiles not yet on their way
    int fill = 0, stage = 0;

    __device__ __forceinline__ Stream(const DecodeArgs& args, uint32_t ring_, const Place& p, int n)
        : a(args), ring(ring_), row_elems(args.Hkv * D), lrow((threadIdx.x & 31) / LANES_ROW), lch((threadIdx.x & 31) % LANES_ROW),
          lane_elems(lrow * row_elems + lch * (16 / (int)sizeof(Elem))), f(p), left(n) {}

    __device__ __forceinline__ void fetch() {
        const int32_t* bt = a.block_table + (long long)f.b * a.max_blocks;
#pragma unroll
        for (int u = 0; u < RUNS; ++u) {
            const int key = f.t * KEYS + 8 * u;
            ids[u] = key < f.keys ? (TSV_IN_BOUNDS(key >> a.bs_log2, a.max_blocks, nullptr) ? bt[key >> a.bs_log2] : -1) : 0;
        }
    }
    // sends tile f on its way into stage `fill`, then fetches the next tile's ids
    __device__ __forceinline__ void load() {
        if (left > 0) {
            const uint32_t dst = ring + fill * STAGE;
            const Elem* kc = static_cast<const Elem*>(a.k_cache);
            const Elem* vc = static_cast<const Elem*>(a.v_cache);
            const long long head = (long long)(f.unit / a.groups) * D + lane_elems;
            bool wrong = false;
#pragma unroll
            for (int u = 0; u < RUNS; ++u) {
                const int key = f.t * KEYS + 8 * u;
                const bool in = static_cast<unsigned>(ids[u]) < static_cast<unsigned>(a.num_blocks);
                wrong |= !in && key < f.keys;
                const long long at = head + (((long long)(in ? ids[u] : 0) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))) * row_elems;
#pragma unroll
                for (int r0 = 0; r0 < 8; r0 += ROWS_IT) {
                    bool take = in && key + r0 + lrow < f.keys;
                    const long long off = take ? at + (long long)r0 * row_elems : 0;
                    // (an index check that fails is reported as a bad block)
                    if (!TSV_IN_BOUNDS(off + 16 / (int)sizeof(Elem) - 1, ((long long)a.num_blocks << a.bs_log2) * row_elems, nullptr))
                        wrong = true, take = false;
                    cp16(dst + Core::place(8 * u + r0 + lrow, lch), kc + off, take);
                    cp16(dst + HALF + Core::place(8 * u + r0 + lrow, lch), vc + off, take);
                }
            }
            bad = (bad & ~(1u << fill)) | (wrong ? 1u << fill : 0u);
            if (--left > 0) {
                f.next<KEYS>(a);
                fetch();
            }
        }
        cp_commit();
        if (++fill == STAGES) fill = 0;
    }
    __device__ __forceinline__ void begin() {
        if (left > 0) fetch();
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) load();
    }
    // the next tile: waits for it, keeps the copies ahead, adds it to the core's state
    __device__ __forceinline__ bool step(Core& core, int live, float* scratch) {
        cp_wait<STAGES - 2>();
        __syncwarp();
        load();
        const uint32_t src = ring + stage * STAGE;
        const bool wrong = ((bad >> stage) & 1u) != 0;
        core.step(src, src + HALF, live, a.scale_log2, scratch);
        __syncwarp();
        if (++stage == STAGES) stage = 0;
        return wrong;
    }
};

template <typename Elem>
__device__ __forceinline__ const Elem* q_of(const DecodeArgs& a, int D, const Place& u) {
    return static_cast<const Elem*>(a.q) + ((long long)u.b * a.Hq + (u.unit / a.groups) * a.G + (u.unit % a.groups) * a.rows) * D;
}
__device__ __forceinline__ int rows_of(const DecodeArgs& a, int unit) { return min(a.rows, a.G - (unit % a.groups) * a.rows); }
__device__ __forceinline__ long long first_head(const DecodeArgs& a, int b, int unit) {
    return (long long)b * a.Hq + (unit / a.groups) * a.G + (unit % a.groups) * a.rows;
}

template <typename Core>
__global__ void __launch_bounds__(kThreads, 2) decode_attn_kernel(const __grid_constant__ DecodeArgs a) {
    using Elem = typename Core::Elem;
    constexpr int D = Core::D, KEYS = Core::KEYS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
    float* scratch = reinterpret_cast<float*>(smem + kWarps * kRingBytes) + warp * kScratch;
    pdl_wait();
    pdl_launch_dependents();
    // sequences without keys: nothing to attend to (zeros), or a length that does not fit (NaN)
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (seq_keys(a, b) > 0) continue;
        const bool empty = a.seq_lens[b] == 0;
        const float x = empty ? 0.0f : __int_as_float(0x7fc00000);
        Elem* out = static_cast<Elem*>(a.out) + (long long)b * a.Hq * D;
        for (int i = tid; i < a.Hq * D; i += kThreads) out[i] = to_elem<Elem>(x);
        if (a.lse != nullptr)
            for (int h = tid; h < a.Hq; h += kThreads) a.lse[(long long)b * a.Hq + h] = empty ? -INFINITY : x;
        if (tid == 0) a.seq_err[b] = empty ? 0 : TSV_DERR_CAPACITY;
    }
    const int me = blockIdx.x * kWarps + warp;
    const int lane_me = me / a.team;
    if (lane_me >= a.lanes) return;
    long long x, x_end, T;
    Place p = locate<KEYS>(a, lane_me, me % a.team, &x, &x_end, &T);
    // for the join: a unit's last lane, where this lane leaves its first piece
    int4 left = make_int4(0, 0, -1, 0);
    const int n = static_cast<int>(x_end - x);
    Stream<Core> stream(a, ring, p, n);
    stream.begin();
    Core core;
    if (n > 0) {
        core.load_q(q_of<Elem>(a, D, p), rows_of(a, p.unit));
        core.reset();
    }
    bool seg_bad = false;
    int seg = 0, t_first = p.t;
    for (int i = 0; i < n; ++i) {
        seg_bad |= stream.step(core, p.keys - p.t * KEYS, scratch);
        if (p.t + 1 < p.tiles && i + 1 < n) {
            ++p.t;
            continue;
        }
        // the segment's end
        const int nrows = rows_of(a, p.unit);
        if (t_first == 0 && p.t + 1 == p.tiles) {
            const long long h = first_head(a, p.b, p.unit);
            core.finish(nrows, ToResult<Elem, D>{static_cast<Elem*>(a.out) + h * D, a.lse ? a.lse + h : nullptr, seg_bad}, scratch);
            if (p.unit == 0 && lane == 0) a.seq_err[p.b] = seg_bad ? TSV_DERR_BLOCK : 0;
        } else {
            const long long slot = 2LL * me + (seg == 0 ? 0 : 1);
            if (!TSV_IN_BOUNDS(slot, 2LL * a.lanes * a.team, a.seq_err + p.b)) return;
            core.finish(nrows, ToSlot<D>{a.part_o + slot * a.rows * D, a.part_m + slot * a.rows, a.part_l + slot * a.rows}, scratch);
            if (lane == 0) a.part_bad[slot] = seg_bad;
            if (t_first == 0)
                left = make_int4(p.b, p.unit, lane_of_tile(x + i - p.t + p.tiles - 1, T, lanes_of(T, a.lanes)), static_cast<int>(slot));
        }
        if (i + 1 < n) {
            p.next<KEYS>(a);
            t_first = 0;
            seg_bad = false;
            ++seg;
            core.load_q(q_of<Elem>(a, D, p), rows_of(a, p.unit));
            core.reset();
        }
    }
    if (!a.by_unit && lane == 0) a.split[me] = left;
}

// Joins the pieces of the units that lie on more than one lane, in lane order.  CTA k joins the
// k-th unit, or the unit whose first piece warp k has left, whichever are fewer: ROWS query rows at a
// time, GROUPS threads to an output element, each with kAhead pieces in flight.  With many pieces a
// unit, 4 to 16 threads share an element's pieces and blockIdx.y divides the rows; with few, small
// CTAs go through all rows.  Time of a call with 1, 4 and 8 threads: 0.6 pieces a unit 32 / - / 46
// us; 9.5 pieces 14.2 / - / 16.2; 11.7 pieces 85.6 / 77.7 / 79.4; 19 pieces 59.7 / 50.2 / 52.9; 64
// pieces - / 12.5 / 10.4; 304 pieces - / - / 28.5, with 16 threads 22.2.
template <typename Elem, int D, int KEYS, int GROUPS, int ROWS>
__global__ void __launch_bounds__(ROWS* GROUPS* D / 4) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int kAhead = 8, VEC = D / 4;
    __shared__ float s_part[GROUPS > 1 ? GROUPS - 1 : 1][ROWS * VEC][6];
    // With a record per unit the schedule is worked out here, from the lengths, which the kernel
    // before this one has waited for before it let this one start: so the pieces are known when
    // the wait ends.
    int4 sp = make_int4(0, 0, -1, 0);
    if (a.by_unit) sp = unit_pieces<KEYS>(a, blockIdx.x);
    pdl_wait();
    pdl_launch_dependents();
    if (!a.by_unit) sp = a.split[blockIdx.x];
    if (sp.z < 0) return;
    const int first_warp = sp.w >> 1, member = first_warp % a.team, k = first_warp / a.team, last = sp.z;
    const int b = sp.x, unit = sp.y;
    const int row0 = (unit % a.groups) * a.rows, nrows = min(a.rows, a.G - row0);
    const int e = threadIdx.x % (ROWS * VEC), grp = threadIdx.x / (ROWS * VEC), d = (e % VEC) * 4;
    for (int r0 = blockIdx.y * ROWS; r0 < nrows; r0 += gridDim.y * ROWS) {
        const int r = r0 + e / VEC;
        if (GROUPS > 1 && r0 > static_cast<int>(blockIdx.y) * ROWS) __syncthreads();  // the last round's sums have been read
        float M = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int bad = 0;
        for (int c = k + grp * kAhead; c <= last; c += kAhead * GROUPS) {
            float m[kAhead], l[kAhead];
            float4 o[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.0f;
                o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c + i <= last && r < nrows) {
                    const long long slot = 2LL * ((c + i) * a.team + member) + (c + i == k ? sp.w & 1 : 0), pr = slot * a.rows + r;
                    m[i] = a.part_m[pr];
                    l[i] = a.part_l[pr];
                    o[i] = *reinterpret_cast<const float4*>(a.part_o + pr * D + d);
                    bad |= a.part_bad[slot];
                }
            }
            float m_new = M;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) m_new = fmaxf(m_new, m[i]);
            const float ms = safe_max(m_new);
            const float f0 = ex2(M - ms);
            M = m_new;
            sum *= f0;
            acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float f = ex2(m[i] - ms);
                sum = fmaf(f, l[i], sum);
                acc = make_float4(fmaf(f, o[i].x, acc.x), fmaf(f, o[i].y, acc.y), fmaf(f, o[i].z, acc.z), fmaf(f, o[i].w, acc.w));
            }
        }
        if (grp > 0) {
            float* s = s_part[grp - 1][e];
            s[0] = M;
            s[1] = sum;
            s[2] = acc.x;
            s[3] = acc.y;
            s[4] = acc.z;
            s[5] = acc.w;
        }
        if (GROUPS > 1) bad = __syncthreads_or(bad);
        if (grp > 0 || r >= nrows) continue;
#pragma unroll
        for (int i = 0; i < GROUPS - 1; ++i) {
            const float* s = s_part[i][e];
            const float m_new = fmaxf(M, s[0]), ms = safe_max(m_new);
            const float f0 = ex2(M - ms), f1 = ex2(s[0] - ms);
            M = m_new;
            sum = sum * f0 + s[1] * f1;
            acc = make_float4(acc.x * f0 + s[2] * f1, acc.y * f0 + s[3] * f1, acc.z * f0 + s[4] * f1, acc.w * f0 + s[5] * f1);
        }
        const long long h = (long long)b * a.Hq + (unit / a.groups) * a.G + row0 + r;
        const ToResult<Elem, D> to{static_cast<Elem*>(a.out) + h * D, a.lse ? a.lse + h : nullptr, bad != 0};
        const float inv = to.factor(sum);
        to.two(0, d, acc.x * inv, acc.y * inv);
        to.two(0, d + 2, acc.z * inv, acc.w * inv);
        if (d == 0) to.row(0, M, sum);
        if (d == 0 && r == 0 && unit == 0) a.seq_err[b] = bad ? TSV_DERR_BLOCK : 0;
    }
}

template <typename Core>
cudaError_t launch_core(const DecodeArgs& a, cudaStream_t stream) {
    thread_local int smem_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != smem_dev) {
        constexpr int smem = static_cast<int>(kDecodeSmem);
        e = cudaFuncSetAttribute(decode_attn_kernel<Core>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        smem_dev = dev;
    }
    const int warps = a.lanes * a.team;
    e = launch_pdl(decode_attn_kernel<Core>, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), dim3(kThreads),
                   kDecodeSmem, stream, 1u, a);
    if (e != cudaSuccess || a.lanes < 2) return e;
    using Elem = typename Core::Elem;
    constexpr int D = Core::D;
    const int all = a.B * a.Hkv * a.groups;  // units
    const unsigned records = static_cast<unsigned>(a.by_unit ? all : warps - a.team);
    const dim3 by_row(records, static_cast<unsigned>(min(a.rows, a.G)));
    if (warps >= 96LL * all) return launch_pdl(decode_join_kernel<Elem, D, Core::KEYS, 16, 1>, by_row, dim3(16 * D / 4), 0, stream, 1u, a);
    if (warps >= 32LL * all) return launch_pdl(decode_join_kernel<Elem, D, Core::KEYS, 8, 1>, by_row, dim3(8 * D / 4), 0, stream, 1u, a);
    if (warps >= 10LL * all) return launch_pdl(decode_join_kernel<Elem, D, Core::KEYS, 4, 1>, by_row, dim3(4 * D / 4), 0, stream, 1u, a);
    return launch_pdl(decode_join_kernel<Elem, D, Core::KEYS, 1, 4>, dim3(records), dim3(4 * D / 4), 0, stream, 1u, a);
}

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.rows <= 16 ? launch_core<Bf16Core<D, 1>>(a, stream) : launch_core<Bf16Core<D, 2>>(a, stream);
    switch (a.rows) {
        case 1: return launch_core<F32Core<D, 1>>(a, stream);
        case 2: return launch_core<F32Core<D, 2>>(a, stream);
        case 4: return launch_core<F32Core<D, 4>>(a, stream);
        default: return launch_core<F32Core<D, 8>>(a, stream);
    }
}

}  // namespace

DecodePlan make_decode_plan(int B, int Hq, int Hkv, int D, int block_size, int max_blocks, bool bf16, int num_sms) {
    DecodePlan p{};
    const int G = Hq / Hkv;
    // a unit's rows: one or two 16-row fragments (bf16); a power of two up to 8 (fp32)
    p.rows = bf16 ? (G <= 16 ? 16 : 32) : (G >= 5 ? 8 : G >= 3 ? 4 : G);
    p.groups = (G + p.rows - 1) / p.rows;
    const int tile = tile_keys(bf16, D), units = Hkv * p.groups;
    const long long cap_tiles = ((long long)max_blocks * block_size + tile - 1) / tile;
    p.team = 1;
    for (int t = 2; t <= kMaxTeam; ++t)
        if (units % t == 0) p.team = t;
    // eight warps an SM, as many as the shared memory takes; never more than share the table's
    // capacity
    const long long cap = (long long)B * (units / p.team) * cap_tiles;
    long long lanes = 2LL * kWarps * num_sms / p.team;
    p.lanes = lanes_of(cap, static_cast<int>(lanes < 1 ? 1 : lanes));
    const size_t warps = (size_t)p.lanes * p.team;
    p.by_unit = (long long)B * units <= static_cast<long long>(warps);
    p.ws_bytes = 2 * warps * ((size_t)p.rows * (D + 2) * sizeof(float) + sizeof(int)) + warps * sizeof(int4);
    return p;
}

cudaError_t launch_decode_attn(const DecodeArgs& a, bool bf16, cudaStream_t stream) {
    return a.D == 64 ? launch_dim<64>(a, bf16, stream) : launch_dim<128>(a, bf16, stream);
}

}  // namespace tsv
