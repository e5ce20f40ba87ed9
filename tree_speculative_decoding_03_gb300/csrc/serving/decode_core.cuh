// decode_core.cuh -- what the single-token attention kernels share: a warp's products and running
// state for a tile of keys, the division of tiles between lanes, and where a segment's rows go.
#pragma once

#include <cuda_bf16.h>

#include "../common.cuh"

namespace tsv {
namespace {

// tiles of a lane, at least: fewer pieces to join when there is little work, more latencies in a
// row (one sequence of 4096 keys with 2 / 3 / 4 / 6 tiles: 11.4 / 12.5 / 10.4 / 14.7 us)
constexpr int kMinTiles = 4;
constexpr int kFewLanes = 64;  // up to here two tiles do (one sequence of 256 fp32 keys 7.9 -> 6.9 us, 16 of 1 to 60 11.6 -> 8.3)

// Keys of a tile: its K and V rows are 8 KB.
__host__ __device__ constexpr int tile_keys(bool bf16, int D) { return 4096 / (D * (bf16 ? 2 : 4)); }

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
// two neighbours of a row of results, for bf16 with their one rounding
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) { *reinterpret_cast<uint32_t*>(p) = pack_bf16(x, y); }
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

    // loads a unit's query rows, row r from q(r) (the running state is untouched: this runs ahead of reset)
    template <typename Q>
    __device__ __forceinline__ void load_q(Q q, int nrows) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r0 = 16 * t + (lane >> 2), r1 = r0 + 8, c = (lane & 3) * 2;
            const Elem *q0 = q(r0) + c, *q1 = q(r1) + c;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int d = kk * 16;
                qf[t][kk][0] = r0 < nrows ? *reinterpret_cast<const uint32_t*>(q0 + d) : 0u;
                qf[t][kk][1] = r1 < nrows ? *reinterpret_cast<const uint32_t*>(q1 + d) : 0u;
                qf[t][kk][2] = r0 < nrows ? *reinterpret_cast<const uint32_t*>(q0 + d + 8) : 0u;
                qf[t][kk][3] = r1 < nrows ? *reinterpret_cast<const uint32_t*>(q1 + d + 8) : 0u;
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

    // the tile's keys [from, live) are attended to
    __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, int from, int live, float sl2, float*) {
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
            if (live < KEYS || from > 0) {
#pragma unroll
                for (int n = 0; n < NF; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * n + k0 + (e & 1) >= live || 8 * n + k0 + (e & 1) < from) s[t][n][e] = -INFINITY;
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
                auto* to = sink.base(row) + (lane & 3) * 2;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) store2(to + 8 * i, o[t][i][2 * r] * inv, o[t][i][2 * r + 1] * inv);
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

    template <typename Q>
    __device__ __forceinline__ void load_q(Q q, int nrows) {
        const int i = (threadIdx.x & 31) % LPK;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            const float* row = q(r) + i * 4;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = r < nrows ? *reinterpret_cast<const float4*>(row + h * LPK * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
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

    __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, int from, int live, float sl2, float* scratch) {
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
            sc[ps] = key < live && key >= from ? v[0] * sl2 : -INFINITY;
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
            auto* to = sink.base(r) + lane * DV;
#pragma unroll
            for (int d = 0; d < DV; d += 2) store2(to + d, o[r][d] * inv, o[r][d + 1] * inv);
        }
        __syncwarp();
    }
};

// ------------------------------------------------------------------ the schedule

__device__ __forceinline__ long long lane_start(int k, long long T, int lanes) { return (long long)k * T / lanes; }
__device__ __forceinline__ int lane_of_tile(long long x, long long T, int lanes) {
    return static_cast<int>(((x + 1) * lanes - 1) / T);
}

// Lanes that share T tiles.
__host__ __device__ __forceinline__ int lanes_of(long long T, int lanes) {
    const long long few = T / 2 < kFewLanes ? T / 2 : kFewLanes, n = T / kMinTiles > few ? T / kMinTiles : few;
    return n < 1 ? 1 : n < lanes ? static_cast<int>(n) : lanes;
}

// ------------------------------------------------------------------ where rows go

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
    __device__ __forceinline__ Elem* base(int r) const { return out + r * D; }
};
template <int D>
struct ToSlot {
    float *o, *m, *l;  // of the slot
    __device__ __forceinline__ void row(int r, float m_, float l_) const {
        m[r] = m_;
        l[r] = l_;
    }
    __device__ __forceinline__ float factor(float) const { return 1.0f; }
    __device__ __forceinline__ float* base(int r) const { return o + r * D; }
};

}  // namespace
}  // namespace tsv
