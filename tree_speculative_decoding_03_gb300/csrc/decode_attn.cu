// decode_attn.cu -- attention of one new token per sequence over the paged KV cache, split
// over the cache's length and joined.
//
//   s_t = scale * q . k_t (t < L),  out = sum_t e^{s_t - m} v_t / l,  m = max s,  l = sum_t e^{s_t - m},
//   lse = m + ln l.
// Each K/V row is read once; the Hq / Hkv query rows of a kv head share it (about that many
// multiply-adds per element), so the call is bound by the cache's bytes.
//
// Work split: a unit is (sequence, kv head, group of query rows).  Its keys are cut into tiles
// of kTileKeys keys; the tiles of all units, sequence-major, form one row that is divided
// evenly between `lanes` CTAs, so every CTA streams the same bytes whatever the mix of
// lengths.  A CTA goes through its tiles as segments, one per unit it touches.  A segment that
// is a whole unit writes the result; the others leave (m, l, O) in a slot of the workspace (a
// CTA has at most two such segments, its first and its last), and a second kernel joins them:
// O = sum_k 2^{m_k - M} O_k, l likewise, in the order of the CTAs, so a result does not depend
// on timing.
//
// Inside a CTA every warp has its own keys of each tile, its own ring of tiles in shared
// memory filled with asynchronous copies, and its own running (m, l, O), so the main loop has
// no block barrier; the warps' states are joined at the end of the segment.
#include <cuda_bf16.h>

#include "common.cuh"
#include "serving_args.cuh"

namespace tsv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kJoinRows = 4;  // query rows of a CTA of the join

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
// the reference point of the exponentials; a row that has seen only -inf scores keeps P = 0
__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.0f : m; }

// ------------------------------------------------------------------ the two element types
// Keys of a warp's chunk, the stage bytes, and the running state of ROWS query rows.

// bf16: products on the tensor cores, 16 rows a fragment (MT fragments).  With at most 16 rows
// per K/V row the tensor rate is far from a limit (about 190 multiply-adds a clock and SM at
// full memory speed), so the warp-level product serves; P is rounded to bf16 for the second
// product (relative error 2^-9 of each weight, averaged over the keys; l sums the unrounded P).
template <int D_, int MT>
struct Bf16Core {
    static constexpr int D = D_, ROWS = 16 * MT, KEYS = 16, ROWB = D * 2, CH = ROWB / 16;
    using Elem = __nv_bfloat16;
    uint32_t qf[MT][D / 16][4];
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];

    // chunk c (16 bytes) of a row sits at c ^ (row & 7): the 8 rows of a fragment load use
    // different banks
    static __device__ __forceinline__ uint32_t place(int row, int c) { return row * ROWB + ((c ^ (row & 7)) << 4); }

    __device__ __forceinline__ void start(const Elem* q, int nrows) {
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
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
        }
    }

    // `live` of the chunk's 16 keys exist
    __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, int live, float sl2, float*) {
        const int lane = threadIdx.x & 31;
        float s[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.0f;
        {
            const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                ldsm4(b, ks + place(row, 2 * kk + ((lane >> 3) & 1)));
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    mma16816(s[t][0], qf[t][kk], b[0], b[1]);
                    mma16816(s[t][1], qf[t][kk], b[2], b[3]);
                }
            }
        }
        const int k0 = (lane & 3) * 2;
        uint32_t p[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (live < KEYS) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * n + k0 + (e & 1) >= live) s[t][n][e] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(s[t][0][2 * r], s[t][0][2 * r + 1]), fmaxf(s[t][1][2 * r], s[t][1][2 * r + 1])) * sl2;
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
                float w[2][2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) w[n][e] = ex2(fmaf(s[t][n][2 * r + e], sl2, -ms));
                l[t][r] += (w[0][0] + w[0][1]) + (w[1][0] + w[1][1]);
                p[t][r] = pack_bf16(w[0][0], w[0][1]);
                p[t][2 + r] = pack_bf16(w[1][0], w[1][1]);
            }
        }
        {
            const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t b[4];
                ldsm4_t(b, vs + place(row, 2 * i + (lane >> 4)));
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    mma16816(o[t][2 * i], p[t], b[0], b[1]);
                    mma16816(o[t][2 * i + 1], p[t], b[2], b[3]);
                }
            }
        }
    }

    // this warp's state as rows of fp32: O [ROWS][D], then (m, l) of each row
    __device__ __forceinline__ void finish(float* so, float* sm, float* sl) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[t][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int row = 16 * t + 8 * r + (lane >> 2);
                if ((lane & 3) == 0) {
                    sm[row] = m[t][r];
                    sl[row] = sum;
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2*>(so + row * D + 8 * i + (lane & 3) * 2) = make_float2(o[t][i][2 * r], o[t][i][2 * r + 1]);
            }
    }
};

// fp32: multiply-adds on the FMA pipe.  For the scores 8 dimensions of each row sit in a lane,
// D / 8 lanes a key, and the lanes' sums are exchanged so that each ends with one row's score;
// for the second product a lane owns D / 32 dimensions of all rows and the weights come from
// shared memory.
template <int D_, int RR>
struct F32Core {
    static constexpr int D = D_, ROWS = RR, KEYS = 8, ROWB = D * 4, CH = ROWB / 16;
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

    __device__ __forceinline__ void start(const Elem* q, int nrows) {
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
#pragma unroll
            for (int d = 0; d < DV; ++d) o[r][d] = 0.0f;
        }
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

    __device__ __forceinline__ void finish(float* so, float* sm, float* sl) {
        const int lane = threadIdx.x & 31, i = lane % LPK;
        float sum = l;
#pragma unroll
        for (int y = LPK; y < 32; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        if (lane < LPK && i % (LPK / RR) == 0) {
            sm[my_row()] = m;
            sl[my_row()] = sum;
        }
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int d = 0; d < DV; ++d) so[r * D + lane * DV + d] = o[r][d];
    }
};

// ------------------------------------------------------------------ the schedule

// Keys of sequence b that are attended to: 0 when its length does not fit the block table.
__device__ __forceinline__ int seq_keys(const DecodeArgs& a, int b) {
    const int L = __ldg(a.seq_lens + b);
    return (L < 0 || (long long)L > ((long long)a.max_blocks << a.bs_log2)) ? 0 : L;
}

__device__ __forceinline__ long long lane_start(int k, long long T, int lanes) { return (long long)k * T / lanes; }
__device__ __forceinline__ int lane_of_tile(long long x, long long T, int lanes) {
    return static_cast<int>(((x + 1) * lanes - 1) / T);
}

struct Place {   // global tile x lies in unit `unit` of sequence b (of `keys` keys), tile t of its `tiles`
    int b, unit, t, tiles, keys;
};

// One warp: all tiles of the call, and where tile run_start(T) lies.
template <int TILE, typename F>
__device__ __forceinline__ long long locate(const DecodeArgs& a, F run_start, Place* p) {
    const int lane = threadIdx.x & 31, units = a.Hkv * a.groups;
    long long T = 0;
    for (int b = lane; b < a.B; b += 32) T += (seq_keys(a, b) + TILE - 1) / TILE;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    T *= units;
    const long long x = run_start(T);
    *p = Place{0, 0, 0, 1, 0};
    long long base = 0;
    for (int b0 = 0; b0 < a.B && x < T; b0 += 32) {
        const int b = b0 + lane;
        const int keys = b < a.B ? seq_keys(a, b) : 0;
        const int tiles = (keys + TILE - 1) / TILE;
        const long long w = (long long)tiles * units;
        long long incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const long long excl = base + incl - w;
        const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && excl <= x && x < excl + w);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const long long off = x - excl;
            p->b = __shfl_sync(0xffffffffu, b, src);
            p->unit = __shfl_sync(0xffffffffu, static_cast<int>(off / (tiles > 0 ? tiles : 1)), src);
            p->t = __shfl_sync(0xffffffffu, static_cast<int>(off % (tiles > 0 ? tiles : 1)), src);
            p->tiles = __shfl_sync(0xffffffffu, tiles, src);
            p->keys = __shfl_sync(0xffffffffu, keys, src);
            break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return T;
}

template <typename T>
__device__ __forceinline__ T to_elem(float x);
template <>
__device__ __forceinline__ float to_elem<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr float kLn2 = 0.69314718055994530942f;

// four elements of a result row: o / l, rounded once
__device__ __forceinline__ void store_row(float* out, float4 o, float inv) {
    *reinterpret_cast<float4*>(out) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* out, float4 o, float inv) {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

template <typename Core>
constexpr size_t decode_smem() {
    constexpr size_t ring = (size_t)kWarps * kStages * Core::KEYS * Core::ROWB * 2;
    constexpr size_t join = (size_t)kWarps * Core::ROWS * Core::D * 4;
    return (ring > join ? ring : join) + kWarps * 2 * Core::ROWS * 4 + kWarps * (Core::KEYS + 1) * 8 * 4;
}

template <typename Core>
__global__ void __launch_bounds__(kThreads) decode_attn_kernel(const __grid_constant__ DecodeArgs a) {
    using Elem = typename Core::Elem;
    constexpr int D = Core::D, KEYS = Core::KEYS, ROWS = Core::ROWS, TILE = KEYS * kWarps;
    constexpr uint32_t HALF = KEYS * Core::ROWB, STAGE = 2 * HALF;
    constexpr size_t RING = (size_t)kWarps * kStages * STAGE, JOIN = (size_t)kWarps * ROWS * D * 4;
    extern __shared__ __align__(128) uint8_t smem[];
    float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][ROWS][D], after the ring has drained
    float* s_m = reinterpret_cast<float*>(smem + (RING > JOIN ? RING : JOIN));  // [kWarps][ROWS]
    float* s_l = s_m + kWarps * ROWS;
    float* s_scratch = s_l + kWarps * ROWS;  // [kWarps][(KEYS + 1) * 8]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.Hkv * a.groups, bs = 1 << a.bs_log2;
    pdl_wait();
    pdl_launch_dependents();
    Place p;  // found by every warp for itself: cheaper than a block barrier
    const long long T = locate<TILE>(a, [&](long long n) { return lane_start(blockIdx.x, n, a.lanes); }, &p);
    // sequences without keys: nothing to attend to (zeros), or a length that does not fit (NaN)
    for (int b = blockIdx.x; b < a.B; b += a.lanes) {
        if (seq_keys(a, b) > 0) continue;
        const bool empty = __ldg(a.seq_lens + b) == 0;
        const float x = empty ? 0.0f : __int_as_float(0x7fc00000);
        Elem* out = static_cast<Elem*>(a.out) + (long long)b * a.Hq * D;
        for (int i = tid; i < a.Hq * D; i += kThreads) out[i] = to_elem<Elem>(x);
        if (a.lse != nullptr)
            for (int h = tid; h < a.Hq; h += kThreads) a.lse[(long long)b * a.Hq + h] = empty ? -INFINITY : x;
        if (tid == 0) a.seq_err[b] = empty ? 0 : TSV_DERR_CAPACITY;
    }
    long long x = lane_start(blockIdx.x, T, a.lanes);
    const long long x_end = lane_start(blockIdx.x + 1, T, a.lanes);
    const int row_elems = a.Hkv * D;  // elements from one slot to the next
    const uint32_t ring = smem_u32(smem) + warp * kStages * STAGE;
    float* scratch = s_scratch + warp * (KEYS + 1) * 8;
    Core core;
    for (int seg = 0; x < x_end; ++seg) {
        const int g = p.unit / a.groups, row0 = (p.unit % a.groups) * a.rows;
        const int nrows = min(a.rows, a.G - row0);
        const int ntl = static_cast<int>(min((long long)(p.tiles - p.t), x_end - x));
        const bool whole = ntl == p.tiles;
        const int32_t* bt = a.block_table + (long long)p.b * a.max_blocks;
        const long long head = (long long)g * D;
        const Elem* kc = static_cast<const Elem*>(a.k_cache) + head;
        const Elem* vc = static_cast<const Elem*>(a.v_cache) + head;
        bool bad = false;

        // this warp's KEYS keys of the segment's tiles: a run of 8 keys lies in one cache block
        constexpr int RUNS = KEYS / 8, LANES_ROW = Core::CH < 32 ? Core::CH : 32, ROWS_IT = 32 / LANES_ROW;
        int ids[RUNS];  // blocks of the next tile to load, fetched a step ahead
        auto fetch = [&](int i) {
            const int key0 = (p.t + i) * TILE + warp * KEYS;
#pragma unroll
            for (int u = 0; u < RUNS; ++u) ids[u] = key0 + 8 * u < p.keys ? __ldg(bt + ((key0 + 8 * u) >> a.bs_log2)) : -2;
        };
        auto load = [&](int i) {
            const uint32_t dst = ring + (i % kStages) * STAGE;
            const int key0 = (p.t + i) * TILE + warp * KEYS, row = lane / LANES_ROW, c = lane % LANES_ROW;
#pragma unroll
            for (int u = 0; u < RUNS; ++u) {
                const bool in = static_cast<unsigned>(ids[u]) < static_cast<unsigned>(a.num_blocks);
                bad |= !in && ids[u] != -2;
                const int t = key0 + 8 * u;
                long long at = row * row_elems + c * (16 / (int)sizeof(Elem));
                if (in) at += (((long long)ids[u] << a.bs_log2) + (t & (bs - 1))) * row_elems;
#pragma unroll
                for (int r0 = 0; r0 < 8; r0 += ROWS_IT) {
                    const bool take = in && t + r0 + row < p.keys;
                    const Elem* src = kc + (take ? at + (long long)r0 * row_elems : 0);
                    cp16(dst + Core::place(8 * u + r0 + row, c), src, take);
                    cp16(dst + HALF + Core::place(8 * u + r0 + row, c), vc + (src - kc), take);
                }
            }
        };
        core.start(static_cast<const Elem*>(a.q) + ((long long)p.b * a.Hq + g * a.G + row0) * D, nrows);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (i < ntl) {
                fetch(i);
                load(i);
            }
            cp_commit();
        }
        if (kStages - 1 < ntl) fetch(kStages - 1);
        for (int i = 0; i < ntl; ++i) {
            cp_wait<kStages - 2>();
            __syncwarp();
            if (i + kStages - 1 < ntl) load(i + kStages - 1);
            cp_commit();
            if (i + kStages < ntl) fetch(i + kStages);
            const uint32_t src = ring + (i % kStages) * STAGE;
            const int live = p.keys - ((p.t + i) * TILE + warp * KEYS);
            if (live > 0) core.step(src, src + HALF, live, a.scale_log2, scratch);
            __syncwarp();
        }
        cp_wait<0>();
        const bool any_bad = __syncthreads_or(bad) != 0;  // and every warp's ring has drained
        core.finish(s_o + warp * ROWS * D, s_m + warp * ROWS, s_l + warp * ROWS);
        __syncthreads();
        // the warps' states joined, four elements of a row a thread
        const long long slot = (long long)blockIdx.x * 2 + (seg == 0 ? 0 : 1);
        for (int e = tid; e < nrows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), d = (e % (D / 4)) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * ROWS + r]);
            const float ms = safe_max(M);
            float sum = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s_m[w * ROWS + r] - ms);
                const float4 o = *reinterpret_cast<const float4*>(s_o + (w * ROWS + r) * D + d);
                sum = fmaf(f, s_l[w * ROWS + r], sum);
                acc.x = fmaf(f, o.x, acc.x);
                acc.y = fmaf(f, o.y, acc.y);
                acc.z = fmaf(f, o.z, acc.z);
                acc.w = fmaf(f, o.w, acc.w);
            }
            if (whole) {
                const long long h = (long long)p.b * a.Hq + g * a.G + row0 + r;
                store_row(static_cast<Elem*>(a.out) + h * D + d, acc, any_bad ? __int_as_float(0x7fc00000) : 1.0f / sum);
                if (d == 0 && a.lse != nullptr) a.lse[h] = any_bad ? __int_as_float(0x7fc00000) : (M + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot * a.rows + r) * D + d) = acc;
                if (d == 0) {
                    a.part_m[slot * a.rows + r] = M;
                    a.part_l[slot * a.rows + r] = sum;
                }
            }
        }
        if (tid == 0) {
            if (!whole)
                a.part_bad[slot] = any_bad ? 1 : 0;
            else if (p.unit == 0)
                a.seq_err[p.b] = any_bad ? TSV_DERR_BLOCK : 0;
        }
        __syncthreads();
        x += ntl;
        // the next unit that has keys
        p.t = 0;
        if (++p.unit == units) {
            p.unit = 0;
            do {
                ++p.b;
                p.keys = p.b < a.B ? seq_keys(a, p.b) : 1;
            } while (p.keys == 0);
            p.tiles = (p.keys + TILE - 1) / TILE;
        }
    }
}

// Joins the pieces of the units that lie on more than one CTA.  CTA (k, y) looks at the
// boundary between lanes k and k + 1: when it falls inside a unit and is the first one there,
// this CTA joins the unit's pieces, in lane order, for query rows [kJoinRows y, ...).  A row's
// D / 4 threads read the pieces' rows as coalesced float4s, kAhead of them in flight.
template <typename Elem, int D, int TILE>
__global__ void __launch_bounds__(kJoinRows * D / 4) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int kAhead = 8;
    // the schedule needs the lengths alone, which the kernel before this one has waited for
    // before it let this one start
    Place p;
    const long long T = locate<TILE>(a, [&](long long n) { return lane_start(blockIdx.x + 1, n, a.lanes); }, &p);
    const long long s0 = lane_start(blockIdx.x, T, a.lanes), x = lane_start(blockIdx.x + 1, T, a.lanes);
    const long long first = x - p.t;  // the unit's first tile
    // not inside a unit; or an earlier boundary is; or an empty lane, whose end is no new boundary
    const bool mine = x < T && p.t != 0 && s0 <= first && s0 != x;
    const int c0 = blockIdx.x, c1 = mine ? lane_of_tile(first + p.tiles - 1, T, a.lanes) : c0;
    const int side0 = s0 == first ? 0 : 1;
    const int g = p.unit / a.groups, row0 = (p.unit % a.groups) * a.rows, nrows = min(a.rows, a.G - row0);
    const int r = blockIdx.y * kJoinRows + threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
    const bool sparse = T < a.lanes;  // some lanes are empty
    pdl_wait();
    pdl_launch_dependents();
    if (!mine || r >= nrows) return;
    // slot of piece c, or -1 for an empty lane
    auto slot = [&](int c) {
        if (sparse && lane_start(c + 1, T, a.lanes) == lane_start(c, T, a.lanes)) return -1;
        return 2 * c + (c == c0 ? side0 : 0);
    };
    float M = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int bad = 0;
    for (int c = c0; c <= c1; c += kAhead) {
        float m[kAhead], l[kAhead];
        float4 o[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int sl = c + i <= c1 ? slot(c + i) : -1;
            m[i] = -INFINITY;
            l[i] = 0.0f;
            o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sl >= 0) {
                const long long pr = (long long)sl * a.rows + r;
                m[i] = a.part_m[pr];
                l[i] = a.part_l[pr];
                o[i] = *reinterpret_cast<const float4*>(a.part_o + pr * D + d);
                bad |= a.part_bad[sl];
            }
        }
        float m_new = M;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) m_new = fmaxf(m_new, m[i]);
        const float ms = safe_max(m_new);
        const float f0 = ex2(M - ms);
        M = m_new;
        sum *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float f = ex2(m[i] - ms);
            sum = fmaf(f, l[i], sum);
            acc.x = fmaf(f, o[i].x, acc.x);
            acc.y = fmaf(f, o[i].y, acc.y);
            acc.z = fmaf(f, o[i].z, acc.z);
            acc.w = fmaf(f, o[i].w, acc.w);
        }
    }
    const long long h = (long long)p.b * a.Hq + g * a.G + row0 + r;
    const float nan = __int_as_float(0x7fc00000);
    store_row(static_cast<Elem*>(a.out) + h * D + d, acc, bad ? nan : 1.0f / sum);
    if (d == 0 && a.lse != nullptr) a.lse[h] = bad ? nan : (M + log2f(sum)) * kLn2;
    if (d == 0 && r == 0 && p.unit == 0) a.seq_err[p.b] = bad ? TSV_DERR_BLOCK : 0;
}

template <typename Core>
cudaError_t launch_core(const DecodeArgs& a, cudaStream_t stream) {
    constexpr size_t smem = decode_smem<Core>();
    thread_local int smem_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != smem_dev) {
        e = cudaFuncSetAttribute(decode_attn_kernel<Core>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        smem_dev = dev;
    }
    e = launch_pdl(decode_attn_kernel<Core>, dim3(static_cast<unsigned>(a.lanes)), dim3(kThreads), smem, stream, 1u, a);
    if (e != cudaSuccess || a.lanes < 2) return e;
    const int most = min(a.rows, a.G);  // query rows of a unit
    return launch_pdl(decode_join_kernel<typename Core::Elem, Core::D, Core::KEYS * kWarps>,
                      dim3(static_cast<unsigned>(a.lanes - 1), static_cast<unsigned>((most + kJoinRows - 1) / kJoinRows)),
                      dim3(kJoinRows * Core::D / 4), 0, stream, 1u, a);
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
    const int tile = (bf16 ? 16 : 8) * kWarps;
    // two CTAs an SM, as many as the shared memory takes; never more than the table has tiles
    const long long cap = (long long)B * Hkv * p.groups * (((long long)max_blocks * block_size + tile - 1) / tile);
    long long lanes = 2LL * num_sms;
    if (lanes > cap) lanes = cap;
    p.lanes = lanes < 1 ? 1 : static_cast<int>(lanes);
    p.ws_bytes = 2 * (size_t)p.lanes * ((size_t)p.rows * (D + 2) * sizeof(float) + sizeof(int));
    return p;
}

cudaError_t launch_decode_attn(const DecodeArgs& a, bool bf16, cudaStream_t stream) {
    return a.D == 64 ? launch_dim<64>(a, bf16, stream) : launch_dim<128>(a, bf16, stream);
}

}  // namespace tsv
