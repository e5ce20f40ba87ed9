// rope_append.cu -- rotary positions of q and k on up to four axes, and the K/V rows
// written into the paged cache at their slots, in one pass.
//
// Pair i of a head turns by theta = pos[axis(i)] * inv_freq[i]:
//   (x, y) <- (x cos - y sin, y cos + x sin),
// pairs (i, i + R/2) or (2i, 2i + 1) of the head's first R elements; the rest passes through.
// q goes to q_out, k and v to cache row slot_map[t].
//
// The pass reads and writes every element once and is bound by memory.  The angles are the
// same for all heads of a token, so a block forms the cosines and sines of its tokens once,
// in shared memory, and each thread keeps those of its part of the head in registers while
// it goes through the heads.  A thread's item is two 16-byte vectors of one head: with pairs
// (i, i + R/2) vector c and its partner R/2 elements on, otherwise vectors 2c and 2c + 1.
#include <cuda_bf16.h>

#include "../common.cuh"
#include "serving_args.cuh"

namespace tsv {
namespace {

constexpr int kRopeThreads = 256;

// cos and sin of pos * f.  The turn count pos * f / (2 pi) is formed as a pair of floats
// (about 44 significant bits), its whole part dropped exactly, and the rest handed to
// sincospif: far positions keep the accuracy of near ones (a float product at position 10^6
// would be off by 0.03 rad).
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    constexpr float kInvTwoPiHi = 0.15915494f;
    constexpr float kInvTwoPiLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(0.15915494f));
    const float fh = __fmul_rn(f, kInvTwoPiHi);  // (rounded products by name: contracted ones would lose what fl and lo hold)
    const float fl = fmaf(f, kInvTwoPiHi, -fh) + f * kInvTwoPiLo;
    const float ph = static_cast<float>(pos);  // exact up to 2^24; past that the rest is added below
    const float hi = __fmul_rn(ph, fh);
    float lo = fmaf(ph, fl, fmaf(ph, fh, -hi));
    if (pos > (1 << 24) || pos < -(1 << 24))
        lo = fmaf(static_cast<float>(static_cast<long long>(pos) - static_cast<long long>(ph)), fh, lo);
    const float r = (hi - rintf(hi)) + lo;
    float s, c;
    sincospif(2.0f * r, &s, &c);
    return make_float2(c, s);
}

template <typename T>
struct Vec;  // one 16-byte vector
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void unpack(const uint4& u, float* x) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(const uint4& u, float* x) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // the one rounding of the result
    __device__ static uint4 pack(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Block: `tok` tokens x head lanes x D / (2 * vector) items of a head.  A thread's first vectors
// are on their way while the block forms the angles, and the next head's while it turns one.
template <typename T, int D, bool NEIGH>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a, int tok) {
    constexpr int VN = Vec<T>::N, ITEMS = D / (2 * VN), LANES = kRopeThreads / ITEMS;
    extern __shared__ __align__(16) float s_turn[];  // cos [tok][R / 2], then sin [tok][R / 2]
    const int tid = threadIdx.x, half = a.R >> 1;
    const int t0 = blockIdx.x * tok;
    const int item = tid % ITEMS, lane = tid / ITEMS;
    const int hl = LANES / tok;  // head lanes of a token
    const int ti = lane / hl, h0 = lane % hl;
    const int t = t0 + ti;
    // this thread's two vectors of a head, and whether they turn
    const int turning = half / VN;  // items that turn
    const bool turns = item < turning;
    const int rest = a.R + (item - turning) * 2 * VN;
    const int e0 = turns ? (NEIGH ? 2 * item * VN : item * VN) : rest;
    const int e1 = turns ? (NEIGH ? e0 + VN : e0 + half) : rest + VN;
    const int heads = a.Hq + 2 * a.Hkv;
    const bool live = t < a.T && h0 < heads;
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + t * a.k_stride - (long long)a.Hq * D;
    const T* v = static_cast<const T*>(a.v) + t * a.v_stride - (long long)(a.Hq + a.Hkv) * D;
    auto source = [&](int h) { return (h < a.Hq ? q : h < a.Hq + a.Hkv ? k : v) + (long long)h * D; };
    pdl_wait();
    pdl_launch_dependents();
    long long slot = -1;
    uint4 u0 = make_uint4(0u, 0u, 0u, 0u), u1 = u0;
    if (live) {
        slot = a.slot_map[t];  // an ordinary load, as of the positions: the kernel before this one may have written them
        u0 = *reinterpret_cast<const uint4*>(source(h0) + e0);
        u1 = *reinterpret_cast<const uint4*>(source(h0) + e1);
    }
    float* s_cos = s_turn;
    float* s_sin = s_turn + tok * half;
    for (int i = tid, ts = t0 + tid / half, p = tid % half; i < tok * half; i += kRopeThreads) {
        float2 cs = make_float2(1.0f, 0.0f);
        if (ts < a.T) cs = turn_of(a.positions[(long long)a.axis[p] * a.T + ts], __ldg(a.inv_freq + p));
        s_cos[i] = cs.x;
        s_sin[i] = cs.y;
        ts += kRopeThreads / half;
        p += kRopeThreads % half;
        if (p >= half) {
            p -= half;
            ++ts;
        }
    }
    __syncthreads();
    if (!live) return;
    T* qo = static_cast<T*>(a.q_out) + t * a.q_out_stride;
    const bool bad = slot >= a.slots;
    if (item == 0 && h0 == 0) a.tok_err[t] = bad ? TSV_DERR_BLOCK : 0;
    if (slot < 0 || bad) {  // a padding row is zero, a row with a bad slot NaN
        float x[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) x[i] = bad ? __int_as_float(0x7fc00000) : 0.0f;
        const uint4 u = Vec<T>::pack(x);
        for (int h = h0; h < a.Hq; h += hl) {
            *reinterpret_cast<uint4*>(qo + (long long)h * D + e0) = u;
            *reinterpret_cast<uint4*>(qo + (long long)h * D + e1) = u;
        }
        return;
    }
    float cs[VN], sn[VN];
#pragma unroll
    for (int i = 0; i < VN; i += 4) {
        const float4 c4 = turns ? *reinterpret_cast<const float4*>(s_cos + ti * half + item * VN + i) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 s4 = turns ? *reinterpret_cast<const float4*>(s_sin + ti * half + item * VN + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        cs[i] = c4.x, cs[i + 1] = c4.y, cs[i + 2] = c4.z, cs[i + 3] = c4.w;
        sn[i] = s4.x, sn[i + 1] = s4.y, sn[i + 2] = s4.z, sn[i + 3] = s4.w;
    }
    T* kc = static_cast<T*>(a.k_cache) + (slot * a.Hkv - a.Hq) * D;
    T* vc = static_cast<T*>(a.v_cache) + (slot * a.Hkv - a.Hq - a.Hkv) * D;
    if (!TSV_IN_BOUNDS((slot + 1) * a.Hkv * D - 1, a.slots * a.Hkv * D, a.tok_err + t)) return;
    for (int h = h0; h < heads; h += hl) {
        uint4 n0 = u0, n1 = u1;
        if (h + hl < heads) {
            n0 = *reinterpret_cast<const uint4*>(source(h + hl) + e0);
            n1 = *reinterpret_cast<const uint4*>(source(h + hl) + e1);
        }
        if (turns && h < a.Hq + a.Hkv) {
            float x[2 * VN];
            Vec<T>::unpack(u0, x);
            Vec<T>::unpack(u1, x + VN);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                float& p = x[NEIGH ? 2 * i : i];
                float& r = x[NEIGH ? 2 * i + 1 : i + VN];
                const float y = p * cs[i] - r * sn[i];
                r = r * cs[i] + p * sn[i];
                p = y;
            }
            u0 = Vec<T>::pack(x);
            u1 = Vec<T>::pack(x + VN);
        }
        T* dst = (h < a.Hq ? qo : h < a.Hq + a.Hkv ? kc : vc) + (long long)h * D;
        *reinterpret_cast<uint4*>(dst + e0) = u0;
        *reinterpret_cast<uint4*>(dst + e1) = u1;
        u0 = n0;
        u1 = n1;
    }
}

template <typename T, int D>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
    // Tokens a block: up to 8, as many as leave a thread at most 8 heads to go through (fewer heads do
    // not pay for the block's angles and start-up, more leave a ragged last wave), more than 8
    // until a thread has two heads, and always at least three blocks an SM.  With 1 / 2 / 4 / 8 / 16
    // tokens: 4096 tokens of 80 heads 30.8 / 29.1 / 28.9 / 29.3 / - us; 20011 of 48 heads 97 / 82 / 78 /
    // 82 / -; 20000 of 24 heads of 64 59 / 36 / 27 / 24 / 27; 1024 of 80 heads 9.6 / 8.8 / 10.9 / 16.4 / -;
    // 27892 of 6 heads of 64 with 8 tokens 16.2, with 32 13.2.
    constexpr int LANES = kRopeThreads * 2 * Vec<T>::N / D;
    const long long heads = a.Hq + 2LL * a.Hkv;
    int tok = 1;
    while (2 * tok <= LANES && a.T >= 3LL * num_sms * 2 * tok && (tok < 8 ? heads * 2 * tok <= 8 * LANES : heads * tok < 2 * LANES))
        tok *= 2;
    const dim3 grid(static_cast<unsigned>((a.T + tok - 1) / tok));
    const size_t smem = (size_t)tok * a.R * sizeof(float);
    return a.neighbours ? launch_pdl(rope_append_kernel<T, D, true>, grid, dim3(kRopeThreads), smem, stream, 1u, a, tok)
                        : launch_pdl(rope_append_kernel<T, D, false>, grid, dim3(kRopeThreads), smem, stream, 1u, a, tok);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    if (bf16)
        return a.D == 64 ? launch_rope<__nv_bfloat16, 64>(a, num_sms, stream) : launch_rope<__nv_bfloat16, 128>(a, num_sms, stream);
    return a.D == 64 ? launch_rope<float, 64>(a, num_sms, stream) : launch_rope<float, 128>(a, num_sms, stream);
}

}  // namespace tsv
