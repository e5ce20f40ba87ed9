// prefix_tc.cu -- the shared prefixes of prefix_attn.cu on the 5th-generation tensor cores (tcgen05,
// accumulators in TMEM, K/V tiles by TMA), bf16.
//
// The R rows of a group and kv head -- the group's sequences times the heads of the kv head -- against the
// group's P keys are two dense products, the second with weights in two parts: 3 R P D multiply-adds on 4 P D
// bytes, so from some 190 rows on the tensor cores are the bound, and below the cache's bytes.
//
// Work split: a unit is (group, kv head, 256 rows).  Its keys are cut into 128-key tiles, the tiles of
// all units form one row, divided evenly between persistent CTAs.  A CTA's segment of a unit ends in
// (m, l, O) of its rows, at the rows' own places if it is the whole unit, else in a slot of the CTA; the
// join of prefix_attn.cu adds them up.
//
// Two streams of softmax, a warpgroup each.  With more than 128 rows they take the two halves of
// the rows, on the same tiles; with fewer they take the same rows, on every other tile, so that one's
// products run during the other's softmax in both cases.
//
// Warp roles (384 threads): warp 0 loads K and V tiles by TMA into a ring of slots, ahead across segments; warps 1
// and 2 issue the products, S = Q K^T into TMEM and O += P V with P in TMEM; warps 4 - 11 are the softmax, a thread
// a row: all 128 scores of a tile in registers, O rescaled only when the maximum has grown by more than 2^8.
//
// Precision: a weight goes into the second product as two bf16 parts, as in the single-token attention
// (the second part's products take half as long again as the others together; with one part alone the result is off by
// another rounding of bf16).  Both lie in the columns of S that the weights came from.
//
// The CTAs that the plan leaves without prefix tiles take the stream of the sequences' own keys, up to eight warps each
// (prefix_stream.cuh).  They are CTAs of this kernel and not a kernel of their own: that one could run beside this one
// only if it did not wait for it, and what the plan has written is promised to a kernel that has waited.
//
// Every wait is bounded.  One that gives up sets TSV_DERR_TIMEOUT for the sequences of all groups from its own
// to the CTA's last: a CTA does nothing more after it.
#include <cuda_bf16.h>

#include "../common.cuh"
#include "../tc_ptx.cuh"
#include "continue_args.cuh"
#include "prefix_stream.cuh"

namespace tsv {
namespace {

constexpr int kThreads = 384;
constexpr int kTileKeys = kPrefixTcKeys;
constexpr int kUnitRows = kPrefixTcRows;
constexpr uint32_t kHalfBytes = 128 * 128;  // 128 rows x 64 bf16 (one 128B-swizzled half)
constexpr int kMaxSlots = 12;
constexpr uint32_t kRegsProducer = 96, kRegsSoftmax = 200, kRegsIdle = 24, kRegsStream = 240;
static_assert(128 * kRegsProducer + 256 * kRegsSoftmax <= 384 * 168, "register split exceeds the launch");
static_assert(128 * kRegsIdle + 256 * kRegsStream <= 384 * 168, "register split exceeds the launch");

// Shared memory: Q tiles | ring of K/V slots | barriers.
struct Layout {
    uint32_t ring, bars, total;
    int slots;
};
template <int D, int QT>  // QT: Q tiles
__host__ __device__ constexpr Layout layout() {
    Layout l{};
    constexpr uint32_t tile = 128u * D * 2u, budget = 232448u - 1024u - 512u;  // max dynamic smem - alignment slack - barriers
    l.ring = QT * tile;
    const int slots = static_cast<int>((budget - l.ring) / tile);
    l.slots = slots > kMaxSlots ? kMaxSlots : slots;
    l.bars = l.ring + l.slots * tile;
    l.total = l.bars + 512 + 1024;
    return l;
}

// A place in the ring: the slot of a fill, and the parity of its barriers' phase.  A parity tells a phase from the next one
// only.  So who waits for a fill has seen the slot's last one land, or knows that this one has been sent (for which the
// producer has waited until the last one was used up): streams on every other tile see each other's fills through neither
// their waits nor the weights, and with 5 or 6 slots a slot goes from one stream to the other.
template <int SLOTS>
struct Slot {
    int slot;
    uint32_t parity;
    __device__ __forceinline__ void skip(int fills) {  // fills <= SLOTS
        slot += fills;
        if (slot >= SLOTS) {
            slot -= SLOTS;
            parity ^= 1;
        }
    }
};

struct Bars {
    static constexpr int kFull = 0;           // [slots]
    static constexpr int kEmpty = kMaxSlots;  // [slots]
    static constexpr int kS = 2 * kMaxSlots;  // [2] scores of a stream's tile are in TMEM
    static constexpr int kP = kS + 2;         // [2] its weights are
    static constexpr int kO = kP + 2;         // [2] a segment's last product with V is done
    static constexpr int kQ = kO + 2;         // a segment's Q rows are in shared memory
    static constexpr int kSeen = kQ + 1;  // both issuers have seen that
    static constexpr int kDone = kSeen + 1;  // [2]
    static constexpr int kStall = kDone + 2;  // never completed (test build: the stalled wait)
    static constexpr int kCount = kStall + 1;
};

#ifdef TSV_TEST_HOOKS
// test build only: the wait for each CTA's n-th tile of the first stream is pointed at a barrier that nothing completes
__device__ int g_test_prefix_stall = 0;
#endif

// A position in the row of tiles: tile t of the `tiles` of unit `unit` of group g.
struct Tile {
    int g, unit, t, tiles, groups;  // groups: of 256 rows
    int4 it;                        // first sequence, first key (0), end, rows
    __device__ __forceinline__ void set(int group, const int4& item) {
        g = group;
        it = item;
        tiles = (it.z + kTileKeys - 1) / kTileKeys;
        groups = (it.w + kUnitRows - 1) / kUnitRows;
    }
    __device__ __forceinline__ void next_unit(const PrefixArgs& a) {
        t = 0;
        if (++unit < groups * a.Hkv) return;
        unit = 0;
        do {
            set(g + 1, a.item[g + 1]);
        } while (!has_tiles(tiles, groups) && g + 1 < a.G);
    }
    __device__ __forceinline__ int head() const { return unit / groups; }
    __device__ __forceinline__ int row0() const { return unit % groups * kUnitRows; }
    __device__ __forceinline__ int rows() const { return min(kUnitRows, it.w - row0()); }
    // both streams on the same rows, each with every other tile
    __device__ __forceinline__ bool by_tile() const { return rows() <= 128; }
};

// The products with descriptors given by their low words.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // 1024 bytes between 8-row groups, version 1, 128-byte swizzle
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 da, db;\nmov.b64 da, {%1, %4};\nmov.b64 db, {%2, %4};\nsetp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 db;\nmov.b64 db, {%2, %4};\nsetp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t opaque_u32(uint32_t x) {
    uint32_t y;
    asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void store_release_smem(uint32_t at, int x) {
    asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ int load_acquire_smem(uint32_t at) {
    int x;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
// Bounded wait until fill `fill` has been sent; *sent: the fills that are known to be.
__device__ __forceinline__ bool wait_sent(uint32_t at, int fill, int* sent, volatile int* abort_flag) {
    if (fill < *sent) return true;
    const unsigned long long t0 = globaltimer();
    while (true) {
        *sent = load_acquire_smem(at);
        if (fill < *sent) return true;
        if (*abort_flag || globaltimer() - t0 > kWaitLimitNs) return false;
    }
}

// One warp: the sequences whose rows a unit holds have a block id outside the cache.
__device__ __forceinline__ void flag_unit(const PrefixArgs& a, const Tile& p) {
    const int r0 = p.row0();
    for (int s = r0 / a.gq + (threadIdx.x & 31); s <= (r0 + p.rows() - 1) / a.gq; s += 32) atomicOr(a.seq_err + p.it.x + s, TSV_DERR_BLOCK);
}

// Two weights (0 or normal numbers) as the sum of two bf16 each, hi and lo: hi is the weight cut off after bf16's
// bits, lo the rest and 2^-23 of the weight more, so that a positive weight has two positive parts, which
// keep an infinite value infinite.
__device__ __forceinline__ void split_bf16_up(float w0, float w1, uint32_t* hi, uint32_t* lo) {
    const uint32_t u0 = __float_as_uint(w0), u1 = __float_as_uint(w1);
    *hi = __byte_perm(u0, u1, 0x7632);
    const float more = 1.0f + 0x1p-23f;
    float l0, l1;
    f2_unpack(f2_fma(f2_pack(w0, w1), f2_pack(more, more),
                     f2_pack(__uint_as_float((u0 & 0xffff0000u) ^ 0x80000000u), __uint_as_float((u1 & 0xffff0000u) ^ 0x80000000u))),
              l0, l1);
    const __nv_bfloat162 l = __floats2bfloat162_rn(l0, l1);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
}

template <int D, int QT, int MT>  // MT: 16-row fragments of a unit of the stream
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    constexpr int HALVES = D / 64;
    constexpr uint32_t SLOT = 128u * D * 2u;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr Layout lay = layout<D, QT>();
    constexpr int nslots = lay.slots;
    using Fill = Slot<nslots>;
    using StreamCore = Bf16Core<D, MT>;
    static_assert(kStreamWarps * (kRingBytes + kScratch * sizeof(float)) <= lay.bars, "the stream's rings fit in front of the barriers");
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + lay.bars);
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + lay.bars + 8 * Bars::kCount);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + lay.bars + 8 * Bars::kCount + 4);
    int* s_lost = reinterpret_cast<int*>(smem + lay.bars + 8 * Bars::kCount + 8);  // first group in which a wait gave up
    const uint32_t sent_at = smem_u32(smem + lay.bars + 8 * Bars::kCount + 12);    // fills sent so far
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [=](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = 1 << a.bs_log2;

    if (tid == 0) {
        for (int i = 0; i < nslots; ++i) {
            mbar_init(bar(Bars::kFull + i), 1);
            mbar_init(bar(Bars::kEmpty + i), 1);
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(bar(Bars::kS + m), 1);
            mbar_init(bar(Bars::kP + m), m == 0 ? 129 : 128);  // and for stream 0, that the tile has landed
            mbar_init(bar(Bars::kO + m), 1);
            mbar_init(bar(Bars::kDone + m), 1);
        }
        mbar_init(bar(Bars::kQ), 256);
        mbar_init(bar(Bars::kSeen), 2);
        mbar_init(bar(Bars::kStall), 1);
        *s_abort = 0;
        *s_lost = a.G;
        store_release_smem(sent_at, 0);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    pdl_wait();  // the plan
    pdl_launch_dependents();
    const int me = blockIdx.x;
    const int4 begin = a.tc_begin[2 * me], item = a.tc_begin[2 * me + 1];  // group, unit, tile, tiles of this CTA
    const int count = begin.w;
    Tile first{};
    if (count > 0) {
        first.set(begin.x, item);
        first.unit = begin.y;
        first.t = begin.z;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    int my_err = 0;
    int err_g = first.g;  // the group in which a wait of this thread is or gave up

    if (count > 0 && warp < 4) regs_dec<kRegsProducer>();
    if (warp == 0 && count > 0) {
        // ============================ TMA producer: a lane for each block of the tile issues that block's boxes.
        // Block ids come 32 at a time, those of some tiles of a unit, a batch ahead.  (Two warps of 16-byte
        // asynchronous copies instead: 4096 rows of 32768 keys 132 us against 140, 24 ragged groups of 64-wide heads 175
        // against 118.)
        const int per_tile = kTileKeys >> a.bs_log2, batch = 32 / per_tile;
        Tile p = first, q = first;  // of the fills, of the next batch
        int q_left = count;         // tiles in no batch yet
        auto fetch = [&]() {
            if (q_left <= 0) return 0;
            const int e = q.t * per_tile + lane, n = min(batch, q.tiles - q.t);
            const int id = e < (q.it.z + bs - 1) >> a.bs_log2 ? a.block_table[(long long)q.it.x * a.max_blocks + e] : 0;
            q_left -= n;
            if (q_left > 0) {
                q.t += n;
                if (q.t >= q.tiles) q.next_unit(a);
            }
            return id;
        };
        int blk = fetch(), blk_next = fetch(), k = 0;  // k: the tile's place in its batch
        int issued = 0;
        const uint64_t policy = l2_evict_first_policy();  // (also for keys that two units read: 122 us against 131)
        for (int j = 0; j < count && !my_err; ++j) {
            const int nblk = (min(kTileKeys, p.it.z - p.t * kTileKeys) + bs - 1) >> a.bs_log2, g = p.head();
            const int cur = __shfl_sync(0xffffffffu, blk, (k * per_tile + lane) & 31);
            const bool mine = lane < nblk, bad = mine && static_cast<unsigned>(cur) >= static_cast<unsigned>(a.num_blocks);
            if (__any_sync(0xffffffffu, bad)) flag_unit(a, p);
            const int slot_row = (bad ? a.num_blocks : cur) << a.bs_log2;  // (a bad id reads zeros past the cache)
            err_g = p.g;
            if (j + 1 < count) {
                ++k;
                if (++p.t >= p.tiles) {
                    p.next_unit(a);
                    k = batch;
                }
                if (k == batch) {
                    blk = blk_next;
                    blk_next = fetch();
                    k = 0;
                }
            }
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const int f = 2 * j + kv, slot = f % nslots, use = f / nslots;
                if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(Bars::kEmpty + slot), (use - 1) & 1, s_abort))) {
                    my_err = 1;
                    break;
                }
                const uint32_t dst = smem_u32(smem + lay.ring + slot * SLOT) + lane * bs * 128;
                if (lane == 0) {
                    mbar_expect_tx(bar(Bars::kFull + slot), static_cast<uint32_t>(nblk * bs * 128 * HALVES));
                    store_release_smem(sent_at, f + 1);
                }
                __syncwarp();
                if (mine) {
#pragma unroll
                    for (int hh = 0; hh < HALVES; ++hh)
                        tma_load_3d(dst + hh * kHalfBytes, kv ? &tmv : &tmk, bar(Bars::kFull + slot), hh * 64, g, slot_row, policy);
                }
                issued = f + 1;
            }
        }
        // never leave with copies in flight
        if (lane == 0) {
            for (int f = max(0, issued - nslots); f < issued; ++f) {
                volatile int never = 0;
                if (!mbar_wait(bar(Bars::kFull + f % nslots), (f / nslots) & 1, &never)) my_err = 1;
            }
        }
    } else if (warp < 3 && count > 0) {
        // ============================ MMA issuers.  The products are issued as fast as the tensor pipe takes them,
        // and it holds few: what the issuing thread does in between (waits, places in the ring) is time that the
        // pipe stands still.  So places are counted on without divisions.  Streams on the same tiles have one
        // issuer, which keeps a stream's O and next S together, while the other warp waits for the fills; streams
        // on every other tile one each, so that neither waits for the other's fills.  (One prompt of 32768 keys, 64 sequences: 134 us, with an issuer
        // each 147, with divisions and 64-bit descriptors 150; 24 ragged groups: 162, with one issuer 166.)
        if (lane == 0) {
            const int me_m = warp - 1;
            constexpr uint32_t idS = idesc_bf16(128, 128, false), idO = idesc_bf16(128, D, true);
            // Descriptors of Q and K tiles (K-major) and V tiles (MN-major): the high words are constants, the low ones
            // hold the address in units of 16 bytes, so that an operand costs one 32-bit add.
            const uint32_t dQ = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem), 16, 1024));
            const uint32_t dK = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + lay.ring), 16, 1024));
            const uint32_t dV = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + lay.ring), kHalfBytes, 1024));
            // S of stream m = Q tile qt . K^T
            auto issue_S = [=](int m, int qt, int slot) {
                const uint32_t qa = opaque_u32(dQ + ((qt * SLOT) >> 4)), kb = opaque_u32(dK + ((slot * SLOT) >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
                    mma_ss(tmem + m * 128, qa + off, kb + off, idS, k > 0);
                }
            };
            // O of stream m += (hi + lo) . V; hi in the first 64 columns of S, lo in the others
            auto issue_PV = [=](int m, int slot, bool more) {
                const uint32_t vb = opaque_u32(dV + ((slot * SLOT) >> 4));
                const uint32_t d = tmem + 256 + m * D, pa = tmem + m * 128;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < kTileKeys / 16; ++k)
                        mma_ts(d, pa + part * 64 + k * 8, vb + ((k * 16 * 128) >> 4), idO, (more || part > 0 || k > 0) ? 1u : 0u);
            };
            int sent = 0;  // fills that are known to have been sent
            auto full = [&](const Fill& f, int fill) {
                return wait_sent(sent_at, fill, &sent, s_abort) && mbar_wait(bar(Bars::kFull + f.slot), f.parity, s_abort);
            };
            auto free_slot = [&](const Fill& f) { mma_commit(bar(Bars::kEmpty + f.slot)); };
            Tile p = first;
            uint32_t n_p[2] = {0, 0};  // tiles of each stream before the segment
            bool ok = true;
            for (int j = 0, seg = 0; j < count && ok; ++seg) {
                const int n = min(p.tiles - p.t, count - j);
                const bool by_tile = p.by_tile();
                err_g = p.g;
                ok = mbar_wait(bar(Bars::kQ), seg & 1, s_abort);
                mbar_arrive(bar(Bars::kSeen));
                Fill fK{2 * j % nslots, static_cast<uint32_t>(2 * j / nslots) & 1u}, fV = fK;  // of the next K and V tile
                fV.skip(1);
                if (!by_tile && me_m == 1) {
                    // what a tile's products read besides the weights: one arrival with those of stream 0, and
                    // not before the last tile's have all come
                    for (int i = 0; i < n && ok; ++i) {
                        fK.skip(2);
                        ok = full(fV, 2 * (j + i) + 1) && (i + 1 == n || full(fK, 2 * (j + i) + 2));
                        if (!ok) break;
                        mbar_arrive(bar(Bars::kP));
                        fV.skip(2);
                        // (after the last tile the next segment's Q says so)
                        if (i + 1 < n) ok = mbar_wait(bar(Bars::kP), (n_p[0] + i) & 1, s_abort);
                    }
                } else if (!by_tile) {
                    ok = ok && full(fK, 2 * j);
                    if (!ok) break;
                    tc_fence_after();
                    for (int m = 0; m < 2; ++m) {
                        issue_S(m, m, fK.slot);
                        mma_commit(bar(Bars::kS + m));
                    }
                    free_slot(fK);
                    fK.skip(2);
                    for (int i = 0; i < n && ok; ++i) {
                        const bool next = i + 1 < n;
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            ok = mbar_wait(bar(Bars::kP + m), (n_p[m] + i) & 1, s_abort);
                            if (!ok) break;
                            tc_fence_after();
                            issue_PV(m, fV.slot, i > 0);
                            if (next) issue_S(m, m, fK.slot);
                            mma_commit(bar((next ? Bars::kS : Bars::kO) + m));
                        }
                        if (!ok) break;
                        free_slot(fV);
                        if (next) free_slot(fK);
                        fV.skip(2);
                        fK.skip(2);
                    }
                } else if (by_tile && me_m < n && ok) {
                    const int m = me_m;
                    if (m > 0) {
                        fK.skip(2);
                        fV.skip(2);
                    }
                    ok = full(fK, 2 * (j + m));
                    if (!ok) break;
                    tc_fence_after();
                    issue_S(m, 0, fK.slot);
                    mma_commit(bar(Bars::kS + m));
                    free_slot(fK);
                    for (int i = m, q = 0; i < n; i += 2, ++q) {
                        ok = full(fV, 2 * (j + i) + 1) && mbar_wait(bar(Bars::kP + m), (n_p[m] + q) & 1, s_abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_PV(m, fV.slot, q > 0);
                        if (i + 2 >= n) mma_commit(bar(Bars::kO + m));
                        free_slot(fV);
                        fV.skip(4);
                        fK.skip(4);
                        if (i + 2 < n) {
                            ok = full(fK, 2 * (j + i) + 4);
                            if (!ok) break;
                            tc_fence_after();
                            issue_S(m, 0, fK.slot);
                            mma_commit(bar(Bars::kS + m));
                            free_slot(fK);
                        }
                    }
                }
                n_p[0] += by_tile ? (n + 1) / 2 : n;
                n_p[1] += by_tile ? n / 2 : n;
                j += n;
                if (j < count) p.next_unit(a);
            }
            if (!ok) my_err = 1;
            // every issued product completes before TMEM is released
            mma_commit(bar(Bars::kDone + me_m));
            volatile int never = 0;
            if (!mbar_wait(bar(Bars::kDone + me_m), 0, &never)) my_err = 1;
        }
    } else if (warp >= 4 && count > 0) {
        // ============================ softmax, a stream each warpgroup
        regs_inc<kRegsSoftmax>();
        const int wg = (warp - 4) >> 2, tw = (tid - 128) & 127;  // stream, row of its M tile (TMEM lane)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + wg * 128, tO = tmem + lane_base + 256 + wg * D;
        const float sl2 = a.scale_log2;
        Tile p = first;
        bool ok = true;
        int n_s = 0, n_o = 0;  // tiles and segments of this stream so far
        for (int j = 0, seg = 0; j < count; ++seg) {
            const int n = min(p.tiles - p.t, count - j);
            const bool by_tile = p.by_tile(), whole = n == p.tiles;
            if (ok) err_g = p.g;
            // This thread's row.  Up to 64 rows that both streams have lie in the tile twice, and the streams take one copy
            // each: their warps, of which a warp's time does not depend on how many rows it has, then run on
            // different schedulers (24 ragged groups with one key of their own 108 us, one copy 114; rows dealt round over all warps the same).
            const int r_tile = by_tile ? 0 : wg * 128, rows_here = min(128, p.rows() - r_tile);
            const bool twice = by_tile && rows_here <= 64;
            const int rl = tw - (twice ? 64 * wg : 0);
            const bool valid = rl >= 0 && rl < rows_here;
            const bool active = __any_sync(0xffffffffu, valid);
            // the place of a row, in [B, Hq]
            auto place_of = [&](int r) {
                const int x = p.row0() + r_tile + r, sq = x / a.gq;  // row and sequence of the item
                return (long long)(p.it.x + sq) * a.Hq + p.head() * a.gq + (x - sq * a.gq);
            };
            const long long place = place_of(max(rl, 0));
            if (!by_tile || wg == 0) {
                // Q rows: 64-element halves of [128 rows x 128 B], 16-byte chunk c of row r at c ^ (r & 7).  A warp copies
                // the rows of its threads, whole rows at a time.
                constexpr int kRowLanes = D / 8, kRows = 32 / kRowLanes;
                const int ql = twice ? tw & 63 : tw, c = lane % kRowLanes;
                const long long q_place = twice ? place_of(ql) : place;
                const bool have = ql < rows_here && TSV_IN_BOUNDS(q_place, (long long)a.B * a.Hq, a.seq_err + p.it.x);
                const int mine = have ? static_cast<int>(q_place) : -1;  // (at most 2^24 places)
                const uint32_t tile = smem_u32(smem + (r_tile >> 7) * SLOT) + (c >> 3) * kHalfBytes;
#pragma unroll
                for (int i = 0; i < 32; i += kRows) {
                    const int r = i + lane / kRowLanes, from = __shfl_sync(0xffffffffu, mine, r), t = (tw & ~31) + r;
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (long long)max(from, 0) * D) + c;
                    cp_async16(tile + (t >> 3) * 1024u + (t & 7) * 128u + (((c & 7) ^ (t & 7)) << 4), src, from >= 0);
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
            }
            // (neither issuer falls two segments behind, even where it has no tile in one.  After a wait that gave up the
            // arrivals go on: all threads' or none's, since a barrier must not get more of them than its phase has room for)
            if (seg > 0) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(Bars::kSeen), (seg - 1) & 1, s_abort));
                if (!ok) *s_abort = 1;
            }
            mbar_arrive(bar(Bars::kQ));
            float m_run = -INFINITY, l_run = 0.0f;
            int steps = 0;
            for (int i = by_tile ? wg : 0; i < n; i += by_tile ? 2 : 1) {
                if (!ok) break;
                const int left = p.it.z - (p.t + i) * kTileKeys;  // keys from the tile's first on
#ifdef TSV_TEST_HOOKS
                const bool stall = g_test_prefix_stall == n_s + 1 && wg == 0;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(stall ? Bars::kStall : Bars::kS + wg), stall ? 0 : n_s & 1, s_abort));
#else
                ok = __all_sync(0xffffffffu, mbar_wait(bar(Bars::kS + wg), n_s & 1, s_abort));
#endif
                if (!ok) {
                    *s_abort = 1;
                    break;
                }
                ++n_s;
                ++steps;
                tc_fence_after();
                if (active) {
                    uint32_t sv[128];
                    tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                    tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
                    tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
                    tmem_wait_ld();
                    if (left < kTileKeys) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) sv[c] = c < left ? sv[c] : 0xff800000u;  // -inf
                    }
                    float mxa[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) mxa[q] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 128; c += 16)
#pragma unroll
                        for (int q = 0; q < 8; ++q) mxa[q] = max3f(mxa[q], __uint_as_float(sv[c + 2 * q]), __uint_as_float(sv[c + 2 * q + 1]));
                    const float mx = sl2 * max3f(max3f(mxa[0], mxa[1], mxa[2]), max3f(mxa[3], mxa[4], mxa[5]), fmaxf(mxa[6], mxa[7]));
                    // The last product of this stream is done before O is rescaled: the issuer committed the S
                    // just waited for after it.  A segment's first product overwrites O.
                    bool rescale = false;
                    float factor = 1.0f;
                    if (m_run == -INFINITY) {
                        m_run = mx;
                    } else if (mx > m_run + 8.0f) {
                        factor = ex2(m_run - mx);
                        m_run = mx;
                        rescale = true;
                    }
                    l_run *= factor;
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                        for (int q4 = 0; q4 < D / 32; ++q4) {
                            uint32_t ov[32];
                            tmem_ld32(tO + q4 * 32, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * factor);
                            tmem_st32(tO + q4 * 32, ov);
                        }
                        tmem_wait_st();
                    }
                    // a row whose scores are all -inf so far keeps weights of 0
                    const float ref = m_run == -INFINITY ? 0.0f : m_run;
                    const unsigned long long sc2 = f2_pack(sl2, sl2), off2 = f2_pack(-ref, -ref);
                    unsigned long long la2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int q32 = 0; q32 < 64; q32 += 32) {
                        uint32_t hi[32], lo[32];
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * (q32 + q)]), __uint_as_float(sv[2 * (q32 + q) + 1])), sc2, off2), x0, x1);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            la2[q & 3] = f2_add(la2[q & 3], f2_pack(p0, p1));
                            split_bf16_up(p0, p1, &hi[q], &lo[q]);
                        }
                        tmem_st32(tS + q32, hi);
                        tmem_st32(tS + 64 + q32, lo);
                    }
                    tmem_wait_st();
                    float s0, s1, s2, s3, s4, s5, s6, s7;
                    f2_unpack(la2[0], s0, s1);
                    f2_unpack(la2[1], s2, s3);
                    f2_unpack(la2[2], s4, s5);
                    f2_unpack(la2[3], s6, s7);
                    l_run += ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
                }
                // V rows behind the prefix are zeroed before the product (they may hold anything, and 0 * NaN is
                // NaN); on a tile of both streams the first does it, whose product is issued first
                if (left < kTileKeys && (by_tile || wg == 0)) {
                    const int fV = 2 * (j + i) + 1;
                    int sent = 0;
                    ok = wait_sent(sent_at, fV, &sent, s_abort) && mbar_wait(bar(Bars::kFull + fV % nslots), (fV / nslots) & 1, s_abort);
                    if (ok) {
                        constexpr int kRowChunks = HALVES * 8, kRowsPerStep = 128 / kRowChunks;
                        uint8_t* vt = smem + lay.ring + (fV % nslots) * SLOT + ((tw % kRowChunks) >> 3) * kHalfBytes + (tw & 7) * 16;
                        for (int row = left + tw / kRowChunks; row < kTileKeys; row += kRowsPerStep)
                            *reinterpret_cast<uint4*>(vt + row * 128) = make_uint4(0, 0, 0, 0);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(Bars::kP + wg));
                if (by_tile && wg == 0 && tw == 0) mbar_arrive(bar(Bars::kP));  // (its issuer waits for the tile itself)
                if (!ok) *s_abort = 1;
            }
            // ---- the segment's (m, l, O)
            if (ok && steps > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(Bars::kO + wg), n_o & 1, s_abort));
                tc_fence_after();
                if (!ok) *s_abort = 1;
                ++n_o;
            }
            if (ok && active) {
                const long long row = whole ? place + (by_tile && wg ? 2LL * a.B * a.Hq : 0LL)
                                            : ((long long)me * 4 + (seg == 0 ? 0 : 2) + wg) * 128 + rl;
                const bool in = valid && TSV_IN_BOUNDS(row, whole ? 3LL * a.B * a.Hq : 512LL * a.tc_lanes, a.seq_err + p.it.x);
                float* o = (whole ? a.whole_o : a.tc_o) + (in ? row * D : 0);
                // They go through shared memory, so that a warp writes whole runs of a row and not 16 bytes of 32 rows:
                // a Q tile that no product reads any more, 16 KB or 32 (QT = 1 has none: streams of every other
                // tile share theirs)
                if (steps > 0 && QT == 2) {
                    constexpr int kCols = D == 128 ? 32 : 16, kChunks = kCols / 4, kRowsIt = 32 / kChunks;  // of a pass, of a row, of a store
                    uint8_t* stage = smem + (by_tile ? SLOT + (warp - 4) * 128 * kCols : wg * SLOT + (warp & 3) * 128 * kCols);
                    const unsigned rows_in = __ballot_sync(0xffffffffu, in);
                    auto swizzle = [](int row) { return kCols == 32 ? row & 7 : (row >> 1) & 3; };
                    const int row = lane / kChunks, chunk = lane % kChunks;  // of the first store; the next are kRowsIt rows on
                    float* to[kChunks];
#pragma unroll
                    for (int i = 0; i < kChunks; ++i)
                        to[i] = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), kRowsIt * i + row));
#pragma unroll 1
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        uint32_t ov[32];
                        tmem_ld32(tO + q4 * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 32 / kCols; ++h) {
                            __syncwarp();
#pragma unroll
                            for (int c = 0; c < kChunks; ++c)
                                *reinterpret_cast<uint4*>(stage + lane * 4 * kCols + ((c ^ swizzle(lane)) << 4)) =
                                    make_uint4(ov[h * kCols + 4 * c], ov[h * kCols + 4 * c + 1], ov[h * kCols + 4 * c + 2], ov[h * kCols + 4 * c + 3]);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < kChunks; ++i) {
                                const int r = kRowsIt * i + row;
                                if ((rows_in >> r) & 1u)
                                    reinterpret_cast<uint4*>(to[i] + q4 * 32 + h * kCols)[chunk] =
                                        *reinterpret_cast<const uint4*>(stage + r * 4 * kCols + ((chunk ^ swizzle(r)) << 4));
                            }
                        }
                    }
                } else if (steps > 0) {
#pragma unroll 1
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        uint32_t ov[32];
                        tmem_ld32(tO + q4 * 32, ov);
                        tmem_wait_ld();
                        if (in) {
#pragma unroll
                            for (int v4 = 0; v4 < 8; ++v4)
                                reinterpret_cast<uint4*>(o + q4 * 32)[v4] = make_uint4(ov[4 * v4], ov[4 * v4 + 1], ov[4 * v4 + 2], ov[4 * v4 + 3]);
                        }
                    }
                }
                if (in) {
                    (whole ? a.whole_m : a.tc_m)[row] = m_run;
                    (whole ? a.whole_l : a.tc_l)[row] = l_run;
                }
            }
            tc_fence_before();
            j += n;
            if (j < count) {
                p.next_unit(a);
                named_bar_sync(1, 256);  // both streams are done with Q
            }
        }
        if (!ok) my_err = 1;
    } else if (count == 0) {
        // ============================ the stream, last in the code: what lies at its beginning is fetched before the
        // CTAs' work begins, and the other roles' first tiles need it more (the stream in front: 64 samples of a 32k prompt 107
        // us, this way 102; 8 samples 21.1 and 19.5)
        if (warp < 4) {
            regs_dec<kRegsIdle>();
        } else {
            regs_inc<kRegsStream>();
            const int w = warp - 4;
            if (w < begin.y)
                stream_tiles<StreamCore>(a, begin.x + w, smem_u32(smem) + w * kRingBytes,
                                         reinterpret_cast<float*>(smem + kStreamWarps * kRingBytes) + w * kScratch);
        }
    }
    if (my_err) {
        *s_abort = 1;
        atomicMin(s_lost, err_g);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*s_lost < a.G) {
        const int4 from = a.tc_begin[2 * blockIdx.x];
        Tile p{};
        p.set(from.x, a.tc_begin[2 * blockIdx.x + 1]);
        p.unit = from.y;
        p.t = from.z;
        for (int left = from.w; left > 0;) {
            if (p.g >= *s_lost)
                for (int q = threadIdx.x; q < p.it.w / a.gq; q += kThreads) atomicOr(a.seq_err + p.it.x + q, TSV_DERR_TIMEOUT);
            left -= p.tiles - p.t;
            if (left > 0) p.next_unit(a);
        }
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int QT, int MT>
cudaError_t launch_tiles(const PrefixArgs& a, cudaStream_t stream) {
    CUtensorMap mk, mv;
    const long long rows = static_cast<long long>(a.num_blocks) << a.bs_log2;
    if (!make_cache_map(&mk, a.k_cache, D, a.Hkv, rows, 1 << a.bs_log2) || !make_cache_map(&mv, a.v_cache, D, a.Hkv, rows, 1 << a.bs_log2))
        return cudaErrorInvalidValue;
    constexpr int total = static_cast<int>(layout<D, QT>().total);
    thread_local int smem_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != smem_dev) {
        e = cudaFuncSetAttribute(prefix_tc_kernel<D, QT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, total);
        if (e != cudaSuccess) return e;
        smem_dev = dev;
    }
    return launch_pdl(prefix_tc_kernel<D, QT, MT>, dim3(static_cast<unsigned>(a.tc_lanes)), dim3(kThreads), total, stream, 1u, a, mk, mv);
}

template <int D, int MT>
cudaError_t launch_dim(const PrefixArgs& a, cudaStream_t stream) {
    // one Q tile where no group can have more rows, which leaves the ring another slot
    return (long long)a.B * a.gq > 128 ? launch_tiles<D, 2, MT>(a, stream) : launch_tiles<D, 1, MT>(a, stream);
}
template <int D>
cudaError_t launch_rows(const PrefixArgs& a, cudaStream_t stream) {
    return a.rows <= 16 ? launch_dim<D, 1>(a, stream) : launch_dim<D, 2>(a, stream);
}

}  // namespace

#ifdef TSV_TEST_HOOKS
// test build only: n = the next calls stall the wait for the n-th tile of each CTA's first stream until it gives up; 0 = none
extern "C" int tsv_test_set_prefix_stall(int mode) {
    return static_cast<int>(cudaMemcpyToSymbol(g_test_prefix_stall, &mode, sizeof(int)));
}
#endif

cudaError_t launch_prefix_tc(const PrefixArgs& a, cudaStream_t stream) {
    return a.D == 64 ? launch_rows<64>(a, stream) : launch_rows<128>(a, stream);
}

}  // namespace tsv
