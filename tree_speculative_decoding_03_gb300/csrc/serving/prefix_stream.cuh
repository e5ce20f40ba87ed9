// prefix_stream.cuh -- the stream of key tiles of prefix_attn.cu: a warp's share of the tiles of the sequences' own keys and, in
// fp32, of the shared prefixes.
#pragma once

#include "../common.cuh"
#include "continue_args.cuh"
#include "decode_core.cuh"

namespace tsv {
namespace {

constexpr int kStreamWarps = 8;    // of an SM: as many rings as its shared memory holds
constexpr int kRingBytes = 24576;  // of a warp
constexpr int kScratch = 136;      // floats of a warp beside its ring

// Whether an item has tiles in a kernel.  (The product of the two may be 2^32: a prefix of 2^20 fp32 keys with heads of
// 64 and the 2^19 rows of 8192 sequences of 64 heads to one K/V head.)
__host__ __device__ constexpr bool has_tiles(int tiles, int units) { return tiles > 0 && units > 0; }
static_assert(has_tiles(1 << 16, 1 << 16) && !has_tiles(0, 5) && !has_tiles(5, 0), "without the product's 32 bits");

// Tiles of an item: from the tile that holds its first key.
template <int TILE>
__device__ __forceinline__ int item_tiles(const int4& it) {
    return it.z > it.y ? (it.z + TILE - 1) / TILE - it.y / TILE : 0;
}
// Units of item i in the stream, a team at a time.  With a tensor-core kernel the prefixes are that one's.
__device__ __forceinline__ int item_units(const PrefixArgs& a, int i, const int4& it) {
    return i < a.G && a.tc_lanes > 0 ? 0 : ((it.w + a.rows - 1) / a.rows) * (a.Hkv / a.team);
}
// ------------------------------------------------------------------ the schedule

// A position in the row of tiles: tile t of the `tiles` of item i, for its `chunk`-th group of rows and
// the team's `heads`-th run of kv heads.
struct Place {
    int i, chunk, heads, t, tiles, units;
    int4 it;     // first sequence, first key, end, rows
    int4 ahead;  // the next item, on its way while this one lasts
    template <int TILE>
    __device__ __forceinline__ void set(const PrefixArgs& a, int item, const int4& now) {
        i = item;
        it = now;
        if (item + 1 < a.G + a.B) ahead = a.item[item + 1];
        tiles = item_tiles<TILE>(it);
        units = item_units(a, i, it);
    }
    template <int TILE>
    __device__ __forceinline__ void next(const PrefixArgs& a) {
        if (++t < tiles) return;
        t = 0;
        ++heads;
        if (heads * a.team < a.Hkv) return;
        heads = 0;
        if (++chunk * a.rows < it.w) return;
        chunk = 0;
        do {
            set<TILE>(a, i + 1, ahead);
        } while (!has_tiles(tiles, units) && i + 1 < a.G + a.B);
    }
    __device__ __forceinline__ int head(const PrefixArgs& a, int member) const { return heads * a.team + member; }
    __device__ __forceinline__ int rows(const PrefixArgs& a) const { return min(a.rows, it.w - chunk * a.rows); }
};

// ------------------------------------------------------------------ the stream of tiles

template <typename Core>
__host__ __device__ constexpr int stages_of() { return kRingBytes / (2 * Core::KEYS * Core::ROWB); }

// A warp's stream of tiles: the copies run STAGES - 1 tiles ahead and the block ids one more.
template <typename Core>
struct Stream {
    using Elem = typename Core::Elem;
    static constexpr int D = Core::D, KEYS = Core::KEYS, STAGES = stages_of<Core>(), RUNS = KEYS / 8;
    static constexpr uint32_t HALF = KEYS * Core::ROWB, STAGE = 2 * HALF;
    static constexpr int LANES_ROW = Core::CH < 32 ? Core::CH : 32, ROWS_IT = 32 / LANES_ROW;
    const PrefixArgs& a;
    const uint32_t ring;
    const int member, row_elems, lrow, lane_elems, lch;
    Place f;           // the tile whose ids were fetched last
    int ids[RUNS];     // its blocks (8 keys lie in one block); all lanes hold the same
    uint32_t bad = 0;  // stages holding a tile with a block id outside the cache
    int left;          // tiles not yet on their way
    int fill = 0, stage = 0;

    __device__ __forceinline__ Stream(const PrefixArgs& args, uint32_t ring_, int member_, const Place& p, int n)
        : a(args), ring(ring_), member(member_), row_elems(args.Hkv * D), lrow((threadIdx.x & 31) / LANES_ROW),
          lane_elems(lrow * row_elems + ((threadIdx.x & 31) % LANES_ROW) * (16 / (int)sizeof(Elem))), lch((threadIdx.x & 31) % LANES_ROW),
          f(p), left(n) {}

    // the tile's first key; the item's first key may lie behind it
    __device__ __forceinline__ static int first_key(const Place& p) { return (p.it.y / KEYS + p.t) * KEYS; }
    __device__ __forceinline__ bool holds(int key) const { return key < f.it.z && key + 8 > f.it.y; }
    __device__ __forceinline__ void fetch() {
        const int32_t* bt = a.block_table + (long long)f.it.x * a.max_blocks;
#pragma unroll
        for (int u = 0; u < RUNS; ++u) {
            const int key = first_key(f) + 8 * u;
            ids[u] = holds(key) ? (TSV_IN_BOUNDS(key >> a.bs_log2, a.max_blocks, nullptr) ? bt[key >> a.bs_log2] : -1) : 0;
        }
    }
    // sends tile f on its way into stage `fill`, then fetches the next tile's ids
    __device__ __forceinline__ void load() {
        if (left > 0) {
            const uint32_t dst = ring + fill * STAGE;
            const Elem* kc = static_cast<const Elem*>(a.k_cache);
            const Elem* vc = static_cast<const Elem*>(a.v_cache);
            const long long head = (long long)f.head(a, member) * D + lane_elems;
            bool wrong = false;
#pragma unroll
            for (int u = 0; u < RUNS; ++u) {
                const int key = first_key(f) + 8 * u;
                const bool in = static_cast<unsigned>(ids[u]) < static_cast<unsigned>(a.num_blocks);
                wrong |= !in && holds(key);
                const long long at = head + (((long long)(in ? ids[u] : 0) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))) * row_elems;
#pragma unroll
                for (int r0 = 0; r0 < 8; r0 += ROWS_IT) {
                    // rows outside the item's keys are zeros: they may hold anything, and 0 * NaN is NaN
                    const int row = key + r0 + lrow;
                    bool take = in && row >= f.it.y && row < f.it.z;
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
    // waits for the next tile, and for all lanes' use of the one before
    __device__ __forceinline__ void wait() {
        cp_wait<STAGES - 2>();
        __syncwarp();
    }
    // adds the next tile, p, to the core's state; true if a block id of it is outside the cache
    __device__ __forceinline__ bool step(Core& core, const Place& p, float* scratch) {
        const uint32_t src = ring + stage * STAGE;
        const bool wrong = ((bad >> stage) & 1u) != 0;
        const int first = first_key(p);
        core.step(src, src + HALF, p.it.y - first, p.it.z - first, a.scale_log2, scratch);
        __syncwarp();
        if (++stage == STAGES) stage = 0;
        return wrong;
    }
};

// Query rows from row `row` of the item on: row r is head r % gq (of the kv head) of its sequence r / gq.
template <typename Elem, int D>
struct ItemRows {
    const Elem* q;  // the kv head's first row of the item's first sequence
    int row, gq, seq;  // seq: elements from a sequence to the next
    __device__ __forceinline__ const Elem* operator()(int r) const {
        const int x = row + r, s = x < gq ? 0 : x / gq;
        return q + (long long)s * seq + (x - s * gq) * D;
    }
};
template <typename Core>
__device__ __forceinline__ void load_rows(const PrefixArgs& a, const Place& p, int member, Core& core) {
    using Elem = typename Core::Elem;
    const Elem* q = static_cast<const Elem*>(a.q) + ((long long)p.it.x * a.Hq + p.head(a, member) * a.gq) * Core::D;
    core.load_q(ItemRows<Elem, Core::D>{q, p.chunk * a.rows, a.gq, a.Hq * Core::D}, p.rows(a));
}

// Where the rows of a whole unit go: each to its own place.
template <int D>
struct ToPlaces {
    float *o, *m, *l;
    int row, gq, Hq;
    long long first;  // the place of the item's row 0
    __device__ __forceinline__ long long place(int r) const {
        const int x = row + r, s = x < gq ? 0 : x / gq;
        return first + (long long)s * Hq + (x - s * gq);
    }
    __device__ __forceinline__ void row_(int r, float m_, float l_) const {
        m[place(r)] = m_;
        l[place(r)] = l_;
    }
};
template <int D>
struct Leave {
    ToPlaces<D> whole;
    ToSlot<D> slot;
    bool in_slot;
    __device__ __forceinline__ void row(int r, float m, float l) const {
        if (in_slot)
            slot.row(r, m, l);
        else
            whole.row_(r, m, l);
    }
    __device__ __forceinline__ float factor(float) const { return 1.0f; }
    __device__ __forceinline__ float* base(int r) const { return in_slot ? slot.base(r) : whole.o + whole.place(r) * D; }
};

// One warp, the me-th of all: its tiles.
template <typename Core>
__device__ __forceinline__ void stream_tiles(const PrefixArgs& a, int me, uint32_t ring, float* scratch) {
    constexpr int D = Core::D, KEYS = Core::KEYS;
    const int lane = threadIdx.x & 31, which = me / a.team, member = me % a.team;
    if (which >= a.lanes) return;
    const int4 begin = a.begin[3 * which], item = a.begin[3 * which + 1];
    const int n = a.begin[3 * which + 2].x;
    if (n == 0) return;
    Place p{};
    p.set<KEYS>(a, begin.x, item);
    p.chunk = begin.y;
    p.heads = begin.z;
    p.t = begin.w;
    Stream<Core> stream(a, ring, member, p, n);
    stream.fetch();
    Core core;
    bool seg_begins = true, seg_bad = false;
    int seg = 0, t_first = p.t;
    // (One copy of each part in the code, which the first tiles wait for: with the copies ahead unrolled and the rows
    // loaded in two places it is 107 KB, this way 28; 32 sequences of 3000 to 4000 keys 102 us and 88.)
#pragma unroll 1
    for (int i = 1 - Stream<Core>::STAGES; i < n; ++i) {
        if (i >= 0) stream.wait();
        stream.load();
        if (i < 0) continue;
        if (seg_begins) {
            load_rows(a, p, member, core);
            core.reset();
            seg_begins = false;
        }
        seg_bad |= stream.step(core, p, scratch);
        if (p.t + 1 < p.tiles && i + 1 < n) {
            ++p.t;
            continue;
        }
        // the segment's end
        const bool prefix = p.i < a.G, piece = t_first > 0 || p.t + 1 < p.tiles;
        const long long rows = (long long)a.B * a.Hq, slot = 2LL * me + (seg == 0 ? 0 : 1);
        const int row0 = p.chunk * a.rows;
        if (!TSV_IN_BOUNDS(slot, 2LL * a.lanes * a.team, a.seq_err + p.it.x)) return;
        const Leave<D> to{
            {a.whole_o, a.whole_m, a.whole_l, row0, a.gq, a.Hq, (prefix ? 0 : rows) + (long long)p.it.x * a.Hq + p.head(a, member) * a.gq},
            {a.part_o + slot * a.rows * D, a.part_m + slot * a.rows, a.part_l + slot * a.rows},
            piece};
        core.finish(p.rows(a), to, scratch);
        if (seg_bad)  // the sequences of the unit's rows are told
            for (int s = row0 / a.gq + lane; s <= (row0 + p.rows(a) - 1) / a.gq; s += 32) atomicOr(a.seq_err + p.it.x + s, TSV_DERR_BLOCK);
        if (i + 1 < n) {
            p.next<KEYS>(a);
            t_first = 0;
            seg_bad = false;
            ++seg;
            seg_begins = true;
        }
    }
}

}  // namespace
}  // namespace tsv
