// What the attention and the weights kernel share: a block's shape, its share
// of the work, the loading of keys and queries, and the scores' products.
// mla.cu describes the whole.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "blackwell.cuh"
#include "mla.cuh"

namespace kvpub {

constexpr int kUnit = 128;                  // keys a step
constexpr int kBlockBytes = KVPUB_BLOCK_SIZE * KVPUB_MAIN_SLOT_BYTES;
constexpr int kSlotBytes = kUnit * 128;     // one tile of a unit
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// kValues: attention; without it only the scores are formed (the weights).
template <int kRowsOf, bool kValues>
struct Shape {
    static constexpr int kRows = kRowsOf;
    static constexpr bool kHasValues = kValues;
    // softmax warps: four for the 128 lanes, times the parts that share the rows
    static constexpr int kWarps = kRows == 16 ? 8 : 16;
    static constexpr int kParts = kWarps / 4;
    static constexpr int kCols = kRows / kParts;           // rows a thread
    static constexpr int kLoadWarp = kWarps;
    static constexpr int kScoreWarp = kWarps + 1;
    static constexpr int kValueWarp = kWarps + 2;
    static constexpr int kKeyWarp = kWarps + 3;
    static constexpr int kThreads = (kWarps + 4) * 32;
    // registers a thread: 20 warps start with 96, and the last four of them
    // leave 64 of theirs to the others (16 each); 12 warps have enough
    static constexpr bool kMoveRegisters = kValues && kWarps == 16;
    static constexpr int kSlots =
        kValues ? (kRows == 64 ? 8 : kRows == 32 ? 9 : 11) : (kRows == 64 ? 9 : 11);
    // A unit's score pieces are waited for and handed on in bunches of kPer:
    // all five, or as many as tensor memory holds two bunches of beside the
    // values' accumulators.
    static constexpr int kPer = kRows < 64 ? 5 : kValues ? 2 : 4;
    static constexpr int kScores = kValues ? 4 * kRows : 0;    // their first column
    static constexpr int kBunches = (5 + kPer - 1) / kPer;     // a unit
    static constexpr int kFull = kRows == 64 ? 6 : 4;          // barriers of loaded bunches
    static constexpr int kGroups = kRows / 16;             // 128-byte rows of P a key
    static constexpr int kTiles = 4 / kGroups > 0 ? 4 / kGroups : 1;   // tiles a group
    static constexpr int kProbs = !kValues ? 0 : kRows == 32 ? 2 : 1;     // P buffers
    // What a segment costs beside its units, in units (queries in, results
    // out and joined, the pipeline's start, first units that move their
    // references more often). Measured without it and with 1 to 4, us: 24 ragged
    // trees of 32 heads (64 rows) 115, 99, 81, 80, 84; 28 sequences of 10k
    // tokens, 32 heads (32 rows) 68, 65, 64, 67, 67; 64 ragged sequences of 16
    // heads 64, 57, 52, 54, 54.
    static constexpr int kOver = !kValues ? 0 : kRows <= 32 ? 2 : 3;
    static constexpr int kColumns = kRows == 16 ? 256 : 512;   // tensor memory
    static constexpr int kQueryTile = kRows * 128;
    static constexpr int kQueryOff = kSlots * kSlotBytes;  // hi 0-3, lo 4-7, rope 8
    static constexpr int kProbOff = kQueryOff + 9 * kQueryTile;
    static constexpr int kMiscOff = kProbOff + kProbs * kSlotBytes;
    static_assert(kGroups * kTiles == 4 && 2 * kRows * kTiles == 128, "P rows are 128 bytes");
    static_assert(kScores + 2 * kPer * kRows <= kColumns, "tensor memory");
    static_assert(kFull % kBunches == 0, "a bunch's barrier knows its size");
    static_assert(kFull / kBunches * 5 >= kSlots, "a bunch's barrier is not in use when its turn comes");
};

// A run of units of one item (a tile of rows of a sequence).
struct Segment {
    Sequence s;
    int seq, tile;
    int begin, end, units;
    bool counts;      // the first of its units to count invalid blocks
};

// What is left of the attention's share: steps of a tile of rows after one
// another, then the sequence's next tile.  An item's steps are `over` empty
// ones, for what a segment costs by itself, and its units.
struct Cursor {
    int seq, tile, step, over;
    int64_t left;
};

template <class S>
struct Misc {
    alignas(16) float scales[2][kUnit][4];
    uint4 keys[S::kHasValues ? kUnit : 192];    // see key_role; or the parts' sums
    uint64_t mask[S::kRows];
    // The four warps of a part write equal values to nref, fac and shift, and none
    // comes round to write again before all have passed the next barrier.
    alignas(16) float factor[S::kRows];            // softmax_scale * log2(e) / the query's power of two
    alignas(16) float nref[S::kRows];              // kShift - the rows' references
    alignas(16) float fac[S::kRows];
    alignas(16) float shift[S::kRows];
    int grown[3][S::kRows];         // what outgrew its reference, fp32 bits; 0: nothing
    float wmax[4][S::kRows];
    float part_lse[S::kRows];          // in a cluster: of this block's part, base 2
    // attention: where a row's output is, in elements (-1: no row); this
    // segment's and the next one's
    int64_t out_at[S::kHasValues ? 2 : 1][S::kHasValues ? S::kRows : 1];
    uint64_t bunch_full[6];         // loaded
    uint64_t slot_empty[11];
    uint64_t piece_full[2], piece_empty[2];
    uint64_t prob_full[2], prob_empty[2];
    uint64_t scale_full[2], scale_empty[2];
    uint64_t keys_full, query_ready, drain[2];
    int64_t total, offset;
    // The softmax warps' place, here and not in their registers, of which they
    // are short.
    Cursor cursor;
    Segment segments[2];
    int seq;
    int valid[2];                   // which of the unit's two blocks exist
    uint32_t ratios;                // with keys: the tiles' largest ratios
    uint32_t tmem;
    int abort;
    // before the work starts
    __device__ __forceinline__ int64_t *scan() { return reinterpret_cast<int64_t *>(wmax); }
};

// Shared-memory addresses of a block's barriers, from the address of Misc.
template <class S>
struct Bars {
    uint32_t base;
    __device__ __forceinline__ uint32_t bunch_full(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, bunch_full)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t slot_empty(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, slot_empty)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t piece_full(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, piece_full)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t piece_empty(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, piece_empty)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t prob_full(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, prob_full)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t prob_empty(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, prob_empty)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t scale_full(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, scale_full)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t scale_empty(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, scale_empty)) + 8 * i;
    }
    __device__ __forceinline__ uint32_t keys_full() const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, keys_full));
    }
    __device__ __forceinline__ uint32_t query_ready() const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, query_ready));
    }
    __device__ __forceinline__ uint32_t drain(int i) const {
        return base + static_cast<uint32_t>(offsetof(Misc<S>, drain)) + 8 * i;
    }
};

// Waits of a role whose warps must not leave it (it has named barriers to
// keep): after one that ran out it goes on without waiting, and what it writes
// then is NaN.  Where another role gave up, these waits run out too: they are
// for what that role no longer hands on.
template <class S>
struct Waiter {
    Misc<S> &m;
    bool alive;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
        if (alive && !mbar_wait(bar, parity)) {
            alive = false;
            m.abort = 1;
        }
    }
};

template <class S>
constexpr int smem_bytes() {
    return S::kMiscOff + static_cast<int>(sizeof(Misc<S>));
}

// ------------------------------------------------------------------ the work

__device__ __forceinline__ int units_of(const Sequence &s) {
    return s.len <= kUnit ? 1 : (s.len + kUnit - 1) / kUnit;
}

// The most units of a sequence under a block table of this width.
__host__ __device__ __forceinline__ int units_at_most(int64_t max_blocks) {
    static_assert(kUnit == 2 * KVPUB_BLOCK_SIZE, "two blocks a unit");
    return max_blocks <= 2 ? 1 : static_cast<int>((max_blocks + 1) / 2);
}

template <class S>
__device__ __forceinline__ int tiles_of(const MlaArgs &a, const Sequence &s) {
    const int tiles = (s.count * a.num_heads + S::kRows - 1) / S::kRows;
    // without query tokens a running sum still decays
    return tiles == 0 && !S::kHasValues ? 1 : tiles;
}

// Inclusive sum over the block.
template <int kThreads>
__device__ __forceinline__ int64_t block_sum_scan(int64_t v, int64_t *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < kThreads / 32; ++w) before += w < warp ? warps[w] : 0;
    return v + before;
}

// This block's equal share of all items' steps (see Cursor), found by a scan
// over the sequences: `left` of them from the `offset`-th of sequence `seq` on.
// All threads call it; m.total is their number.
struct Share {
    int seq, over;
    int64_t offset, left;
};

// total * i / n and value / by, in 32 bits where they fit (i, n <= kMaxCtas).
__device__ __forceinline__ int64_t portion(int64_t total, int i, int n) {
    if (total < (1 << 24)) return static_cast<uint32_t>(total) * i / static_cast<uint32_t>(n);
    return total * i / n;
}

__device__ __forceinline__ int64_t quotient(int64_t value, int by) {
    if (value <= INT32_MAX) return static_cast<uint32_t>(value) / static_cast<uint32_t>(by);
    return value / by;
}

// The block of n whose portion holds unit `at`.
__device__ __forceinline__ int block_of(int64_t at, int64_t total, int n) {
    return static_cast<int>(((at + 1) * n - 1) / total);
}

template <class S>
__device__ Share find_work(const MlaArgs &a, Misc<S> &m, int *blocks) {
    constexpr int kThreads = S::kThreads;
    const int tid = threadIdx.x;
    // units, and items times 2^40 (at most 65,535 sequences of 128 tiles); of
    // calls that may have 2^40 units, the units alone
    constexpr int kItems = 40;
    const int64_t most = static_cast<int64_t>(a.num_seqs) *
                         ((a.max_query_len * a.num_heads + S::kRows - 1) / S::kRows) *
                         (a.max_blocks / 2 + 1);
    const bool weigh = S::kOver != 0 && most < (1ll << kItems);
    auto work = [&](int b) -> int64_t {
        if (b >= a.num_seqs) return 0;
        const Sequence s = sequence(a, b);
        const int64_t tiles = tiles_of<S>(a, s);
        return tiles * units_of(s) + (weigh ? tiles << kItems : 0);
    };
    const int64_t first = work(tid);
    int64_t mine = first;
    for (int b = tid + kThreads; b < a.num_seqs; b += kThreads) mine += work(b);
    const int64_t sum = block_sum_scan<kThreads>(mine, m.scan());
    if (tid == kThreads - 1) m.total = sum;
    __syncthreads();
    const int64_t units_mask = weigh ? (1ll << kItems) - 1 : -1ll;
    const int64_t units = m.total & units_mask;
    // With few units a block the longest run of them counts.
    const int over = weigh && units >= 4 * gridDim.x ? S::kOver : 0;
    auto steps = [&](int64_t w) {
        return (w & units_mask) + (over != 0 ? (w >> kItems) * over : 0);
    };
    const int64_t total = steps(m.total);
    *blocks = static_cast<int>(units < gridDim.x ? units : gridDim.x);
    Share c{0, over, 0, 0};
    __syncthreads();                    // all have read m.total
    if (tid == 0) m.total = total;
    if (static_cast<int>(blockIdx.x) >= *blocks) return c;
    const int64_t begin = portion(total, blockIdx.x, *blocks);
    c.left = portion(total, blockIdx.x + 1, *blocks) - begin;
    auto found = [&](int b, int64_t end, int64_t v) {
        if (begin >= end - v && begin < end) {
            m.seq = b;
            m.offset = begin - (end - v);
        }
    };
    if (a.num_seqs <= kThreads) {
        found(tid, steps(sum), steps(first));
        __syncthreads();
    } else {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
            const int64_t v = steps(work(b0 + tid));
            const int64_t end = base + block_sum_scan<kThreads>(v, m.scan());
            found(b0 + tid, end, v);
            if (tid == kThreads - 1) m.total = end;
            __syncthreads();
            base = m.total;
            __syncthreads();
            if (base > begin) break;
        }
        if (tid == 0) m.total = total;
        __syncthreads();
    }
    c.seq = m.seq;
    c.offset = m.offset;
    return c;
}

// ------------------------------------------------------------------ loading

// A position in a ring: slot number and how often the ring has been passed.
template <int kN>
struct Ring {
    int at = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void step(int n = 1) {
        at += n;
        if (at >= kN) {
            at -= kN;
            pass ^= 1;
        }
    }
};

// The position after `count` steps from the start.
template <int kN>
__device__ __forceinline__ Ring<kN> ring_at(uint32_t count) {
    Ring<kN> r;
    r.at = static_cast<int>(count % kN);
    r.pass = (count / kN) & 1;
    return r;
}

// The load warp: the five tiles and the scales of every unit.  A block that
// the sequence does not have, or whose table entry is out of range, is
// loaded from the row past the cache's end, which TMA fills with zeros.
template <class S, typename Source>
__device__ void load_role(const MlaArgs &a, const CUtensorMap *tiles, const CUtensorMap *scales,
                          uint8_t *smem, Misc<S> &m, Source source) {
    const int lane = threadIdx.x & 31;
    const int past = static_cast<int>(a.num_blocks * KVPUB_BLOCK_SIZE);
    const Bars<S> bars{smem_addr(&m)};
    Ring<S::kSlots> ring;
    Ring<S::kFull> bunch;
    Ring<2> sring;
    int issued = 0, scales_issued = 0;     // whole bunches, scales
    Segment g;
    bool ok = true;
    while (ok && source.next(a, g)) {
        unsigned long long bad = (g.counts && g.begin == 0 && g.s.clamped) ? 1 : 0;
        int32_t id = -1;
        for (int u = g.begin; ok && u < g.end; ++u) {
            const int in = (u - g.begin) & 15;
            if (in == 0) {
                const int page = 2 * u + lane;
                id = static_cast<int64_t>(page) * KVPUB_BLOCK_SIZE < g.s.len
                         ? a.block_table[g.seq * a.table_stride + page]
                         : -2;
                const bool there = static_cast<int64_t>(page) * KVPUB_BLOCK_SIZE < g.s.len &&
                                   page < 2 * g.end;
                if (g.counts)
                    bad += __popc(__ballot_sync(~0u, there && (id < 0 || id >= a.num_blocks)));
            }
            const int p0 = __shfl_sync(~0u, id, 2 * in), p1 = __shfl_sync(~0u, id, 2 * in + 1);
            if (lane == 0) {
                const bool v0 = p0 >= 0 && p0 < a.num_blocks, v1 = p1 >= 0 && p1 < a.num_blocks;
                const int y0 = v0 ? p0 * KVPUB_BLOCK_SIZE : past;
                const int y1 = v1 ? p1 * KVPUB_BLOCK_SIZE : past;
                for (int i = 0; ok && i < 5; ++i) {
                    const uint32_t full = bars.bunch_full(bunch.at);
                    ok = mbar_wait(bars.slot_empty(ring.at), ring.pass ^ 1);
                    if (!ok) break;
                    const uint32_t dst = smem_addr(smem) + ring.at * kSlotBytes;
                    const int x = i == 0 ? KVPUB_LATENT_DIM + 16 : (i - 1) * 128;
                    mbar_expect_tx(full, kSlotBytes);
                    tma_load_2d(dst, tiles, x, y0, full);
                    tma_load_2d(dst + kSlotBytes / 2, tiles, x, y1, full);
                    ring.step();
                    if (i % S::kPer == S::kPer - 1 || i == 4) {
                        bunch.step();
                        ++issued;
                    }
                    if (i == 0) {
                        const uint32_t sf = bars.scale_full(sring.at);
                        ok = mbar_wait(bars.scale_empty(sring.at), sring.pass ^ 1);
                        if (!ok) break;
                        m.valid[sring.at] = (v0 ? 1 : 0) | (v1 ? 2 : 0);
                        const uint32_t sd = smem_addr(m.scales[sring.at]);
                        mbar_expect_tx(sf, kUnit * 16);
                        tma_load_2d(sd, scales, KVPUB_LATENT_DIM, y0, sf);
                        tma_load_2d(sd + kUnit * 8, scales, KVPUB_LATENT_DIM, y1, sf);
                        ++scales_issued;
                        sring.step();
                    }
                }
            }
            ok = __shfl_sync(~0u, ok, 0);
        }
        if (lane == 0 && bad != 0 && a.invalid_count != nullptr) atomicAdd(a.invalid_count, bad);
    }
    if (!ok && lane == 0) {
        m.abort = 1;
        // given up: let the copies in flight land before the block ends
        // (a bunch that was not issued whole leaves its barrier's phase open:
        // its copies are older than the limit of the wait that ran out)
        for (int i = 0; i < S::kFull && i < issued; ++i)
            for (int k = 0; k < 4096; ++k)
                if (mbar_try_wait(bars.bunch_full(i), i < bunch.at ? bunch.pass : bunch.pass ^ 1))
                    break;
        for (int i = 0; i < 2 && i < scales_issued; ++i)
            for (int k = 0; k < 4096; ++k)
                if (mbar_try_wait(bars.scale_full(i), i < sring.at ? sring.pass : sring.pass ^ 1))
                    break;
    }
    __syncwarp();
}

// Softmax warps: the segment's query rows into shared memory, each scaled by
// a power of two to a largest value in [128, 256) and split into E4M3 and
// E5M2 (exact for values of at least 2^-13 of the largest, the others off by at
// most 2^-21 of it), the rope kept in bf16.
template <class S>
__device__ void load_queries(const MlaArgs &a, const Segment &g, uint8_t *smem, Misc<S> &m,
                             int64_t *out_at) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = g.s.count * a.num_heads;
    // two rows a warp at a time: the code, which is cold, stays short
    constexpr int kAll = S::kRows / S::kWarps, kEach = kAll < 2 ? kAll : 2;
#pragma unroll 1
    for (int j0 = 0; j0 < kAll; j0 += kEach) {
        uint4 xs[kEach][2];
        uint32_t ropes[kEach];
        uint2 masks[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {     // all of the warp's loads at once
            const int row = g.tile * S::kRows + warp + (j0 + j) * S::kWarps;
            const bool live = row < rows;
            const int i = static_cast<unsigned>(row) / static_cast<unsigned>(a.num_heads);
            const int head = row - i * a.num_heads;
            const int64_t token = g.s.first + i;
            const uint16_t *ql = a.q_latent + token * a.q_latent_token + head * a.q_latent_head;
            const uint16_t *qr = a.q_rope + token * a.q_rope_token + head * a.q_rope_head;
            xs[j][0] = load16_if(live, ql + 16 * lane);
            xs[j][1] = load16_if(live, ql + 16 * lane + 8);
            ropes[j] = load4_if(live, qr + 2 * lane);
            if (a.tree_mask != nullptr) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(a.tree_mask + token);
                masks[j] = make_uint2(load4_if(live, w), load4_if(live, w + 1));
            } else {
                const uint64_t chain = live ? chain_mask(i) : 0;
                masks[j] = make_uint2(static_cast<uint32_t>(chain), static_cast<uint32_t>(chain >> 32));
            }
            if (S::kHasValues && lane == 0)
                out_at[warp + (j0 + j) * S::kWarps] =
                    live ? token * a.out_token + head * a.out_head : -1;
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int r = warp + (j0 + j) * S::kWarps;
            const uint4(&x)[2] = xs[j];
            const uint32_t rope = ropes[j];
            const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
            uint32_t top = rope & 0x7fff7fffu;
            for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
            top = __reduce_max_sync(~0u, top);
            // 2^k with k = 7 - floor(log2(largest)), kept in [-120, 100]
            int k = 7 + 127 - static_cast<int>(top >> 7);
            k = top == 0 ? 0 : (k > 100 ? 100 : (k < -120 ? -120 : k));
            const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            uint32_t hi[4], lo[4];
            for (int e = 0; e < 4; ++e) {
                const uint32_t v0 = w[2 * e], v1 = w[2 * e + 1];
                split_f8(half2_from(__uint_as_float(v0 << 16) * up,
                                    __uint_as_float(v0 & 0xffff0000u) * up),
                         half2_from(__uint_as_float(v1 << 16) * up,
                                    __uint_as_float(v1 & 0xffff0000u) * up),
                         hi[e], lo[e]);
            }
            uint8_t *q = smem + S::kQueryOff + (lane >> 3) * S::kQueryTile + r * 128 +
                         (((lane & 7) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4 *>(q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(q + 4 * S::kQueryTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            const float ra = __uint_as_float(rope << 16) * up;
            const float rb = __uint_as_float(rope & 0xffff0000u) * up;
            uint8_t *qr = smem + S::kQueryOff + 8 * S::kQueryTile + r * 128 +
                          (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2);
            // exact: only the exponent changes
            *reinterpret_cast<uint32_t *>(qr) =
                (__float_as_uint(ra) >> 16) | (__float_as_uint(rb) & 0xffff0000u);
            if (lane == 0) {
                // a NaN or Inf in the query makes the whole row NaN
                m.factor[r] = top >= 0x7f80u ? __uint_as_float(0x7fffffffu)
                                             : a.softmax_scale * kLog2e * down;
                m.mask[r] = masks[j].x | static_cast<uint64_t>(masks[j].y) << 32;
            }
        }
    }
}

// ----------------------------------------------------------------- products

// The scores' piece i (0 rope, 1-4 latent tiles) into tensor memory `d`.
template <class S>
__device__ __forceinline__ void score_piece(uint32_t smem, int slot, int i, uint32_t d) {
    const uint64_t key = operand_desc(smem + slot * kSlotBytes);
    const uint64_t query = operand_desc(smem + S::kQueryOff);
    constexpr uint64_t tile = S::kQueryTile >> 4;
    if (i == 0) {
        constexpr uint32_t desc = mma_desc(kBf16, kBf16, S::kRows, false);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_f16(d, key + 2 * k, query + 8 * tile + 2 * k, desc, k != 0);
    } else {
        constexpr uint32_t hi = mma_desc(kE4m3, kE4m3, S::kRows, false);
        constexpr uint32_t lo = mma_desc(kE4m3, kE5m2, S::kRows, false);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_f8(d, key + 2 * k, query + (i - 1) * tile + 2 * k, hi, k != 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_f8(d, key + 2 * k, query + (i + 3) * tile + 2 * k, lo, 1);
    }
}

// Where a thread of the softmax warps stands.
struct Lane {
    int warp, lane, part, key;
    uint32_t tmem;      // its lanes of tensor memory
};

__device__ __forceinline__ Lane softmax_lane(uint32_t tmem) {
    Lane t;
    t.warp = threadIdx.x >> 5;
    t.lane = threadIdx.x & 31;
    t.part = t.warp >> 2;
    t.key = (t.warp & 3) * 32 + t.lane;
    t.tmem = tmem + (static_cast<uint32_t>((t.warp & 3) * 32) << 16);
    return t;
}

// One bunch of this thread's key's scores against its part of the rows, in
// units of the rows' factors: to acc (zero before the first) the rope's piece
// and scale[t] * the tiles' pieces. The loops stay loops: what a unit runs
// through should fit the instruction caches.
template <class S>
__device__ __forceinline__ void add_bunch(const Lane &t, const Bars<S> &bars, Waiter<S> &wait,
                                          Ring<2> pieces, int bunch, const float *scale,
                                          float2 (&acc)[S::kCols / 2]) {
    constexpr int kC = S::kCols;
    wait(bars.piece_full(pieces.at), pieces.pass);
    tcgen05_after_sync();
    uint32_t at = t.tmem + S::kScores + pieces.at * S::kPer * S::kRows + t.part * kC;
    const int first = bunch * S::kPer, end = min(first + S::kPer, 5);
#pragma unroll 1
    for (int i = first; i < end; ++i) {
        float v[kC];
        tmem_load<kC>(at, v);
        const float w = i == 0 ? 1.f : scale[i - 1];
        tmem_load_wait();
#pragma unroll
        for (int c = 0; c < kC / 2; ++c)
            acc[c] = fma2(make_float2(w, w), make_float2(v[2 * c], v[2 * c + 1]), acc[c]);
        at += S::kRows;
    }
    tcgen05_before_sync();
    __syncwarp();
    if (t.lane == 0) mbar_arrive(bars.piece_empty(pieces.at));
}

// The warps that issue the products, one for the scores and one for the
// values. The whole warp runs and one lane issues: with everything uniform
// over the warp a product costs the tensor pipe's time (40 cycles at 16 rows,
// 48 at 64, where reading the operands from shared memory at 128 bytes a cycle
// bounds it); from inside a branch of one lane it cost 100 and more. Waiting
// on a barrier and committing to one cost about 100 cycles each, so the
// pieces go in bunches, and one warp for both would leave the pipe idle.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(~0u, mbar_wait(bar, parity));
}

// Given up: lets the products in flight end before the block does.
template <class S>
__device__ void drain_products(Misc<S> &m, uint32_t bar) {
    m.abort = 1;
    if (elect_one()) tcgen05_commit(bar);
    __syncwarp();
    for (int i = 0; i < 4096 && !mbar_try_wait(bar, 0); ++i) {}
}

template <class S, typename Source>
__device__ void score_role(const MlaArgs &a, uint32_t smem, Misc<S> &m, Source source) {
    const Bars<S> bars{smem_addr(&m)};
    const uint32_t tmem = __shfl_sync(~0u, m.tmem, 0) + S::kScores;
    Ring<S::kSlots> slots;
    Ring<S::kFull> bunch;
    Ring<2> pieces;
    uint32_t pass = 0;
    Segment g;
    while (source.next(a, g)) {
        if (!warp_wait(bars.query_ready(), pass)) return drain_products<S>(m, bars.drain(0));
        pass ^= 1;
        for (int u = g.begin; u < g.end; ++u) {
#pragma unroll
            for (int b = 0; b < 5; b += S::kPer) {
                if (!warp_wait(bars.bunch_full(bunch.at), bunch.pass) ||
                    !warp_wait(bars.piece_empty(pieces.at), pieces.pass ^ 1))
                    return drain_products<S>(m, bars.drain(0));
                tcgen05_after_sync();
                Ring<S::kSlots> read = slots;
                const uint32_t d = tmem + pieces.at * S::kPer * S::kRows;
                const bool leader = elect_one();
#pragma unroll
                for (int i = b; i < b + S::kPer && i < 5; ++i) {
                    if (leader) score_piece<S>(smem, slots.at, i, d + (i - b) * S::kRows);
                    slots.step();
                }
                if (leader) {
                    tcgen05_commit(bars.piece_full(pieces.at));
                    // the values need the latent tiles once more
#pragma unroll
                    for (int i = b; i < b + S::kPer && i < 5; ++i) {
                        if (i == 0 || !S::kHasValues)
                            tcgen05_commit(bars.slot_empty(read.at));
                        read.step();
                    }
                }
                __syncwarp();
                bunch.step();
                pieces.step();
            }
        }
    }
}

template <class S>
__device__ __forceinline__ uint8_t *block_setup(uint8_t *raw, Misc<S> *&m) {
    uint8_t *smem = raw;
    m = reinterpret_cast<Misc<S> *>(smem + S::kMiscOff);
    if (threadIdx.x == 0) {
        m->abort = 0;
        for (int i = 0; i < S::kFull; ++i) {
            const int at = i % S::kBunches * S::kPer;      // a bunch: its slots' arrivals
            mbar_init(smem_addr(&m->bunch_full[i]), 5 - at < S::kPer ? 5 - at : S::kPer);
        }
        for (int i = 0; i < S::kSlots; ++i) mbar_init(smem_addr(&m->slot_empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&m->piece_full[i]), 1);
            mbar_init(smem_addr(&m->piece_empty[i]), S::kWarps);
            mbar_init(smem_addr(&m->drain[i]), 1);
            mbar_init(smem_addr(&m->prob_full[i]), S::kWarps);
            mbar_init(smem_addr(&m->prob_empty[i]), 1);
            mbar_init(smem_addr(&m->scale_full[i]), 1);
            mbar_init(smem_addr(&m->scale_empty[i]), S::kWarps);
        }
        mbar_init(smem_addr(&m->keys_full), 1);
        mbar_init(smem_addr(&m->query_ready), S::kWarps);
        mbar_init_fence();
    }
    if (threadIdx.x >> 5 == S::kScoreWarp) tmem_alloc<S::kColumns>(smem_addr(&m->tmem));
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    return smem;
}

template <class S>
__device__ __forceinline__ void block_end(const MlaArgs &a, Misc<S> &m) {
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (threadIdx.x >> 5 == S::kScoreWarp) tmem_free<S::kColumns>(m.tmem);
    if (threadIdx.x == 0 && m.abort != 0 && a.invalid_count != nullptr)
        atomicAdd(a.invalid_count, 1ull);
}

}  // namespace kvpub
