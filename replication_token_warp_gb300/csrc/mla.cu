// Absorbed latent attention over the paged fp8 Main cache.  The C ABI is
// declared in kvpub.h.
//
// A block works on S::kRows query rows (token, head) of a sequence and walks
// its keys 128 at a time (a unit).  Keys are the M side of both products, so
// that 16 rows fill the tensor cores as well as 64 do:
//
//   S^T[key, row]  = K Q^T        A = the cache's codes, K-major
//   O^T[dim, row] += V^T P^T      A = the same bytes, MN-major
//
// and the cache's E4M3 codes go from TMA to the tensor cores as they are;
// nothing is decoded.  What makes that exact enough is to hold the other
// operand as the sum of two 8-bit floats, E4M3 for the value and E5M2 for
// what is left: a bf16 query splits exactly (8 significant bits, 4 + 4), a
// probability keeps 8 bits, as bf16 would.  Two products at the fp8 rate cost
// what one costs in bf16, without the decoded copy of the keys in shared
// memory.
//
// A row of the cache has a scale for each 128 of its 512 values.  A key is a
// lane of the accumulators, so its scale multiplies one thread's numbers:
// the four tiles' partial scores and the rope's are separate accumulators
// ("pieces") that the softmax threads sum as scale[t] * piece[t] in fp32.
// For the values the scale goes into the probability, one P^T for each tile:
// P_t = 2^(s - m) * scale[t], relative to the running maximum m of s + log2
// of the key's largest scale, and to the tile's own largest such ratio so
// far.  Scores, maxima, sums and accumulators are fp32.
//
// Roles: 8 or 16 softmax warps (two or four threads a key, each with its part
// of the rows), one warp that loads, one that issues the scores' products, one
// the values', and one that prepares the keys' scales.  The keys' tiles live in
// a ring of 16 KB slots, five a unit of 128 keys: rope, then the four latent
// tiles.  The next unit's scores are formed and read while this unit's
// probabilities go to the tensor cores.
//
// Work is cut into as many equal runs as there are blocks, of units and, for
// what a segment costs by itself, a few steps more; a run may begin and end
// inside a sequence.  Partial results go to the workspace and a second launch
// joins them.  Small calls give each sequence's tile of rows to a cluster, whose
// blocks join their parts through each other's shared memory.
//
// What bounds it.  With 16 rows the keys' loads: a unit takes some 4,200
// cycles, where 80 KB of cache take 3,650 at the memory's rate (64 ragged
// sequences of up to 40k tokens, 16 heads: 52 us, half of the memory's rate
// with what starts, ends and joins).  With 64 rows the softmax warps between
// the products: a unit takes some 7,700 cycles, its products 3,300 (reading
// their operands from shared memory), its instructions 3,200 issue slots of
// each scheduler (48 sequences of 8k tokens, 64 heads: 109 us, 2.4 TB/s; 64
// drafts of 64 heads over 4 x 16k tokens: 670 us, 0.69 PFLOP/s).

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "blackwell.cuh"
#include "host.cuh"
#include "kvpub.h"
#include "mla.cuh"
#include "mla_host.cuh"
#include "mla_units.cuh"

namespace kvpub {
namespace {

namespace cg = cooperative_groups;

// Probabilities are held times 2^kShift.  They may outgrow the reference
// maximum by 2^kGrowth before it is moved (and the accumulators rescaled):
// 2^(kShift + kGrowth) stays below E4M3's 448.  Of the two 8-bit parts' sum 8 bits
// are right down to 2^-12 of the row's largest probability; smaller ones are off by
// up to 2^-20 of that, and by up to four times as much as powers of two stand for
// the key's largest scale and for the tile's largest ratio.  (A move
// costs a third of a unit; with 7 and 1.75 the attention took 2 % longer.)
constexpr float kShift = 6.0f;
constexpr float kGrowth = 2.75f;

struct Partial {      // in the workspace, one a block: the item that begins in
    int last;         // this block and ends in block `last`
    int rows, row0;   // its sequence's rows, and its first one
    int first;        // the sequence's first query token
};

struct Workspace {
    Partial *partial;     // [kMaxCtas]
    float *lse;           // [2 * kMaxCtas, rows], base 2
    float *out;           // [2 * kMaxCtas, rows / 4, 512, 4]
};

// A tile's largest ratio so far as a byte, the exponent of the power of two
// above it (0: none).  A finer step would follow the largest
// ratio more closely, and would have to be moved far more often.
__device__ __forceinline__ uint32_t ratio_byte(float ratio) {
    const uint32_t e = (__float_as_uint(ratio) >> 23) & 255u;
    return e == 0 ? 0 : e + 1;
}

__device__ __forceinline__ float byte_ratio(uint32_t bytes, int i) {
    return __uint_as_float(((bytes >> (8 * i)) & 255u) << 23);
}

template <class S>
struct Segments {
    Cursor c;
    __device__ __forceinline__ bool next(const MlaArgs &a, Segment &g) {
        while (c.left > 0 && c.seq < a.num_seqs) {
            g.s = sequence(a, c.seq);
            if (c.tile >= tiles_of<S>(a, g.s)) {
                ++c.seq;
                c.tile = 0;
                continue;
            }
            g.units = units_of(g.s);
            g.seq = c.seq;
            g.tile = c.tile;
            const int64_t n = static_cast<int64_t>(g.units) + c.over - c.step;
            const int64_t end = c.step + (n < c.left ? n : c.left);
            g.begin = max(c.step - c.over, 0);
            g.end = static_cast<int>(max(end - c.over, static_cast<int64_t>(0)));
            g.counts = c.tile == 0;
            c.left -= end - c.step;
            c.step = 0;
            ++c.tile;
            if (g.end == g.begin) continue;     // none of its units
            return true;
        }
        return false;
    }
};

// The key warp: once a unit, what the softmax threads need of each key beside
// its scales, as 16 bytes:
//   x, y  the four tiles' ratios of scale to the power of two below the key's
//         largest, relative to the power of two above the largest such ratio
//         so far (m.ratios), in fp16: below 1
//   z     log2 of that power of two, fp32
//   w     bits 0-7 its exponent; bit 8: the key exists; bits 9-12: the tile's
//         scale is not finite (its ratio is 0 and its values are to be cleared)
template <class S, typename Source>
__device__ void key_role(const MlaArgs &a, Misc<S> &m, Source source) {
    const int lane = threadIdx.x & 31;
    const Bars<S> bars{smem_addr(&m)};
    Waiter<S> wait{m, true};
    Ring<2> ring;
    Segment g;
    while (source.next(a, g)) {
        uint32_t most = 0;
        for (int u = g.begin; u < g.end; ++u) {
            wait(bars.scale_full(ring.at), ring.pass);
            // a key's four ratios, in a few registers: all are formed twice
            auto key = [&](int k, float (&ratio)[4], uint32_t &ge, uint32_t &wild) {
                const float4 s = *reinterpret_cast<const float4 *>(m.scales[ring.at][k]);
                const float scale[4] = {s.x, s.y, s.z, s.w};
                const bool on = ((m.valid[ring.at] >> (k >> 6)) & 1) && u * kUnit + k < g.s.len;
                uint32_t biggest = 0;
                wild = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t bits = __float_as_uint(scale[i]) & 0x7fffffffu;
                    if (bits >= 0x7f800000u) wild |= 1u << i;
                    else biggest = max(biggest, bits);
                }
                ge = on ? min(max(biggest >> 23, 1u), 250u) : 127u;
                const float ginv = __uint_as_float((254u - ge) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ratio[i] = !on || ((wild >> i) & 1) ? 0.f : scale[i] * ginv;
                return on;
            };
            float ratio[4];
            uint32_t ge, wild, te = 0;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                key(32 * j + lane, ratio, ge, wild);
#pragma unroll
                for (int i = 0; i < 4; ++i) te = __vmaxu4(te, ratio_byte(ratio[i]) << (8 * i));
            }
            for (int d = 1; d < 32; d <<= 1) te = __vmaxu4(te, __shfl_xor_sync(~0u, te, d));
            most = __vmaxu4(most, te);
            // the softmax threads have read the last unit's
            wait(bars.scale_empty(ring.at ^ 1), ring.at == 0 ? ring.pass ^ 1 : ring.pass);
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const bool on = key(32 * j + lane, ratio, ge, wild);
                float rt[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = (most >> (8 * i)) & 255u;
                    rt[i] = b == 0 ? 0.f : ratio[i] * __uint_as_float((254u - b) << 23);
                }
                m.keys[32 * j + lane] =
                    make_uint4(half2_from(rt[0], rt[1]), half2_from(rt[2], rt[3]),
                               __float_as_uint(static_cast<float>(static_cast<int>(ge) - 127)),
                               ge | (on ? 256u : 0u) | (wild << 9));
            }
            if (lane == 0) m.ratios = most;
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.keys_full());
            ring.step();
        }
    }
}

// ---------------------------------------------------------------- attention

// The warp's sums of each of kC columns: column (lane % kC)'s. The halves of
// the columns are exchanged between halves of the lanes, so that each step
// moves half of what the last one did.
template <int kC>
__device__ __forceinline__ float column_sums(const float2 (&l)[kC / 2], int lane) {
    float v[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) v[c] = c & 1 ? l[c / 2].y : l[c / 2].x;
#pragma unroll
    for (int n = kC / 2; n >= 1; n /= 2) {
        const bool up = lane & n;
#pragma unroll
        for (int c = 0; c < n; ++c) {
            const float keep = up ? v[n + c] : v[c], give = up ? v[c] : v[n + c];
            v[c] = keep + __shfl_xor_sync(~0u, give, n);
        }
    }
#pragma unroll
    for (int d = kC; d < 32; d *= 2) v[0] += __shfl_xor_sync(~0u, v[0], d);
    return v[0];
}

template <class S, bool kCluster>
__device__ void softmax_role(const MlaArgs &a, const Workspace &ws, uint8_t *smem,
                             Misc<S> &m, Segments<S> source, int blocks) {
    constexpr int kC = S::kCols;
    constexpr int kAll = S::kParts + 1;         // barrier of all softmax warps; parts have 1..
    const Lane t = softmax_lane(m.tmem);
    const int row0 = t.part * kC;
    // the key's row of P, at the thread's first 16-byte chunk (swizzled)
    const uint32_t prob_row = smem_addr(smem) + S::kProbOff + t.key * 128 +
                              ((((row0 >> 4) ^ (t.key & 7)) << 4) | (row0 & 15));
    const Bars<S> bars{smem_addr(&m)};
    Waiter<S> wait{m, true};
    // Units before the one whose probabilities are formed; all places in rings
    // follow from it (registers are short).
    uint32_t n = 0;
    auto probs_at = [](uint32_t unit, int grp) { return ring_at<S::kProbs>(unit * S::kGroups + grp); };
    if (threadIdx.x == 0) m.cursor = source.c;
    bool some = false;   // a segment's units are done
    int buffer = 0;      // of m.segments and m.out_at: the last one's
    float2 l[kC / 2];
    float ref = -INFINITY;          // lane c < kC: row c's reference
    uint32_t texp = 0;              // the tiles' largest ratios, a byte each
    for (;;) {
        named_barrier(kAll, S::kWarps * 32);     // the last queries and maxima are done with
        const Segment &g = m.segments[buffer];
        const bool whole = g.begin == 0 && g.end == g.units;
        const int part = 2 * blockIdx.x + (g.begin == 0 ? 1 : 0);
        const int64_t *out_at = m.out_at[buffer];
        if (some) {
            // the rows' sums over all keys
            float total = column_sums<kC>(l, t.lane);
            if (t.lane < kC) m.wmax[t.warp & 3][row0 + t.lane] = total;
            named_barrier(1 + t.part, 128);
            if (t.lane < kC) {
                const int r = row0 + t.lane;
                total = ((m.wmax[0][r] + m.wmax[1][r]) + m.wmax[2][r]) + m.wmax[3][r];
                if (m.abort != 0) total = NAN;      // see Waiter
                const float lse2 = total == 0.f ? -INFINITY
                                                : (ref == -INFINITY ? 0.f : ref) - kShift +
                                                      log2f(total);
                m.fac[r] = total == 0.f ? 0.f : 1.f / total;
                if ((t.warp & 3) == 0) {
                    if (!whole) {
                        if (kCluster) m.part_lse[r] = lse2;
                        else ws.lse[part * S::kRows + r] = lse2;
                    } else if (a.lse != nullptr && out_at[r] >= 0) {
                        const int64_t row = g.tile * S::kRows + r;
                        a.lse[static_cast<int64_t>(g.s.first) * a.num_heads + row] = lse2 * kLn2;
                    }
                }
            }
        }
        // The next segment's queries, so that its first scores are formed
        // while the last one's results are written.
        Segments<S> rest{m.cursor};
        Segment next;
        const bool have = rest.next(a, next);
        if (have) load_queries<S>(a, next, smem, m, m.out_at[buffer ^ 1]);
        fence_async_smem();
        named_barrier(kAll, S::kWarps * 32);
        if (have) {
            if (threadIdx.x == 0) {
                m.cursor = rest.c;
                m.segments[buffer ^ 1] = next;
            }
            if (t.lane == 0) mbar_arrive(bars.query_ready());
        }
        // The join's launch overlaps with the last results: 64 ragged sequences
        // of 16 heads 52.5 -> 51.8 us, at 64 rows no difference.
        if (!have && !kCluster) launch_next_kernel();
        if (some) {
            __syncwarp();
            const Ring<S::kProbs> last = probs_at(n - 1, S::kGroups - 1);
            wait(bars.prob_empty(last.at), last.pass);
            tcgen05_after_sync();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                float o[kC];
                tmem_load<kC>(t.tmem + i * S::kRows + row0, o);
                tmem_load_wait();
                const float up = wait.alive ? byte_ratio(texp, i) : NAN;
                const int dim = i * 128 + t.key;
#pragma unroll
                for (int c = 0; c < kC; ++c) o[c] *= m.fac[row0 + c] * up;
                if (!whole && kCluster) {
                    // for the cluster's blocks, where the keys were
                    float *to = reinterpret_cast<float *>(smem) + row0 * KVPUB_LATENT_DIM + dim;
#pragma unroll
                    for (int c = 0; c < kC; ++c) to[c * KVPUB_LATENT_DIM] = o[c];
                } else if (!whole) {
                    // four rows of a value side by side, then the values: whole
                    // lines a store
                    float4 *to = reinterpret_cast<float4 *>(ws.out) +
                                 (static_cast<int64_t>(part) * S::kRows + row0) / 4 *
                                     KVPUB_LATENT_DIM + dim;
#pragma unroll
                    for (int c = 0; c < kC; c += 4)
                        to[c / 4 * KVPUB_LATENT_DIM] =
                            make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                } else {
                    // two lanes exchange halves: each gets two dims of every other row
                    const bool odd = t.lane & 1;
#pragma unroll
                    for (int c = 0; c < kC; c += 2) {
                        const float other = __shfl_xor_sync(~0u, odd ? o[c] : o[c + 1], 1);
                        const int64_t to = out_at[row0 + c + odd];
                        uint32_t b;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                            : "=r"(b) : "f"(odd ? o[c + 1] : other), "f"(odd ? other : o[c]));
                        if (to >= 0) *reinterpret_cast<uint32_t *>(a.out + to + (dim & ~1)) = b;
                    }
                }
            }
            tcgen05_before_sync();
        }
        if (!have) break;
        some = true;
        buffer ^= 1;
        // The unit up to which some row may have no reference: it has seen no key
        // (skipped blocks, or scores of -inf), its sums and accumulators are 0,
        // and the first unit that shows it one gives it its reference.  Until
        // then -inf stands as 0.
        int fresh = next.begin;
        const int end = next.end;

        const int prefix = next.s.len - next.s.count;
#pragma unroll
        for (int c = 0; c < kC / 2; ++c) l[c] = make_float2(0.f, 0.f);
        ref = -INFINITY;
        if (t.lane < kC) m.nref[row0 + t.lane] = kShift;
        __syncwarp();
        texp = 0;
        int par = 0;                    // which of m.grown is in use
        // The next unit's scores are read while this unit's probabilities wait
        // for the tensor cores.
        float2 z[kC / 2];
        auto add = [&](uint32_t unit, int bunch) {
            if (bunch == 0) {
#pragma unroll
                for (int c = 0; c < kC / 2; ++c) z[c] = make_float2(0.f, 0.f);
            }
            add_bunch<S>(t, bars, wait, ring_at<2>(unit * S::kBunches + bunch), bunch,
                         m.scales[unit & 1][t.key], z);
        };
        wait(bars.keys_full(), n & 1);
#pragma unroll 1
        for (int i = 0; i < S::kBunches; ++i) add(n, i);

        for (int u = fresh; u < end; ++u) {
            const bool unset = u == fresh;
            const uint4 info = m.keys[t.key];
            const uint32_t tnew = m.ratios;
            __syncwarp();
            if (t.lane == 0) mbar_arrive(bars.scale_empty(n & 1));
            const bool on = info.w & 256u;
            const float gexp = __uint_as_float(info.z);
            // z = s + log2 of the key's power of two, relative to the references
            const float2 gexp2 = make_float2(gexp, gexp);
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < kC / 4; ++c) {
                const float4 f = *reinterpret_cast<const float4 *>(&m.factor[row0 + 4 * c]);
                const float4 r = *reinterpret_cast<const float4 *>(&m.nref[row0 + 4 * c]);
                z[2 * c] = fma2(z[2 * c], make_float2(f.x, f.y), add2(gexp2, make_float2(r.x, r.y)));
                z[2 * c + 1] =
                    fma2(z[2 * c + 1], make_float2(f.z, f.w), add2(gexp2, make_float2(r.z, r.w)));
            }
            if (!on) {
#pragma unroll
                for (int c = 0; c < kC / 2; ++c) z[c] = make_float2(-INFINITY, -INFINITY);
            } else if (u * kUnit + t.key >= prefix) {
                const int j = u * kUnit + t.key - prefix;
#pragma unroll
                for (int c = 0; c < kC / 2; ++c) {
                    if (!((m.mask[row0 + 2 * c] >> j) & 1)) z[c].x = -INFINITY;
                    if (!((m.mask[row0 + 2 * c + 1] >> j) & 1)) z[c].y = -INFINITY;
                }
            }
#pragma unroll
            for (int c = 0; c < kC / 2; ++c) top = fmaxf(top, fmaxf(z[c].x, z[c].y));
            // Where nothing outgrows its reference one barrier settles that.
            constexpr float kMost = kShift + kGrowth;
            // What did is gathered row by row: few do.
            if (!unset && top > kMost) {
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float w = c & 1 ? z[c / 2].y : z[c / 2].x;
                    if (w > kMost) atomicMax(&m.grown[par][row0 + c], __float_as_int(w));
                }
            }
            const bool moves = any_of_part(
                1 + t.part, top > (unset ? -INFINITY : kMost) || tnew != texp);
            uint32_t rows = 0;      // that moved, a bit each
            if (moves) {
                const int r = row0 + (t.lane & (kC - 1));
                float mine = -INFINITY;     // row r's new maximum, where it has one
                if (unset) {
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        const float w = warp_max(c & 1 ? z[c / 2].y : z[c / 2].x);
                        if (t.lane == c) mine = w;
                    }
                    if (t.lane < kC) m.wmax[t.warp & 3][r] = mine;
                    m.grown[0][r] = m.grown[1][r] = m.grown[2][r] = 0;
                    named_barrier(1 + t.part, 128);
                    mine = fmaxf(fmaxf(m.wmax[0][r], m.wmax[1][r]),
                                 fmaxf(m.wmax[2][r], m.wmax[3][r]));
                } else {
                    const int w = m.grown[par][r];
                    if (w != 0) mine = __int_as_float(w);
                    // The one used before this is cleared: all have read it
                    // before the barrier, and none uses it before the next.
                    m.grown[par == 0 ? 2 : par - 1][r] = 0;
                    par = par == 2 ? 0 : par + 1;
                }
                // back from relative to the reference (-inf stands as 0)
                const float was = ref == -INFINITY ? 0.f : ref;
                const float now = mine + (was - kShift);
                const float old = ref;
                if (now > ref) ref = now;
                if (unset) {
                    if (now != now) ref = 0.f;     // scores of NaN alone: no maximum
                    if (__any_sync(~0u, ref == -INFINITY)) fresh = u + 1;
                }
                rows = __ballot_sync(~0u, t.lane < kC && old != ref);
                const float moved = ref == -INFINITY ? 0.f : ref;
                m.nref[r] = kShift - moved;
                m.fac[r] = old == ref ? 1.f : exp2_approx(old - ref);
                // z moves by the change of what it is relative to (through
                // shared memory, which is cheaper than a shuffle a row)
                m.shift[r] = was - moved;
                __syncwarp();
#pragma unroll
                for (int c = 0; c < kC / 4; ++c) {
                    const float4 d = *reinterpret_cast<const float4 *>(&m.shift[row0 + 4 * c]);
                    const float4 f = *reinterpret_cast<const float4 *>(&m.fac[row0 + 4 * c]);
                    z[2 * c] = add2(z[2 * c], make_float2(d.x, d.y));
                    z[2 * c + 1] = add2(z[2 * c + 1], make_float2(d.z, d.w));
                    l[2 * c] = mul2(l[2 * c], make_float2(f.x, f.y));
                    l[2 * c + 1] = mul2(l[2 * c + 1], make_float2(f.z, f.w));
                }
            } else if (unset) {
                fresh = u + 1;
            }

            // probabilities, their sum in fp32, and in fp16 for the products
            // (11 bits, where the two 8-bit parts keep 8)
            const float ginv = __uint_as_float((254u - (info.w & 255u)) << 23);
            const float2 ginv2 = make_float2(ginv, ginv);
            uint32_t p[kC / 2];
#pragma unroll
            for (int c = 0; c < kC / 2; ++c) {
                const float2 x = make_float2(exp2_approx(z[c].x), exp2_approx(z[c].y));
                l[c] = fma2(x, ginv2, l[c]);
                p[c] = half2_from(x.x, x.y);
            }
            if (moves && texp != 0) {
                // The accumulators follow the references, once the last
                // unit's values are in (without ratios so far there are none).
                const Ring<S::kProbs> last = probs_at(n - 1, S::kGroups - 1);
                wait(bars.prob_empty(last.at), last.pass);
                tcgen05_after_sync();
                // Mostly a row or two: their columns of the four tiles at once
                // take 0.2 us a row, all of the thread's 0.8 (when this was added, a
                // tree of 64 drafts over 4 x 16k tokens went from 704 to 676 us).
                if (tnew == texp && __popc(rows) <= 4) {
                    for (; rows != 0; rows &= rows - 1) {
                        const int c = __ffs(rows) - 1;
                        const uint32_t at = t.tmem + row0 + c;
                        float o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) tmem_load<1>(at + i * S::kRows, o + i);
                        const float f = m.fac[row0 + c];
                        tmem_load_wait();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[i] *= f;
                            tmem_store<1>(at + i * S::kRows, o + i);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = t.tmem + i * S::kRows + row0;
                        float o[kC];
                        tmem_load<kC>(at, o);
                        const float most = byte_ratio(tnew, i);     // powers of two: exact
                        const float ft = most == 0.f ? 0.f : __fdividef(byte_ratio(texp, i), most);
                        tmem_load_wait();
#pragma unroll
                        for (int c = 0; c < kC / 2; ++c) {
                            const float2 f = *reinterpret_cast<const float2 *>(&m.fac[row0 + 2 * c]);
                            const float2 x = mul2(make_float2(o[2 * c], o[2 * c + 1]),
                                                  mul2(f, make_float2(ft, ft)));
                            o[2 * c] = x.x;
                            o[2 * c + 1] = x.y;
                        }
                        tmem_store<kC>(at, o);
                    }
                }
                tmem_store_wait();
                tcgen05_before_sync();
            }
            texp = tnew;
            // one P^T for each tile, in two 8-bit parts
            const bool more = u + 1 < end;
            if (more) wait(bars.keys_full(), (n + 1) & 1);
            uint32_t clear = on ? info.w >> 9 : 15u;      // tiles whose values go
            unsigned long long ratios = info.x | static_cast<unsigned long long>(info.y) << 32;
#pragma unroll 1
            for (int grp = 0; grp < S::kGroups; ++grp) {
                uint32_t hi[S::kTiles][kC / 4], lo[S::kTiles][kC / 4];
#pragma unroll
                for (int i = 0; i < S::kTiles; ++i) {
                    const uint32_t r2 = __byte_perm(static_cast<uint32_t>(ratios), 0, 0x1010);
                    ratios >>= 16;
#pragma unroll
                    for (int c = 0; c < kC / 4; ++c)
                        split_f8(half2_mul(p[2 * c], r2), half2_mul(p[2 * c + 1], r2), hi[i][c],
                                 lo[i][c]);
                }
                const Ring<S::kProbs> probs = probs_at(n, grp);
                wait(bars.prob_empty(probs.at), probs.pass ^ 1);
                const uint32_t row = prob_row + probs.at * kSlotBytes;
#pragma unroll
                for (int i = 0; i < S::kTiles; ++i) {
                    // 16-byte chunk 2 i kRows / 16 (+ kRows / 16) after the
                    // thread's first, in swizzled order
                    const uint32_t to_hi = row ^ (2 * i * S::kRows), to_lo = to_hi ^ S::kRows;
                    if constexpr (kC == 8) {
                        st_shared(to_hi, make_uint2(hi[i][0], hi[i][1]));
                        st_shared(to_lo, make_uint2(lo[i][0], lo[i][1]));
                    } else {
                        st_shared(to_hi, make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]));
                        st_shared(to_lo, make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]));
                    }
                }
                // Rows that hold no key, and tiles whose scale is not finite,
                // may hold NaN codes, which 0 * NaN would spread: their values
                // are cleared (the scores are read already; a row that sees
                // such a key is NaN by its probability).
                if (clear != 0) {
                    for (int i = 0; i < S::kTiles; ++i) {
                        const int tile = grp * S::kTiles + i;
                        if (!((clear >> tile) & 1)) continue;
                        const int s = (n * 5 + 1 + tile) % S::kSlots;
                        uint4 *v = reinterpret_cast<uint4 *>(smem + s * kSlotBytes + t.key * 128 +
                                                             t.part * (128 / S::kParts));
#pragma unroll
                        for (int c = 0; c < 8 / S::kParts; ++c) v[c] = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (t.lane == 0) mbar_arrive(bars.prob_full(probs.at));
                // The last bunch's tile may wait for a slot that this unit's
                // values free: not before all of them are handed over.
                if (more && (grp < S::kBunches - 1 || grp == S::kGroups - 1)) {
#pragma unroll 1
                    for (int i = min(grp, S::kBunches - 1);
                         i < (grp == S::kGroups - 1 ? S::kBunches : grp + 1); ++i)
                        add(n + 1, i);
                }
            }
            ++n;
        }
    }
    if (!kCluster && threadIdx.x == 0) {
        // the item that begins in this block's last segment and ends later
        Partial p{-1, 0, 0, 0};
        const Segment &g = m.segments[buffer];
        if (some && g.begin == 0 && g.end < g.units) {
            const int64_t at = portion(m.total, blockIdx.x + 1, blocks);     // steps before the next block
            const int64_t end = at + (g.units - g.end);                 // .. before the item's end
            p.rows = g.s.count * a.num_heads;
            p.row0 = g.tile * S::kRows;
            p.first = g.s.first;
            p.last = block_of(end - 1, m.total, blocks);
        }
        ws.partial[blockIdx.x] = p;
    }
}

template <class S>
__device__ void value_role(const MlaArgs &a, uint32_t smem, Misc<S> &m, Segments<S> source) {
    const Bars<S> bars{smem_addr(&m)};
    const uint32_t tmem = __shfl_sync(~0u, m.tmem, 0);
    Ring<S::kSlots> slots;
    Ring<S::kProbs> probs;
    constexpr uint32_t hi = mma_desc(kE4m3, kE4m3, S::kRows, true);
    constexpr uint32_t lo = mma_desc(kE4m3, kE5m2, S::kRows, true);
    Segment g;
    while (source.next(a, g)) {
        for (int u = g.begin; u < g.end; ++u) {
            slots.step();
            const uint32_t first = u != g.begin;
#pragma unroll
            for (int grp = 0; grp < S::kGroups; ++grp) {
                if (!warp_wait(bars.prob_full(probs.at), probs.pass))
                    return drain_products<S>(m, bars.drain(1));
                tcgen05_after_sync();
                const bool leader = elect_one();
#pragma unroll
                for (int i = 0; i < S::kTiles; ++i) {
                    const uint64_t v = operand_desc(smem + slots.at * kSlotBytes);
                    const uint64_t p = operand_desc(smem + S::kProbOff + probs.at * kSlotBytes +
                                                    2 * i * S::kRows);
                    const uint32_t d = tmem + (grp * S::kTiles + i) * S::kRows;
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(d, v + 256 * k, p + 256 * k, hi, k == 0 ? first : 1u);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(d, v + 256 * k, p + (S::kRows >> 4) + 256 * k, lo, 1u);
                        tcgen05_commit(bars.slot_empty(slots.at));
                    }
                    slots.step();
                }
                if (leader) tcgen05_commit(bars.prob_empty(probs.at));
                __syncwarp();
                probs.step();
            }
        }
    }
}

// The cluster's join: `parts` blocks have their normalised results in shared
// memory, [rows][512], and their rows' log-sum-exps in part_lse; each takes its
// share of the rows' values.
template <class S>
__device__ void join_cluster(const MlaArgs &a, uint8_t *smem, Misc<S> &m, int rank, int parts) {
    cg::cluster_group cluster = cg::this_cluster();
    const Segment &g = m.segments[1];
    const int rows = min(g.s.count * a.num_heads - g.tile * S::kRows, S::kRows);
    constexpr int kThreads = S::kWarps * 32;
    for (int i = rank * kThreads + threadIdx.x; i < rows * (KVPUB_LATENT_DIM / 4);
         i += parts * kThreads) {
        const int r = i / (KVPUB_LATENT_DIM / 4), d = i % (KVPUB_LATENT_DIM / 4);
        float top = -INFINITY;
        for (int p = 0; p < parts; ++p)
            top = fmaxf(top, cluster.map_shared_rank(&m, p)->part_lse[r]);
        if (top == -INFINITY) top = 0.f;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < parts; ++p) {
            const float w = exp2f(cluster.map_shared_rank(&m, p)->part_lse[r] - top);
            const float4 y = reinterpret_cast<const float4 *>(cluster.map_shared_rank(smem, p))[i];
            sum += w;
            o.x = fmaf(w, y.x, o.x);
            o.y = fmaf(w, y.y, o.y);
            o.z = fmaf(w, y.z, o.z);
            o.w = fmaf(w, y.w, o.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint2 b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b.x) : "f"(o.y * inv), "f"(o.x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b.y) : "f"(o.w * inv), "f"(o.z * inv));
        *reinterpret_cast<uint2 *>(a.out + m.out_at[1][r] + 4 * d) = b;
        if (d == 0 && a.lse != nullptr)
            a.lse[static_cast<int64_t>(g.s.first) * a.num_heads + g.tile * S::kRows + r] =
                sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// kCluster: a cluster takes one item, its blocks equal runs of the units, and
// joins them itself; else the work is cut as find_work says.
template <int kRows, bool kCluster>
__global__ void __launch_bounds__(Shape<kRows, true>::kThreads, 1)
mla_attention_kernel(const MlaArgs a, const Workspace ws, const __grid_constant__ CUtensorMap tiles,
                     const __grid_constant__ CUtensorMap scales) {
    using S = Shape<kRows, true>;
    extern __shared__ __align__(1024) uint8_t raw[];
    Misc<S> *m;
    if (threadIdx.x == S::kLoadWarp * 32) {
        prefetch_tensormap(&tiles);
        prefetch_tensormap(&scales);
    }
    uint8_t *smem = block_setup<S>(raw, m);
    wait_previous_kernel();
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
    auto work = [&](const Segments<S> &source, int blocks) {
        if (warp < S::kWarps) {
            if constexpr (S::kMoveRegisters)
                asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
            softmax_role<S, kCluster>(a, ws, smem, *m, source, blocks);
        } else {
            if constexpr (S::kMoveRegisters)
                asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
            if (warp == S::kLoadWarp)
                load_role<S>(a, &tiles, &scales, smem, *m, source);
            else if (warp == S::kScoreWarp)
                score_role<S>(a, smem_addr(smem), *m, source);
            else if (warp == S::kValueWarp)
                value_role<S>(a, smem_addr(smem), *m, source);
            else if (warp == S::kKeyWarp)
                key_role<S>(a, *m, source);
        }
        __syncwarp();
    };
    if constexpr (kCluster) {
        cg::cluster_group cluster = cg::this_cluster();
        const int blocks = static_cast<int>(cluster.num_blocks());
        const int rank = static_cast<int>(cluster.block_rank());
        const int tiles_most = (a.max_query_len * a.num_heads + kRows - 1) / kRows;
        const int item = blockIdx.x / blocks, seq = item / tiles_most;
        const int tile = item - seq * tiles_most;
        const Sequence s = sequence(a, seq);
        const int units = units_of(s), parts = min(blocks, units);
        const bool takes = rank < parts && tile < tiles_of<S>(a, s);
        if (takes) {
            const int begin = static_cast<int>(portion(units, rank, parts));
            const int end = static_cast<int>(portion(units, rank + 1, parts));
            work(Segments<S>{{seq, tile, begin, 0, end - begin}}, 0);
        }
        cluster.sync();
        if (takes && parts > 1 && warp < S::kWarps) join_cluster<S>(a, smem, *m, rank, parts);
        cluster.sync();     // the parts are read
    } else {
        int blocks;
        const Share share = find_work<S>(a, *m, &blocks);
        if (static_cast<int>(blockIdx.x) >= blocks) {
            if (threadIdx.x == 0) ws.partial[blockIdx.x] = Partial{-1, 0, 0, 0};
        } else {
            const int steps = units_of(sequence(a, share.seq)) + share.over;
            const int tile = static_cast<int>(quotient(share.offset, steps));
            work(Segments<S>{{share.seq, tile,
                              static_cast<int>(share.offset - static_cast<int64_t>(tile) * steps),
                              share.over, share.left}},
                 blocks);
        }
    }
    block_end<S>(a, *m);
}

// Joins the parts of each item that more than one block worked on: blocks
// (x, ., .) take 128 values of eight rows each of the item that begins in
// attention block x, two lanes a pair of values: four rows each. The part that
// begins the item is 2 x + 1, the later blocks' are 2 y.
constexpr int kJoinRows = 8, kJoinDims = 128;

template <int kRows>
__global__ void __launch_bounds__(kJoinDims)
mla_join_kernel(const MlaArgs a, const Workspace ws) {
    // parts in flight: with 16 rows an item has more parts and the grid fewer
    // blocks (when measured: 64 ragged sequences, 16 heads 50.9 us with 8, 51.7 with 4;
    // 48 of 8k tokens, 64 heads 110.2 and 108.5)
    constexpr int kJoinParts = kRows == 16 ? 8 : 4;
    wait_previous_kernel();
    const int x = blockIdx.x, lane = threadIdx.x & 31;
    const Partial p = ws.partial[x];
    const int r0 = blockIdx.y * kJoinRows;
    if (p.last <= x || p.row0 + r0 >= p.rows) return;
    const int parts = p.last - x + 1;
    auto part = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * x + 1 : 2 * (x + i)); };
    const int dim = blockIdx.z * kJoinDims + (threadIdx.x >> 1 << 1), mine = (lane & 1) * 4;
    const float *from = ws.out + ((r0 + mine) / 4 * KVPUB_LATENT_DIM + dim) * 4;
    float4 y[kJoinParts][2];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i) {
            if (i0 + i >= parts) break;
            const float *at = from + part(i0 + i) * KVPUB_LATENT_DIM * kRows;
            y[i][0] = *reinterpret_cast<const float4 *>(at);
            y[i][1] = *reinterpret_cast<const float4 *>(at + 4);
        }
    };
    load(0);     // before the weights are known
    // lane 8 i + r: row r's parts i, i + 4, ..
    const int r = lane & 7;
    auto lse = [&](int i) { return i < parts ? ws.lse[part(i) * kRows + r0 + r] : -INFINITY; };
    const float lse0 = lse(lane >> 3);
    float top = lse0;
    for (int i = 4 + (lane >> 3); i < parts; i += 4) top = fmaxf(top, lse(i));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
    if (top == -INFINITY) top = 0.f;
    float sum = exp2f(lse0 - top);
    for (int i = 4 + (lane >> 3); i < parts; i += 4) sum += exp2f(lse(i) - top);
    sum += __shfl_xor_sync(~0u, sum, 8);
    sum += __shfl_xor_sync(~0u, sum, 16);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (threadIdx.x < kJoinRows && blockIdx.z == 0 && a.lse != nullptr && p.row0 + r0 + r < p.rows)
        a.lse[static_cast<int64_t>(p.first) * a.num_heads + p.row0 + r0 + r] =
            sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;

    float o[2][4] = {};
    for (int i0 = 0; i0 < parts; i0 += kJoinParts) {
        if (i0 != 0) load(i0);
        float weight[kJoinParts / 4];
#pragma unroll
        for (int j = 0; j < kJoinParts / 4; ++j)
            weight[j] = exp2f(lse(i0 + 4 * j + (lane >> 3)) - top) * inv;
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i) {
            if (i0 + i >= parts) break;
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __shfl_sync(~0u, weight[i / 4], 8 * (i % 4) + mine + k);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                o[k][0] = fmaf(w[0], y[i][k].x, o[k][0]);
                o[k][1] = fmaf(w[1], y[i][k].y, o[k][1]);
                o[k][2] = fmaf(w[2], y[i][k].z, o[k][2]);
                o[k][3] = fmaf(w[3], y[i][k].w, o[k][3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = p.row0 + r0 + mine + j;
        if (row >= p.rows) break;
        const int i = row / a.num_heads, head = row - i * a.num_heads;
        uint32_t b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(o[1][j]), "f"(o[0][j]));
        *reinterpret_cast<uint32_t *>(a.out + (p.first + static_cast<int64_t>(i)) * a.out_token +
                                      head * a.out_head + dim) = b;
    }
}

// ---------------------------------------------------------------- host side

// How a call is cut: rows of a tile, and blocks. A unit of keys costs some
// 4,200 cycles with 16 rows, 5,100 with 32 and 8,000 with 64, a segment by itself
// 9,000, 14,000 and 17,000, and the second launch that joins parts 8,000 to
// 11,000. Large calls take the most rows that their sequences fill and runs of
// equal length; smaller ones what gives the shortest run by the longest lengths
// that the block table allows, and if one cluster (or block) an item does that
// and all fit the GPU at once, without the second launch. Measured in a graph, us
// (* is what the rule takes, not always the best: it knows only the longest length):
//                                                runs with 16, 32, 64 rows   clusters
//   1 sequence, 16 heads, 509 tokens              10.5                       10.0* (4 blocks, 16 rows)
//   1 tree of 8 drafts, 16 heads, 777 tokens      13.4   15.7   19.6         13.8* (8 blocks, 16 rows)
//   2 sequences, 128 heads, 3,000 tokens          21.8*  22.0   23.9         20.8  (4 blocks, 16 rows)
//   4 trees of up to 3 drafts, 32 heads, 5,000    24.6   28.8*  37.4         41.0  (4 blocks, 32 rows)
//   50 sequences, 64 heads, 15 to 751 tokens      27.7   25.6*  23.2         35.6  (a block, 64 rows)
//   42 sequences, 128 heads, 2 to 78 tokens       26.8   23.0   19.2         16.0* (a block, 64 rows)
struct Split {
    int rows, blocks;
    int cluster;      // blocks an item, 0: cut by find_work and joined by a second launch
};

template <int kRows>
kvpub_status attention_clusters(int dev, int (*out)[3]) {
    using S = Shape<kRows, true>;
    return clusters_at_once<mla_attention_kernel<kRows, true>>(dev, S::kThreads, smem_bytes<S>(),
                                                               out);
}

Split split_work(const MlaCall &c, int sms, const int (&clusters)[3][3]) {
    const int most = rows_for(c.num_heads, c.max_query_len);
    const int64_t units = units_at_most(c.max_blocks);
    const int64_t unit_cost[3] = {42, 51, 80}, segment_cost[3] = {90,140,170};
    const int64_t join_cost[3] = {80,95,110}, cluster_cost[3] = {45, 50, 60};
    int64_t best = INT64_MAX;
    Split split{most, sms, 0};
    for (int i = 0; 16 << i <= most; ++i) {
        const int64_t tiles = (c.max_query_len * c.num_heads + (16 << i) - 1) >> (4 + i);
        const int64_t items = c.num_seqs * tiles;
        const int n = items * units < sms ? static_cast<int>(items * units) : sms;
        const int64_t cost = (items + n - 1) / n * segment_cost[i] +
                             (items * units + n - 1) / n * unit_cost[i] + join_cost[i];
        if (cost < best) {
            best = cost;
            split = Split{16 << i, n, 0};
        }
        for (int j = 0; j <= 3 && 1 << j < 2 * units; ++j) {
            const int k = 1 << j;
            if (items > (j == 0 ? sms : clusters[i][j - 1])) break;     // all at once
            const int64_t each = segment_cost[i] + (units + k - 1) / k * unit_cost[i] +
                                 (j == 0 ? 0 : cluster_cost[i]);
            if (each < best) {
                best = each;
                split = Split{16 << i, static_cast<int>(items * k), k};
            }
        }
    }
    return split;
}

size_t workspace_for(int rows, uint8_t *base, Workspace *ws) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    uint8_t *partial = take(sizeof(Partial) * kMaxCtas);
    uint8_t *lse = take(sizeof(float) * 2 * kMaxCtas * rows);
    uint8_t *out = take(sizeof(float) * 2 * kMaxCtas * rows * KVPUB_LATENT_DIM);
    if (ws != nullptr)
        *ws = Workspace{reinterpret_cast<Partial *>(partial), reinterpret_cast<float *>(lse),
                        reinterpret_cast<float *>(out)};
    return at;
}

template <int kRows>
kvpub_status launch_attention(const MlaArgs &a, const Workspace &ws, const CUtensorMap &tiles,
                              const CUtensorMap &scales, const Split &split, cudaStream_t stream) {
    using S = Shape<kRows, true>;
    static_assert(S::kSlots * kSlotBytes >= kRows * KVPUB_LATENT_DIM * 4, "a cluster's parts fit");
    static std::atomic<bool> opted[2][kMaxDevices];
    if (split.cluster != 0)
        return launch_opted("mla_attention", mla_attention_kernel<kRows, true>, opted[1],
                            split.cluster, split.blocks, S::kThreads, smem_bytes<S>(), stream, a,
                            ws, tiles, scales);
    kvpub_status st = launch_opted("mla_attention", mla_attention_kernel<kRows, false>, opted[0], 1,
                                   split.blocks, S::kThreads, smem_bytes<S>(), stream, a, ws,
                                   tiles, scales);
    if (st != KVPUB_OK) return st;
    const dim3 grid(split.blocks, kRows / kJoinRows, KVPUB_LATENT_DIM / kJoinDims);
    (void)launch_smem(mla_join_kernel<kRows>, grid, kJoinDims, 0, stream, 1, a, ws);
    return launched("mla_join");
}

kvpub_status attention(const MlaCall &c, void *out, int64_t out_token, int64_t out_head,
                       float *lse, void *workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    MlaArgs a;
    bool empty;
    kvpub_status st = check_call(c, false, &a, &empty);
    if (st != KVPUB_OK) return st;
    if (empty) return ok();
    if (out == nullptr) return fail(KVPUB_ERR_INVALID_ARG, "out is NULL");
    if (!aligned(out, 16)) return fail(KVPUB_ERR_ALIGNMENT, "out is not 16-byte aligned");
    if (out_token % 8 != 0 || out_head % 8 != 0)
        return fail(KVPUB_ERR_ALIGNMENT, "out strides %lld, %lld are not multiples of 8 elements",
                    (long long)out_token, (long long)out_head);
    const int64_t most = INT64_MAX / 8 / INT32_MAX;
    if (out_token < KVPUB_LATENT_DIM || out_head < KVPUB_LATENT_DIM || out_token > most ||
        out_head > most ||
        !(out_token >= (c.num_heads - 1) * out_head + KVPUB_LATENT_DIM ||
          out_head >= (c.num_tokens - 1) * out_token + KVPUB_LATENT_DIM))
        return fail(KVPUB_ERR_INVALID_ARG, "out strides %lld, %lld: rows overlap",
                    (long long)out_token, (long long)out_head);
    if (!aligned(lse, 4)) return fail(KVPUB_ERR_ALIGNMENT, "lse is misaligned");
    const size_t need = kvpub_mla_workspace_bytes(c.num_heads, c.max_query_len);
    if (workspace == nullptr) return fail(KVPUB_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, 256))
        return fail(KVPUB_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    if (workspace_bytes < need)
        return fail(KVPUB_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes,
                    need);
    a.out = static_cast<uint16_t *>(out);
    a.out_token = out_token;
    a.out_head = out_head;
    a.lse = lse;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev)) != KVPUB_OK || (st = sm_count(dev, &sms)) != KVPUB_OK)
        return st;
    CUtensorMap tiles, scales;
    if ((st = map_cache(a, 128, CU_TENSOR_MAP_SWIZZLE_128B, &tiles)) != KVPUB_OK ||
        (st = map_cache(a, 16, CU_TENSOR_MAP_SWIZZLE_NONE, &scales)) != KVPUB_OK)
        return st;
    int clusters[3][3];     // with 16, 32 and 64 rows
    if ((st = attention_clusters<16>(dev, &clusters[0])) != KVPUB_OK ||
        (st = attention_clusters<32>(dev, &clusters[1])) != KVPUB_OK ||
        (st = attention_clusters<64>(dev, &clusters[2])) != KVPUB_OK)
        return st;
    const Split split = split_work(c, sms < kMaxCtas ? sms : kMaxCtas, clusters);
    Workspace ws;
    workspace_for(split.rows, static_cast<uint8_t *>(workspace), &ws);
    switch (split.rows) {
        case 16: return launch_attention<16>(a, ws, tiles, scales, split, stream);
        case 32: return launch_attention<32>(a, ws, tiles, scales, split, stream);
        default: return launch_attention<64>(a, ws, tiles, scales, split, stream);
    }
}

}  // namespace
}  // namespace kvpub

using namespace kvpub;

extern "C" size_t kvpub_mla_workspace_bytes(int num_heads, int max_query_len) {
    if (num_heads < 1 || num_heads > KVPUB_MAX_HEADS || max_query_len < 1 ||
        max_query_len > KVPUB_MAX_QUERY_TOKENS)
        return 0;
    return workspace_for(rows_for(num_heads, max_query_len), nullptr, nullptr);
}

extern "C" kvpub_status kvpub_mla_decode_fp8(
    const void *q_latent, int64_t q_latent_token_stride, int64_t q_latent_head_stride,
    const void *q_rope, int64_t q_rope_token_stride, int64_t q_rope_head_stride,
    int64_t num_seqs, int num_heads, const void *main_cache, int64_t num_blocks, int block_size,
    const int32_t *block_table, int64_t block_table_stride, int64_t max_blocks,
    const int32_t *seq_lens, float softmax_scale, void *out, int64_t out_token_stride,
    int64_t out_head_stride, float *lse, unsigned long long *invalid_count, void *workspace,
    size_t workspace_bytes, kvpub_stream_t stream) {
    const MlaCall c{q_latent,   q_latent_token_stride, q_latent_head_stride, q_rope,
                    q_rope_token_stride, q_rope_head_stride, num_seqs, num_seqs, 1, num_heads,
                    main_cache, num_blocks, block_size, block_table, block_table_stride,
                    max_blocks, seq_lens, nullptr, nullptr, softmax_scale, invalid_count};
    return attention(c, out, out_token_stride, out_head_stride, lse, workspace, workspace_bytes,
                     (cudaStream_t)stream);
}

extern "C" kvpub_status kvpub_mla_tree_fp8(
    const void *q_latent, int64_t q_latent_token_stride, int64_t q_latent_head_stride,
    const void *q_rope, int64_t q_rope_token_stride, int64_t q_rope_head_stride,
    int64_t num_tokens, const int32_t *query_start, const uint64_t *tree_mask, int64_t num_seqs,
    int max_query_len, int num_heads, const void *main_cache, int64_t num_blocks, int block_size,
    const int32_t *block_table, int64_t block_table_stride, int64_t max_blocks,
    const int32_t *seq_lens, float softmax_scale, void *out, int64_t out_token_stride,
    int64_t out_head_stride, float *lse, unsigned long long *invalid_count, void *workspace,
    size_t workspace_bytes, kvpub_stream_t stream) {
    const MlaCall c{q_latent,   q_latent_token_stride, q_latent_head_stride, q_rope,
                    q_rope_token_stride, q_rope_head_stride, num_tokens, num_seqs, max_query_len,
                    num_heads, main_cache, num_blocks, block_size, block_table,
                    block_table_stride, max_blocks, seq_lens, query_start, tree_mask,
                    softmax_scale, invalid_count};
    if (query_start == nullptr) return fail(KVPUB_ERR_INVALID_ARG, "query_start is NULL");
    return attention(c, out, out_token_stride, out_head_stride, lse, workspace, workspace_bytes,
                     (cudaStream_t)stream);
}

