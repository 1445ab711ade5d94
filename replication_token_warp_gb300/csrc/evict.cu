// Eviction by accumulated attention weight.  The C ABI is declared in kvpub.h.
//
// Launch 1 works on a sequence with a cluster of 1 to 8 blocks.  It turns the
// weights and positions into order-preserving integer keys, held in
// registers, finds the budget-th largest by radix selection (passes of eight
// bits, histograms in shared memory, added over the cluster; once 32 or fewer
// keys are left, one warp ranks them), and then ranks the places in order with
// ballots and one scan: it writes the kept entries below the budget, and lists
// the holes (evicted places below the budget) and the movers (kept places at
// or above it), which are equally many.  A sequence too long for the registers
// is read again in every pass.  It is bound by latency: of its barriers, and
// of the one load of the weights and positions.
//
// Launch 2 moves the movers' rows into the holes, in every replica.  Sources
// lie at or above the budget and destinations below it, so all moves go at
// once.  It is bound by the rows' bytes, 788 read and written a row and
// replica.

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "host.cuh"
#include "kvpub.h"

namespace kvpub {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kMoveThreads = 256;

struct EvictArgs {
    const float *weights_in;
    int64_t weights_in_stride;
    const int32_t *positions_in;
    int64_t positions_in_stride;
    int64_t width;
    const int32_t *seq_lens;
    int num_seqs;
    const int32_t *block_table;
    int64_t table_stride;
    int64_t max_blocks;
    uint8_t *main[KVPUB_MAX_REPLICAS];
    uint8_t *indexer[KVPUB_MAX_REPLICAS];
    int num_replicas;
    int64_t num_blocks;
    int budget;
    int64_t num_sink, num_recent;
    float *weights_out;
    int64_t weights_out_stride;
    int32_t *positions_out;
    int64_t positions_out_stride;
    int32_t *lens_out;
    unsigned long long *invalid_count;
    int32_t *moves;     // [num_seqs]: how many rows move
    int32_t *holes;     // [num_seqs, budget]
    int32_t *movers;    // [num_seqs, budget]
    int rounds;         // places a thread of the selection holds
    int batch;          // moves a warp takes at a time
};

// Larger weight, larger key.  -0 as 0; NaN above every number; protected
// tokens above NaN.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int position_at(const EvictArgs &a, int b, int k) {
    return a.positions_in != nullptr ? a.positions_in[b * a.positions_in_stride + k] : k;
}

__device__ __forceinline__ uint32_t key_of(const EvictArgs &a, float w, int pos, int newest) {
    if (pos < a.num_sink || static_cast<int64_t>(pos) > newest - a.num_recent) return 0xffffffffu;
    return weight_key(w);
}

struct SelectShared {
    // read by the cluster's other blocks
    uint32_t hist[kBins];
    uint4 total;
    int newest;
    uint32_t few, left[32];     // the last keys to choose from

    uint4 warps[32];
    uint32_t sums[32];
    uint32_t bin, need, count;
};

// kThreads a block; kKeep places a thread can hold in registers (0: none, they
// are read again); kCluster: more than one block a sequence.  A warp owns
// consecutive places, 32 a round.
template <int kThreads, int kKeep, bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
    constexpr int kWarps = kThreads / 32;
    wait_previous_kernel();
    __shared__ SelectShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = kCluster ? static_cast<int>(cluster.num_blocks()) : 1;
    const int rank = kCluster ? static_cast<int>(cluster.block_rank()) : 0;
    auto sync_all = [&] {
        if (kCluster) cluster.sync();
        else __syncthreads();
    };
    auto peer = [&](int r) { return kCluster ? cluster.map_shared_rank(&s, r) : &s; };

    int64_t cap = a.max_blocks * KVPUB_BLOCK_SIZE;
    if (cap > a.width) cap = a.width;
    const int given = a.seq_lens[b];
    const int len = given < 0 ? 0 : (given > cap ? static_cast<int>(cap) : given);
    const bool evicts = len > a.budget;
    const float *w_in = a.weights_in + b * a.weights_in_stride;
    const int rounds = a.rounds;
    const int64_t begin64 = static_cast<int64_t>(rank * kWarps + warp) * rounds * 32 + lane;
    const int begin = begin64 > len ? len : static_cast<int>(begin64);
    if (tid == 0) {
        s.newest = -1;
        s.few = 0;
    }
    __syncthreads();

    constexpr int kHeld = kKeep > 0 ? kKeep : 1;
    uint32_t key[kHeld];
    int newest = -1;
    {
        float w[kHeld];
        int pos[kHeld];
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            const int k = j < rounds ? begin + 32 * j : len;
            w[j] = evicts && k < len ? w_in[k] : 0.f;
            pos[j] = evicts && k < len ? position_at(a, b, k) : -1;
        }
#pragma unroll
        for (int j = 0; j < kKeep; ++j) newest = max(newest, pos[j]);
        if (kKeep == 0 && evicts) {
            for (int j = 0; j < rounds; ++j) {
                const int k = begin + 32 * j;
                if (k < len) newest = max(newest, position_at(a, b, k));
            }
        }
        newest = __reduce_max_sync(~0u, newest);
        if (lane == 0) atomicMax(&s.newest, newest);
        sync_all();
        // A block may only read the others' shared memory while they are sure to
        // run: here the barriers below keep them.  A sequence within its budget
        // meets no more barriers, and needs no newest position.
        if (evicts)
            for (int r = 0; r < blocks; ++r) newest = max(newest, peer(r)->newest);
        // (lens_out may be seq_lens: all blocks have read it by now)
        if (rank == 0 && tid == 0) {
            if (given != len && a.invalid_count != nullptr) atomicAdd(a.invalid_count, 1ull);
            a.lens_out[b] = min(len, a.budget);
        }
#pragma unroll
        for (int j = 0; j < kKeep; ++j) key[j] = key_of(a, w[j], pos[j], newest);
    }
    // f(place, key) for the thread's places in order; the place is len where
    // there is none
    auto each = [&](auto f) {
        if constexpr (kKeep > 0) {
#pragma unroll
            for (int j = 0; j < kKeep; ++j)
                if (j < rounds) f(min(begin + 32 * j, len), key[j]);
        } else {
            for (int j = 0; j < rounds; ++j) {
                const int k = min(begin + 32 * j, len);
                uint32_t x = 0;
                if (evicts && k < len) x = key_of(a, w_in[k], position_at(a, b, k), newest);
                f(k, x);
            }
        }
    };

    // of the keys that start with `prefix`, `need` stay
    uint32_t prefix = 0, need = a.budget;
    if (evicts) {
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < kBins) s.hist[tid] = 0;
            __syncthreads();
            each([&](int k, uint32_t x) {
                const bool in =
                    k < len && (shift == 24 || (x >> (shift + 8)) == (prefix >> (shift + 8)));
                if (!__any_sync(~0u, in)) return;
                const uint32_t bin = in ? (x >> shift) & 255u : kBins;
                // equal weights are common: one addition for a warp of them
                int same;
                __match_all_sync(~0u, bin, &same);
                if (same) {
                    if (in && lane == 0) atomicAdd(&s.hist[bin], 32u);
                } else if (in) {
                    atomicAdd(&s.hist[bin], 1u);
                }
            });
            sync_all();
            // thread t < 256 holds bin 255 - t: the largest first
            const int bin = kBins - 1 - tid;
            uint32_t n = 0;
            if (tid < kBins) {
#pragma unroll
                for (int r = 0; r < (kCluster ? kMaxCluster : 1); ++r)
                    if (r < blocks) n += peer(r)->hist[bin];
            }
            uint32_t sum = n;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t z = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += z;
            }
            if (lane == 31) s.sums[warp] = sum;
            __syncthreads();
            uint32_t before = sum - n;
#pragma unroll
            for (int w = 0; w < kBins / 32; ++w) before += w < warp ? s.sums[w] : 0;
            if (tid < kBins && before < need && need <= before + n) {
                s.bin = bin;
                s.need = need - before;
                s.count = n;
            }
            sync_all();      // every block's histogram is read
            prefix |= s.bin << shift;
            need = s.need;
            if (shift == 16 && s.count <= 32) {
                // Few keys start so: gather them, and let every warp find the
                // one of which `need` stay.
                each([&](int k, uint32_t x) {
                    if (k < len && (x >> 16) == (prefix >> 16)) s.left[atomicAdd(&s.few, 1u)] = x;
                });
                sync_all();
                uint32_t mine = 0;
                int first = 0;
                for (int r = 0; r < blocks; ++r) {
                    const int there = static_cast<int>(peer(r)->few);
                    if (lane >= first && lane < first + there) mine = peer(r)->left[lane - first];
                    first += there;
                }
                uint32_t above = 0, equal = 0;
                for (int i = 0; i < 32; ++i) {
                    const uint32_t x = __shfl_sync(~0u, mine, i);
                    above += x > mine;
                    equal += x == mine;
                }
                const uint32_t it =
                    __ballot_sync(~0u, mine != 0 && above < need && need <= above + equal);
                const int at = __ffs(it) - 1;
                prefix = __shfl_sync(~0u, mine, at);
                need -= __shfl_sync(~0u, above, at);
                break;
            }
        }
    }

    // Keys above `prefix` stay, and the first `need` of those equal to it.
    // Counted a warp, below the budget (x, z) and not (y, w): keys above
    // `prefix`, and equal to it.
    const uint32_t below = (1u << lane) - 1;
    uint4 at = make_uint4(0, 0, 0, 0);
    if (evicts) {
        uint4 n = make_uint4(0, 0, 0, 0);
        each([&](int k, uint32_t x) {
            const uint32_t low = __ballot_sync(~0u, k < a.budget);
            const uint32_t gt = __ballot_sync(~0u, k < len && x > prefix);
            const uint32_t eq = __ballot_sync(~0u, k < len && x == prefix);
            n.x += __popc(gt & low);
            n.y += __popc(gt & ~low);
            n.z += __popc(eq & low);
            n.w += __popc(eq & ~low);
        });
        if (lane == 0) s.warps[warp] = n;
        __syncthreads();
        uint4 all = make_uint4(0, 0, 0, 0);
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) {
            const uint4 v = s.warps[w];
            if (w == warp) at = all;
            all.x += v.x, all.y += v.y, all.z += v.z, all.w += v.w;
        }
        if (kCluster) {
            if (tid == 0) s.total = all;
            cluster.sync();
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                if (r < rank) {
                    const uint4 v = peer(r)->total;
                    at.x += v.x, at.y += v.y, at.z += v.z, at.w += v.w;
                }
            }
            cluster.sync();
        }
    }
    // In order of the places the equal ones below the budget come before the
    // others, so what stays before this warp follows from the counts.
    uint32_t tie = at.z + at.w;
    const uint32_t tie_low = min(need, at.z);
    const int start = begin - lane < a.budget ? begin - lane : a.budget;     // places below the budget
    uint32_t nholes = (start < len ? start : len) - at.x - tie_low;
    uint32_t nmovers = at.y + min(need, tie) - tie_low;
    int32_t *holes = a.holes + static_cast<int64_t>(b) * a.budget;
    int32_t *movers = a.movers + static_cast<int64_t>(b) * a.budget;
    uint32_t kept = 0;      // a bit a round: the entry stays where it is
    int j = 0;
    auto copy = [&](int k) {
        a.weights_out[b * a.weights_out_stride + k] = w_in[k];
        if (a.positions_out != nullptr)
            a.positions_out[b * a.positions_out_stride + k] = position_at(a, b, k);
    };
    each([&](int k, uint32_t x) {
        bool keep = k < len;
        if (evicts) {
            const bool equal = k < len && x == prefix;
            const uint32_t votes = __ballot_sync(~0u, equal);
            keep = k < len && (x > prefix || (equal && tie + __popc(votes & below) < need));
            tie += __popc(votes);
            const bool hole = k < len && k < a.budget && !keep, mover = keep && k >= a.budget;
            const uint32_t h = __ballot_sync(~0u, hole), m = __ballot_sync(~0u, mover);
            if (hole) holes[nholes + __popc(h & below)] = k;
            if (mover) movers[nmovers + __popc(m & below)] = k;
            nholes += __popc(h);
            nmovers += __popc(m);
        }
        keep = keep && k < a.budget;
        if (kKeep == 0 && keep) copy(k);
        kept |= static_cast<uint32_t>(keep) << j;
        ++j;
    });
    if (rank == blocks - 1 && tid == kThreads - 32) a.moves[b] = evicts ? nholes : 0;
    // the entries that stay, all loads before the stores
    if constexpr (kKeep > 0) {
        float w[kKeep];
        int pos[kKeep];
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if ((kept >> i) & 1) {
                w[i] = w_in[begin + 32 * i];
                if (a.positions_out != nullptr) pos[i] = position_at(a, b, begin + 32 * i);
            }
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if ((kept >> i) & 1) {
                a.weights_out[b * a.weights_out_stride + begin + 32 * i] = w[i];
                if (a.positions_out != nullptr)
                    a.positions_out[b * a.positions_out_stride + begin + 32 * i] = pos[i];
            }
        }
    }
}

// A warp takes `batch` moves (a power of two, at most 8): its lanes look the
// places up in the table (the destinations in the first half, the sources in
// the second), and then the rows follow one another, the loads of kReplicas
// replicas before their stores.  A row is 41 chunks of 16 bytes in the Main
// cache, 8 in the Indexer cache, and its scale.  The loads of more rows before
// their stores cost the registers of the warps that hide them: when this was
// tried, 2 x 2 rows made 64 sequences of up to 8,192 places in two replicas take
// 46 us instead of 40.
template <int kReplicas>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    wait_previous_kernel();
    const int lane = threadIdx.x & 31, b = blockIdx.y, batch = a.batch;
    const int n = a.moves[b];
    const int stride = gridDim.x * (kMoveThreads / 32) * batch;
    // this lane's second chunk: Main 32-40, Indexer 0-7, the scale
    const bool more = lane < 9, codes = lane >= 9 && lane < 17, scale = lane == 17;
    for (int i0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * batch; i0 < n;
         i0 += stride) {
        const int count = min(batch, n - i0), mine = lane & 15;
        int64_t slot = -1;
        int place = 0;
        if (mine < count) {
            place = (lane < 16 ? a.holes : a.movers)[static_cast<int64_t>(b) * a.budget + i0 + mine];
            const int64_t blk = a.block_table[b * a.table_stride + (place >> 6)];
            if (blk >= 0 && blk < a.num_blocks) slot = blk * 64 + (place & 63);
        }
        const int from = __shfl_down_sync(~0u, place, 16);
        const bool bad = slot < 0;
        const bool bad_from = __shfl_down_sync(~0u, bad, 16);
        for (int m = 0; m < count; ++m) {
            const int64_t to = __shfl_sync(~0u, slot, m), src = __shfl_sync(~0u, slot, 16 + m);
            if (to < 0 || src < 0) continue;
            for (int r0 = 0; r0 < a.num_replicas; r0 += kReplicas) {
                uint4 x[kReplicas], y[kReplicas];
#pragma unroll
                for (int r = 0; r < kReplicas; ++r) {
                    if (r0 + r >= a.num_replicas) continue;
                    const uint4 *row = reinterpret_cast<const uint4 *>(
                        a.main[r0 + r] + src * KVPUB_MAIN_SLOT_BYTES);
                    const uint8_t *index = a.indexer[r0 + r] + (src >> 6) * KVPUB_INDEXER_BLOCK_BYTES;
                    x[r] = row[lane];
                    if (more) y[r] = row[32 + lane];
                    if (codes)
                        y[r] = reinterpret_cast<const uint4 *>(index + (src & 63) * 128)[lane - 9];
                    if (scale) y[r].x = reinterpret_cast<const uint32_t *>(index + 8192)[src & 63];
                }
#pragma unroll
                for (int r = 0; r < kReplicas; ++r) {
                    if (r0 + r >= a.num_replicas) continue;
                    uint4 *row =
                        reinterpret_cast<uint4 *>(a.main[r0 + r] + to * KVPUB_MAIN_SLOT_BYTES);
                    uint8_t *index = a.indexer[r0 + r] + (to >> 6) * KVPUB_INDEXER_BLOCK_BYTES;
                    row[lane] = x[r];
                    if (more) row[32 + lane] = y[r];
                    if (codes) reinterpret_cast<uint4 *>(index + (to & 63) * 128)[lane - 9] = y[r];
                    if (scale) reinterpret_cast<uint32_t *>(index + 8192)[to & 63] = y[r].x;
                }
            }
        }
        if (lane < count) {
            a.weights_out[b * a.weights_out_stride + place] =
                a.weights_in[b * a.weights_in_stride + from];
            if (a.positions_out != nullptr)
                a.positions_out[b * a.positions_out_stride + place] = position_at(a, b, from);
            if ((bad || bad_from) && a.invalid_count != nullptr) atomicAdd(a.invalid_count, 1ull);
        }
    }
}

template <int kThreads, int kKeep, bool kCluster>
cudaError_t launch_select(const EvictArgs &a, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster, a.num_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<kThreads, kKeep, kCluster>, a);
}

// One block for sequences of up to 4,096 places: with 256 threads up to 1,024,
// where its barriers are most of the time. Above that a cluster that leaves a
// thread about 8 places, 16 at most (256 threads with 24 places each took 34 us
// instead of 27 for 16 x 40,960 places);
// longer sequences are read again in every pass.
cudaError_t select(EvictArgs &a, int64_t longest, cudaStream_t stream) {
    int cluster = 1;
    while (cluster < kMaxCluster && longest > cluster * 512 * 8) cluster *= 2;
    const int64_t threads = longest <= 1024 ? 256 : longest > cluster * 512 * 16 ? 1024 : 512;
    a.rounds = static_cast<int>((longest + cluster * threads - 1) / (cluster * threads));
    if (threads == 1024) return launch_select<1024, 0, true>(a, cluster, stream);
    if (threads == 256) return launch_select<256, 4, false>(a, cluster, stream);
    if (cluster == 1) return launch_select<512, 8, false>(a, cluster, stream);
    if (a.rounds <= 8) return launch_select<512, 8, true>(a, cluster, stream);
    return launch_select<512, 16, true>(a, cluster, stream);
}

constexpr int64_t kMaxBudget = 1 << 24;

}  // namespace
}  // namespace kvpub

using namespace kvpub;

extern "C" size_t kvpub_evict_workspace_bytes(int64_t num_seqs, int64_t budget) {
    if (num_seqs < 1 || num_seqs > 65535 || budget < 1 || budget > kMaxBudget) return 0;
    return static_cast<size_t>(num_seqs) * (static_cast<size_t>(budget) * 8 + 4) + 16;
}

extern "C" kvpub_status kvpub_evict_fp8(
    const float *weights_in, int64_t weights_in_stride, const int32_t *positions_in,
    int64_t positions_in_stride, int64_t width, const int32_t *seq_lens, int64_t num_seqs,
    const int32_t *block_table, int64_t block_table_stride, int64_t max_blocks,
    void *const *main_caches, void *const *indexer_caches, int num_replicas, int64_t num_blocks,
    int block_size, int64_t budget, int64_t num_sink, int64_t num_recent, float *weights_out,
    int64_t weights_out_stride, int32_t *positions_out, int64_t positions_out_stride,
    int32_t *lens_out, unsigned long long *invalid_count, void *workspace, size_t workspace_bytes,
    kvpub_stream_t stream) {
    if (num_replicas < 1) return fail(KVPUB_ERR_INVALID_ARG, "num_replicas %d < 1", num_replicas);
    if (num_replicas > KVPUB_MAX_REPLICAS)
        return fail(KVPUB_ERR_TOO_MANY_REPLICAS, "num_replicas %d > %d", num_replicas,
                    KVPUB_MAX_REPLICAS);
    if (block_size != KVPUB_BLOCK_SIZE)
        return fail(KVPUB_ERR_INVALID_ARG, "block_size %d != %d", block_size, KVPUB_BLOCK_SIZE);
    if (num_blocks < 1 || num_blocks > INT64_MAX / (KVPUB_BLOCK_SIZE * KVPUB_MAIN_SLOT_BYTES))
        return fail(KVPUB_ERR_INVALID_ARG, "num_blocks %lld out of range", (long long)num_blocks);
    if (num_seqs < 0 || num_seqs > 65535)
        return fail(KVPUB_ERR_INVALID_ARG, "num_seqs %lld outside [0, 65535]", (long long)num_seqs);
    if (budget < 1 || budget > kMaxBudget)
        return fail(KVPUB_ERR_INVALID_ARG, "budget %lld outside [1, %lld]", (long long)budget,
                    (long long)kMaxBudget);
    if (num_sink < 0 || num_recent < 0 || num_sink > budget || num_recent > budget - num_sink)
        return fail(KVPUB_ERR_INVALID_ARG, "num_sink %lld and num_recent %lld exceed the budget",
                    (long long)num_sink, (long long)num_recent);
    const int64_t most = INT64_MAX / 8 / 65536;
    if (width < 0 || width > (1 << 30) || weights_in_stride < width || weights_in_stride > most ||
        (positions_in != nullptr && (positions_in_stride < width || positions_in_stride > most)))
        return fail(KVPUB_ERR_INVALID_ARG, "width %lld does not fit the input rows",
                    (long long)width);
    const int64_t kept = budget < width ? budget : width;
    if (weights_out_stride < kept || weights_out_stride > most ||
        (positions_out != nullptr && (positions_out_stride < kept || positions_out_stride > most)))
        return fail(KVPUB_ERR_INVALID_ARG, "the output rows hold fewer than %lld entries",
                    (long long)kept);
    if (max_blocks < 0 || max_blocks > INT32_MAX / KVPUB_BLOCK_SIZE - 2 ||
        block_table_stride < max_blocks || block_table_stride > most)
        return fail(KVPUB_ERR_INVALID_ARG, "block_table of %lld blocks with row stride %lld",
                    (long long)max_blocks, (long long)block_table_stride);
    if (main_caches == nullptr || indexer_caches == nullptr)
        return fail(KVPUB_ERR_INVALID_ARG, "cache pointer arrays are NULL");
    if (!aligned(invalid_count, 8))
        return fail(KVPUB_ERR_ALIGNMENT, "invalid_count is not 8-byte aligned");
    EvictArgs a{};
    for (int r = 0; r < num_replicas; ++r) {
        if (main_caches[r] == nullptr || indexer_caches[r] == nullptr)
            return fail(KVPUB_ERR_INVALID_ARG, "cache pointer of replica %d is NULL", r);
        if (!aligned(main_caches[r], 16) || !aligned(indexer_caches[r], 16))
            return fail(KVPUB_ERR_ALIGNMENT, "cache of replica %d is not 16-byte aligned", r);
        a.main[r] = static_cast<uint8_t *>(main_caches[r]);
        a.indexer[r] = static_cast<uint8_t *>(indexer_caches[r]);
    }
    if (num_seqs == 0) return ok();
    if (weights_in == nullptr || seq_lens == nullptr || block_table == nullptr ||
        weights_out == nullptr || lens_out == nullptr)
        return fail(KVPUB_ERR_INVALID_ARG,
                    "weights_in, seq_lens, block_table, weights_out or lens_out is NULL");
    if (positions_in != nullptr && positions_out == nullptr)
        return fail(KVPUB_ERR_INVALID_ARG, "positions_out is NULL");
    if (!aligned(weights_in, 4) || !aligned(positions_in, 4) || !aligned(seq_lens, 4) ||
        !aligned(block_table, 4) || !aligned(weights_out, 4) || !aligned(positions_out, 4) ||
        !aligned(lens_out, 4))
        return fail(KVPUB_ERR_ALIGNMENT, "a weights, positions, length or table pointer is misaligned");
    // (a single row has no use for its stride)
    if (num_seqs > 1 && ((weights_in == weights_out && weights_in_stride != weights_out_stride) ||
                         (positions_in != nullptr && positions_in == positions_out &&
                          positions_in_stride != positions_out_stride)))
        return fail(KVPUB_ERR_INVALID_ARG, "in place needs one row stride");
    const size_t bytes = kvpub_evict_workspace_bytes(num_seqs, budget);
    if (workspace == nullptr) return fail(KVPUB_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, 16))
        return fail(KVPUB_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
    if (workspace_bytes < bytes)
        return fail(KVPUB_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes,
                    bytes);
    a.weights_in = weights_in;
    a.weights_in_stride = weights_in_stride;
    a.positions_in = positions_in;
    a.positions_in_stride = positions_in_stride;
    a.width = width;
    a.seq_lens = seq_lens;
    a.num_seqs = static_cast<int>(num_seqs);
    a.block_table = block_table;
    a.table_stride = block_table_stride;
    a.max_blocks = max_blocks;
    a.num_replicas = num_replicas;
    a.num_blocks = num_blocks;
    a.budget = static_cast<int>(budget);
    a.num_sink = num_sink;
    a.num_recent = num_recent;
    a.weights_out = weights_out;
    a.weights_out_stride = weights_out_stride;
    a.positions_out = positions_out;
    a.positions_out_stride = positions_out_stride;
    a.lens_out = lens_out;
    a.invalid_count = invalid_count;
    a.moves = static_cast<int32_t *>(workspace);
    a.holes = a.moves + num_seqs;
    a.movers = a.holes + num_seqs * budget;
    (void)cudaGetLastError();
    const cudaStream_t st_ = (cudaStream_t)stream;
    // the longest a sequence can be
    int64_t longest = max_blocks * KVPUB_BLOCK_SIZE;
    if (longest > width) longest = width;
    (void)select(a, longest, st_);
    kvpub_status st = launched("evict_select");
    if (st != KVPUB_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev)) != KVPUB_OK || (st = sm_count(dev, &sms)) != KVPUB_OK)
        return st;
    // As few moves a warp as leave 32 warps an SM, if all that can move do, and
    // 8 at most: alone a move's latency counts, in a large launch the look-ups
    // before the rows do (64 sequences of 513 to 8,192 places in two replicas: 51.5 us
    // with 1, 44.3 with 8, 59 with 16, which leave too few warps).
    const int64_t most_moves = longest <= budget ? 0 : budget < longest - budget ? budget : longest - budget;
    a.batch = 1;
    while (a.batch < 8 && most_moves * num_seqs > static_cast<int64_t>(sms) * 32 * a.batch)
        a.batch *= 2;
    const int64_t each = a.batch * (kMoveThreads / 32);
    const int64_t blocks = most_moves < 1 ? 1 : (most_moves + each - 1) / each;
    const dim3 grid(static_cast<unsigned>(blocks), a.num_seqs);
    if (num_replicas == 1)
        (void)launch_smem(evict_move_kernel<1>, grid, kMoveThreads, 0, st_, 1, a);
    else if (num_replicas == 2)
        (void)launch_smem(evict_move_kernel<2>, grid, kMoveThreads, 0, st_, 1, a);
    else
        (void)launch_smem(evict_move_kernel<4>, grid, kMoveThreads, 0, st_, 1, a);
    return launched("evict_move");
}
