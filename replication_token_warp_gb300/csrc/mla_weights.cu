// Each cached token's attention weight.  The C ABI is declared in kvpub.h.
//
//   weights_out[k] = decay * weights_in[k] + sum over rows of 2^(s[k, row] - lse[row])
//
// The scores are formed as in mla.cu: K Q^T on the tensor cores, the cache's
// codes undecoded, keys as the accumulators' lanes.  A thread sums its key's
// weights over its part of the rows, the parts are added through shared
// memory, and one thread a key updates its sum: no atomics, and the same order
// every time.  For that the rows' tiles of a run of keys are done by the same
// block one after another (their keys come from L2 after the first), or, where
// units are few, by the blocks of a cluster, whose first one adds them up.
// Bound by the cache's bytes up to 64 rows a sequence: 32 sequences of 8k
// tokens, 64 heads, take 39 us, 4.2 TB/s.

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

// The weights' share: a run of units of a sequence for all of its tiles. The
// run's ends are rounded down to whole units, the same for both neighbours.
template <class S>
struct Runs {
    Share share;
    int tiles;
    bool more;      // tiles of the run at hand

    __device__ __forceinline__ bool next(const MlaArgs &a, Segment &g) {
        if (more && ++g.tile < tiles) {
            g.counts = false;
            return true;
        }
        more = false;
        while (share.left > 0 && share.seq < a.num_seqs) {
            g.s = sequence(a, share.seq);
            tiles = tiles_of<S>(a, g.s);
            g.units = units_of(g.s);
            const int64_t all = static_cast<int64_t>(tiles) * g.units;
            int64_t end = share.offset + share.left;
            if (end > all) end = all;
            g.seq = share.seq;
            g.tile = 0;
            g.counts = true;
            if (tiles > 0) {
                g.begin = static_cast<int>(share.offset / tiles);
                g.end = static_cast<int>(end / tiles);
            }
            share.left -= end - share.offset;
            share.offset = 0;
            ++share.seq;
            if (tiles > 0 && g.begin < g.end) {
                more = true;
                return true;
            }
        }
        return false;
    }
};

// A cluster's share: one unit of a sequence, whose tiles its blocks take in
// turn. A block adds up its own, and the first one adds the blocks' sums.
template <class S>
struct OneUnit {
    int seq, unit, tile, step;

    __device__ __forceinline__ bool next(const MlaArgs &a, Segment &g) {
        g.s = sequence(a, seq);
        g.units = units_of(g.s);
        if (unit >= g.units || tile >= tiles_of<S>(a, g.s)) return false;
        g.seq = seq;
        g.tile = tile;
        g.begin = unit;
        g.end = unit + 1;
        g.counts = tile == 0;
        tile += step;
        return true;
    }
};

// In a cluster: where a block's sums of the unit's keys are for the first
// block (the other half of the parts' buffers).
template <class S>
__device__ __forceinline__ float *unit_sums(Misc<S> &m, int unit) {
    return reinterpret_cast<float *>(m.keys) + ((unit & 1) ^ 1) * 3 * kUnit;
}

template <class S, bool kCluster, typename Source>
__device__ void sum_role(const MlaArgs &a, uint8_t *smem, Misc<S> &m, Source source) {
    constexpr int kC = S::kCols;
    constexpr int kAll = S::kParts + 1;         // barrier of all of these warps
    const Lane t = softmax_lane(m.tmem);
    const int row0 = t.part * kC;
    float *sums = reinterpret_cast<float *>(m.keys);
    const Bars<S> bars{smem_addr(&m)};
    Waiter<S> wait{m, true};
    Ring<2> pieces, sring;
    Segment g;
    float total = 0.f;      // in a cluster, over this block's tiles
    while (source.next(a, g)) {
        named_barrier(kAll, S::kWarps * 32);     // the last segment's rows are done with
        load_queries<S>(a, g, smem, m, nullptr);
        if (threadIdx.x < S::kRows) {
            const int row = g.tile * S::kRows + threadIdx.x;
            m.nref[threadIdx.x] =
                row < g.s.count * a.num_heads
                    ? -kLog2e * a.lse_in[static_cast<int64_t>(g.s.first) * a.num_heads + row]
                    : -INFINITY;
            // lse -inf: the row adds nothing
            if (m.nref[threadIdx.x] == INFINITY) m.nref[threadIdx.x] = -INFINITY;
        }
        fence_async_smem();
        named_barrier(kAll, S::kWarps * 32);
        if (t.lane == 0) mbar_arrive(bars.query_ready());
        const int prefix = g.s.len - g.s.count;
        for (int u = g.begin; u < g.end; ++u) {
            wait(bars.scale_full(sring.at), sring.pass);
            const bool there = (m.valid[sring.at] >> (t.key >> 6)) & 1;
            const int key = u * kUnit + t.key;
            const bool on = there && key < g.s.len;

            // the running sum, asked for early
            const bool writes = t.part == 0 && key < g.s.len && key < a.width;
            float before = 0.f;
            if (writes && !kCluster) {
                if (g.tile > 0)
                    before = a.weights_out[g.seq * a.weights_out_stride + key];
                else if (a.weights_in != nullptr)
                    before = a.decay * a.weights_in[g.seq * a.weights_in_stride + key];
            }

            float2 z[kC / 2];
#pragma unroll
            for (int c = 0; c < kC / 2; ++c) z[c] = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int i = 0; i < S::kBunches; ++i) {
                add_bunch<S>(t, bars, wait, pieces, i, m.scales[sring.at][t.key], z);
                pieces.step();
            }
            if (t.lane == 0) mbar_arrive(bars.scale_empty(sring.at));
            sring.step();
            float2 sum2 = make_float2(0.f, 0.f);
            const int j = key - prefix;
#pragma unroll
            for (int c = 0; c < kC / 4; ++c) {
                const float4 f = *reinterpret_cast<const float4 *>(&m.factor[row0 + 4 * c]);
                const float4 r = *reinterpret_cast<const float4 *>(&m.nref[row0 + 4 * c]);
                float2 x = fma2(z[2 * c], make_float2(f.x, f.y), make_float2(r.x, r.y));
                float2 y = fma2(z[2 * c + 1], make_float2(f.z, f.w), make_float2(r.z, r.w));
                x.x = r.x == -INFINITY ? 0.f : exp2_approx(x.x);
                x.y = r.y == -INFINITY ? 0.f : exp2_approx(x.y);
                y.x = r.z == -INFINITY ? 0.f : exp2_approx(y.x);
                y.y = r.w == -INFINITY ? 0.f : exp2_approx(y.y);
                if (j >= 0 && on) {
                    const uint64_t *mask = &m.mask[row0 + 4 * c];
                    if (!((mask[0] >> j) & 1)) x.x = 0.f;
                    if (!((mask[1] >> j) & 1)) x.y = 0.f;
                    if (!((mask[2] >> j) & 1)) y.x = 0.f;
                    if (!((mask[3] >> j) & 1)) y.y = 0.f;
                }
                sum2 = add2(sum2, add2(x, y));
            }
            float sum = !wait.alive ? NAN : on ? sum2.x + sum2.y : 0.f;     // see Waiter
            // two buffers: a part is at most one barrier ahead
            float *part = sums + (u & 1) * 3 * kUnit;
            if (t.part > 0) part[(t.part - 1) * kUnit + t.key] = sum;
            named_barrier(kAll, S::kWarps * 32);
            if (writes) {
#pragma unroll
                for (int p = 1; p < S::kParts; ++p) sum += part[(p - 1) * kUnit + t.key];
                if (kCluster) total += sum;
                else a.weights_out[g.seq * a.weights_out_stride + key] = before + sum;
            }
        }
    }
    if constexpr (kCluster)
        if (t.part == 0) unit_sums<S>(m, source.unit)[t.key] = total;
}

template <int kRows, bool kCluster>
__global__ void __launch_bounds__(Shape<kRows, false>::kThreads, 1)
mla_weights_kernel(const MlaArgs a, const __grid_constant__ CUtensorMap tiles,
                   const __grid_constant__ CUtensorMap scales) {
    using S = Shape<kRows, false>;
    extern __shared__ __align__(1024) uint8_t raw[];
    Misc<S> *m;
    uint8_t *smem = block_setup<S>(raw, m);
    wait_previous_kernel();
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
    auto work = [&](auto source) {
        if (warp < S::kWarps)
            sum_role<S, kCluster>(a, smem, *m, source);
        else if (warp == S::kLoadWarp)
            load_role<S>(a, &tiles, &scales, smem, *m, source);
        else if (warp == S::kScoreWarp)
            score_role<S>(a, smem_addr(smem), *m, source);
        __syncwarp();
    };
    if constexpr (kCluster) {
        cg::cluster_group cluster = cg::this_cluster();
        const int blocks = static_cast<int>(cluster.num_blocks());
        const int rank = static_cast<int>(cluster.block_rank());
        const int longest = units_at_most(a.max_blocks), unit = blockIdx.x / blocks % longest;
        const int seq = blockIdx.x / blocks / longest, key = unit * kUnit + threadIdx.x;
        work(OneUnit<S>{seq, unit, rank, blocks});
        cluster.sync();
        if (rank == 0 && threadIdx.x < kUnit && key < sequence(a, seq).len && key < a.width) {
            float sum = 0.f;
            if (a.weights_in != nullptr)
                sum = a.decay * a.weights_in[seq * a.weights_in_stride + key];
            for (int r = 0; r < blocks; ++r)
                sum += cluster.map_shared_rank(unit_sums<S>(*m, unit), r)[threadIdx.x];
            a.weights_out[seq * a.weights_out_stride + key] = sum;
        }
        cluster.sync();     // the sums are read
    } else {
        int blocks;
        const Share share = find_work<S>(a, *m, &blocks);
        if (static_cast<int>(blockIdx.x) < blocks) work(Runs<S>{share, 0, false});
    }
    block_end<S>(a, *m);
}

// Without clusters a block does all tiles of a run of units, so that no more
// blocks than units work. Clusters share out the tiles of single units. A tile
// costs about 3 us and each of its units 2 (one alone 5), which gives the
// faster form, by the longest lengths that the table allows: 11 sequences of
// 119 to 233 tokens with 6 x 96 rows take 50 us without clusters and 19 with
// them; 3 of 2,000 tokens with 64 x 64 rows 335 and 170; 8 of 1,000 tokens with
// 6 x 32 rows 19 and 14.
inline int weights_cluster(int64_t units, int64_t tiles, int sms, const int (&clusters)[3]) {
    int64_t best = tiles * (3 + 2 * ((units + sms - 1) / sms));
    int cluster = 1;
    for (int i = 0; i < 3 && (1 << i) < tiles && units < (1 << 20) && clusters[i] > 0; ++i) {
        const int64_t n = 2 << i, waves = (units + clusters[i] - 1) / clusters[i];
        const int64_t cost = waves * ((tiles + n - 1) / n) * 5;
        if (cost < best) {
            best = cost;
            cluster = static_cast<int>(n);
        }
    }
    return cluster;
}

template <int kRows>
kvpub_status launch_weights(const MlaArgs &a, const CUtensorMap &tiles, const CUtensorMap &scales,
                            int sms, cudaStream_t stream) {
    using S = Shape<kRows, false>;
    static std::atomic<bool> opted[kMaxDevices];
    if constexpr (kRows == 64) {
        static std::atomic<bool> opted_cluster[kMaxDevices];
        int dev, clusters[3];
        kvpub_status st = current_device(&dev);
        if (st == KVPUB_OK)
            st = clusters_at_once<mla_weights_kernel<64, true>>(dev, S::kThreads, smem_bytes<S>(),
                                                                &clusters);
        if (st != KVPUB_OK) return st;
        const int64_t units = static_cast<int64_t>(a.num_seqs) * units_at_most(a.max_blocks);
        const int tiles_most = (a.num_heads * a.max_query_len + S::kRows - 1) / S::kRows;
        const int cluster = weights_cluster(units, tiles_most, sms, clusters);
        if (cluster > 1)
            return launch_opted("mla_weights", mla_weights_kernel<64, true>, opted_cluster, cluster,
                                static_cast<int>(units) * cluster, S::kThreads, smem_bytes<S>(),
                                stream, a, tiles, scales);
    }
    return launch_opted("mla_weights", mla_weights_kernel<kRows, false>, opted, 1, sms,
                        S::kThreads, smem_bytes<S>(), stream, a, tiles, scales);
}

}  // namespace
}  // namespace kvpub

using namespace kvpub;

extern "C" kvpub_status kvpub_mla_weights_fp8(
    const void *q_latent, int64_t q_latent_token_stride, int64_t q_latent_head_stride,
    const void *q_rope, int64_t q_rope_token_stride, int64_t q_rope_head_stride, const float *lse,
    int64_t num_tokens, const int32_t *query_start, const uint64_t *tree_mask, int64_t num_seqs,
    int max_query_len, int num_heads, const void *main_cache, int64_t num_blocks, int block_size,
    const int32_t *block_table, int64_t block_table_stride, int64_t max_blocks,
    const int32_t *seq_lens, float softmax_scale, const float *weights_in,
    int64_t weights_in_stride, float decay, float *weights_out, int64_t weights_out_stride,
    int64_t width, unsigned long long *invalid_count, kvpub_stream_t stream) {
    const MlaCall c{q_latent,   q_latent_token_stride, q_latent_head_stride, q_rope,
                    q_rope_token_stride, q_rope_head_stride, num_tokens, num_seqs, max_query_len,
                    num_heads, main_cache, num_blocks, block_size, block_table,
                    block_table_stride, max_blocks, seq_lens, query_start, tree_mask,
                    softmax_scale, invalid_count};
    MlaArgs a;
    bool empty;
    kvpub_status st = check_call(c, true, &a, &empty);
    if (st != KVPUB_OK) return st;
    if (!(fabsf(decay) <= 3.402823466e38f))
        return fail(KVPUB_ERR_INVALID_ARG, "decay is not finite");
    if (width < 0) return fail(KVPUB_ERR_INVALID_ARG, "width %lld < 0", (long long)width);
    if (empty || width == 0) return ok();
    // no query tokens, and sums that stay as they are
    if (num_tokens == 0 && weights_in == weights_out && decay == 1.f) return ok();
    if ((num_tokens > 0 && lse == nullptr) || weights_out == nullptr)
        return fail(KVPUB_ERR_INVALID_ARG, "lse or weights_out is NULL");
    if (!aligned(lse, 4) || !aligned(weights_in, 4) || !aligned(weights_out, 4))
        return fail(KVPUB_ERR_ALIGNMENT, "lse, weights_in or weights_out is misaligned");
    const int64_t most = INT64_MAX / 8 / 65536;
    if (weights_out_stride < width || weights_out_stride > most ||
        (weights_in != nullptr && (weights_in_stride < width || weights_in_stride > most)))
        return fail(KVPUB_ERR_INVALID_ARG, "weights row stride below width %lld",
                    (long long)width);
    // (a single row has no use for its stride)
    if (num_seqs > 1 && weights_in == weights_out && weights_in_stride != weights_out_stride)
        return fail(KVPUB_ERR_INVALID_ARG, "weights in place need one row stride");
    a.lse_in = lse;
    a.weights_in = weights_in;
    a.weights_in_stride = weights_in_stride;
    a.decay = decay;
    a.weights_out = weights_out;
    a.weights_out_stride = weights_out_stride;
    a.width = width;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev)) != KVPUB_OK || (st = sm_count(dev, &sms)) != KVPUB_OK)
        return st;
    CUtensorMap tiles, scales;
    if ((st = map_cache(a, 128, CU_TENSOR_MAP_SWIZZLE_128B, &tiles)) != KVPUB_OK ||
        (st = map_cache(a, 16, CU_TENSOR_MAP_SWIZZLE_NONE, &scales)) != KVPUB_OK)
        return st;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (rows_for(num_heads, max_query_len)) {
        case 16: return launch_weights<16>(a, tiles, scales, sms, s);
        case 32: return launch_weights<32>(a, tiles, scales, sms, s);
        default: return launch_weights<64>(a, tiles, scales, sms, s);
    }
}
