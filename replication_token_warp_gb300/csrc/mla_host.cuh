// The host side that the attention and the weights calls share: checks of
// their arguments and the cache's tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "host.cuh"
#include "kvpub.h"
#include "mla.cuh"

namespace kvpub {

inline kvpub_status check_q(const void *p, int64_t token, int64_t head, const char *name) {
    if (p == nullptr) return fail(KVPUB_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 16)) return fail(KVPUB_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
    if (token < 0 || head < 0)
        return fail(KVPUB_ERR_INVALID_ARG, "%s has a negative stride", name);
    if (token % 8 != 0 || head % 8 != 0)
        return fail(KVPUB_ERR_ALIGNMENT, "%s strides %lld, %lld are not multiples of 8 elements",
                    name, (long long)token, (long long)head);
    if (token > INT64_MAX / 8 / INT32_MAX || head > INT64_MAX / 8 / KVPUB_MAX_HEADS)
        return fail(KVPUB_ERR_INVALID_ARG, "%s strides are too large", name);
    return KVPUB_OK;
}

struct MlaCall {
    const void *q_latent;
    int64_t q_latent_token, q_latent_head;
    const void *q_rope;
    int64_t q_rope_token, q_rope_head;
    int64_t num_tokens, num_seqs;
    int max_query_len, num_heads;
    const void *main_cache;
    int64_t num_blocks;
    int block_size;
    const int32_t *block_table;
    int64_t table_stride, max_blocks;
    const int32_t *seq_lens;
    const int32_t *query_start;
    const uint64_t *tree_mask;
    float softmax_scale;
    unsigned long long *invalid_count;
};

// What the three calls check alike.  *empty: there is nothing to do.  sums: a
// sequence without query tokens has a sum to update.
inline kvpub_status check_call(const MlaCall &c, bool sums, MlaArgs *out, bool *empty) {
    *empty = false;
    if (c.block_size != KVPUB_BLOCK_SIZE)
        return fail(KVPUB_ERR_INVALID_ARG, "block_size %d != %d", c.block_size, KVPUB_BLOCK_SIZE);
    if (c.num_heads < 1 || c.num_heads > KVPUB_MAX_HEADS)
        return fail(KVPUB_ERR_INVALID_ARG, "num_heads %d outside [1, %d]", c.num_heads,
                    KVPUB_MAX_HEADS);
    if (c.max_query_len < 1 || c.max_query_len > KVPUB_MAX_QUERY_TOKENS)
        return fail(KVPUB_ERR_INVALID_ARG, "max_query_len %d outside [1, %d]", c.max_query_len,
                    KVPUB_MAX_QUERY_TOKENS);
    if (c.num_seqs < 0 || c.num_seqs > 65535)
        return fail(KVPUB_ERR_INVALID_ARG, "num_seqs %lld outside [0, 65535]",
                    (long long)c.num_seqs);
    if (c.num_tokens < 0 || c.num_tokens > c.num_seqs * c.max_query_len)
        return fail(KVPUB_ERR_INVALID_ARG, "num_tokens %lld outside [0, num_seqs * max_query_len]",
                    (long long)c.num_tokens);
    if (c.query_start == nullptr && c.num_tokens != c.num_seqs)
        return fail(KVPUB_ERR_INVALID_ARG, "num_tokens %lld != num_seqs %lld without query_start",
                    (long long)c.num_tokens, (long long)c.num_seqs);
    // a slot is a 32-bit row coordinate of the cache's tensor map
    if (c.num_blocks < 1 || c.num_blocks > (INT32_MAX - 128) / KVPUB_BLOCK_SIZE)
        return fail(KVPUB_ERR_INVALID_ARG, "num_blocks %lld out of range", (long long)c.num_blocks);
    if (c.max_blocks < 0 || c.max_blocks > INT32_MAX / KVPUB_BLOCK_SIZE - 2 ||
        c.table_stride < c.max_blocks || c.table_stride > INT64_MAX / 8 / 65536)
        return fail(KVPUB_ERR_INVALID_ARG, "block_table of %lld blocks with row stride %lld",
                    (long long)c.max_blocks, (long long)c.table_stride);
    if (!(c.softmax_scale > 0.f) || c.softmax_scale > 3.402823466e38f)
        return fail(KVPUB_ERR_INVALID_ARG, "softmax_scale is not a positive finite number");
    if (c.invalid_count != nullptr && !aligned(c.invalid_count, 8))
        return fail(KVPUB_ERR_ALIGNMENT, "invalid_count is not 8-byte aligned");
    if (c.num_seqs == 0 || (c.num_tokens == 0 && !sums)) {
        *empty = true;
        return KVPUB_OK;
    }
    kvpub_status st;
    if (c.num_tokens > 0 &&
        ((st = check_q(c.q_latent, c.q_latent_token, c.q_latent_head, "q_latent")) != KVPUB_OK ||
         (st = check_q(c.q_rope, c.q_rope_token, c.q_rope_head, "q_rope")) != KVPUB_OK))
        return st;
    if (c.main_cache == nullptr) return fail(KVPUB_ERR_INVALID_ARG, "main_cache is NULL");
    if (!aligned(c.main_cache, 16))
        return fail(KVPUB_ERR_ALIGNMENT, "main_cache is not 16-byte aligned");
    if (c.block_table == nullptr || c.seq_lens == nullptr)
        return fail(KVPUB_ERR_INVALID_ARG, "block_table or seq_lens is NULL");
    if (!aligned(c.block_table, 4) || !aligned(c.seq_lens, 4) || !aligned(c.query_start, 4))
        return fail(KVPUB_ERR_ALIGNMENT, "block_table, seq_lens or query_start is misaligned");
    if (!aligned(c.tree_mask, 8))
        return fail(KVPUB_ERR_ALIGNMENT, "tree_mask is not 8-byte aligned");
    MlaArgs a{};
    a.q_latent = static_cast<const uint16_t *>(c.q_latent);
    a.q_rope = static_cast<const uint16_t *>(c.q_rope);
    a.q_latent_token = c.q_latent_token;
    a.q_latent_head = c.q_latent_head;
    a.q_rope_token = c.q_rope_token;
    a.q_rope_head = c.q_rope_head;
    a.main_cache = static_cast<const uint8_t *>(c.main_cache);
    a.num_blocks = c.num_blocks;
    a.block_table = c.block_table;
    a.table_stride = c.table_stride;
    a.max_blocks = c.max_blocks;
    a.seq_lens = c.seq_lens;
    a.query_start = c.query_start;
    a.tree_mask = c.tree_mask;
    a.num_tokens = c.num_tokens;
    a.num_seqs = static_cast<int>(c.num_seqs);
    a.num_heads = c.num_heads;
    a.max_query_len = c.max_query_len;
    a.softmax_scale = c.softmax_scale;
    a.invalid_count = c.invalid_count;
    *out = a;
    return KVPUB_OK;
}

// Launches a kernel with `bytes` of dynamic shared memory, in clusters of `cluster`.  The opt-in that
// this takes is made once a device, and again where a device reset undid it.
template <typename... KArgs, typename... Args>
kvpub_status launch_opted(const char *name, void (*kernel)(KArgs...), std::atomic<bool> *opted,
                          int cluster, int blocks, int threads, int bytes, cudaStream_t stream,
                          Args... args) {
    int dev = 0;
    kvpub_status st = current_device(&dev);
    if (st != KVPUB_OK) return st;
    (void)cudaGetLastError();
    bool known = opted[dev].load(std::memory_order_relaxed);
    for (;; known = false) {
        if (!known) {
            cudaError_t e = cudaFuncSetAttribute(
                (const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess)
                return fail(KVPUB_ERR_CUDA, "shared memory: %s", cudaGetErrorString(e));
            opted[dev].store(true, std::memory_order_relaxed);
        }
        cudaError_t e =
            launch_smem(kernel, dim3(blocks), threads, bytes, stream, cluster, args...);
        if (e != cudaErrorInvalidValue || !known) return launched(name);
        (void)cudaGetLastError();
    }
}

// How many clusters of 2, 4 or 8 blocks of a kernel fit the GPU at once (of blocks
// that take an SM each, 152 SMs hold 76, 36 and 15), asked for once a device.  `Kernel`
// is an argument of the template so that each kernel has its own answers.
template <auto Kernel>
kvpub_status clusters_at_once(int dev, int threads, int bytes, int (*out)[3]) {
    static std::atomic<int> cached[kMaxDevices][3];
    for (int i = 0; i < 3; ++i) {
        int n = cached[dev][i].load(std::memory_order_relaxed);
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = bytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2 << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            cudaError_t e = cudaFuncSetAttribute(
                (const void *)Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg);
            if (e != cudaSuccess)
                return fail(KVPUB_ERR_CUDA, "clusters: %s", cudaGetErrorString(e));
            cached[dev][i].store(n, std::memory_order_relaxed);
        }
        (*out)[i] = n;
    }
    return KVPUB_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline kvpub_status encode_tiled(EncodeTiled *out) {
    static std::atomic<EncodeTiled> cached{nullptr};
    EncodeTiled f = cached.load(std::memory_order_relaxed);
    if (f == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                         cudaEnableDefault, &found);
        if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || p == nullptr)
            return fail(KVPUB_ERR_CUDA, "cuTensorMapEncodeTiled: %s", cudaGetErrorString(e));
        f = reinterpret_cast<EncodeTiled>(p);
        cached.store(f, std::memory_order_relaxed);
    }
    *out = f;
    return KVPUB_OK;
}

// The cache as rows of 656 bytes: boxes of 64 slots by `width` bytes.
inline kvpub_status map_cache(const MlaArgs &a, int width, CUtensorMapSwizzle swizzle,
                       CUtensorMap *map) {
    EncodeTiled encode;
    kvpub_status st = encode_tiled(&encode);
    if (st != KVPUB_OK) return st;
    const cuuint64_t dims[2] = {KVPUB_MAIN_SLOT_BYTES,
                                static_cast<cuuint64_t>(a.num_blocks) * KVPUB_BLOCK_SIZE};
    const cuuint64_t strides[1] = {KVPUB_MAIN_SLOT_BYTES};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(width), KVPUB_BLOCK_SIZE};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                              const_cast<uint8_t *>(a.main_cache), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KVPUB_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
    return KVPUB_OK;
}

// Rows of a block: the fewest that hold a sequence's rows, at most 64.
inline int rows_for(int num_heads, int max_query_len) {
    const int rows = num_heads * max_query_len;
    return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}

}  // namespace kvpub
