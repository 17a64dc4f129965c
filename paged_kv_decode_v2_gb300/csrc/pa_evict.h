// pa_evict.h -- host-side interface of the operators that decide which tokens of a
// paged cache stay (accumulated attention weights, eviction), between their C entry
// points (pa_evict_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_decode.h"
#include "pa_internal.h"

namespace pa {

constexpr int kWeighAgain = 16;  // new tokens from which scores are computed twice, not kept
constexpr int kWeighTile = 1024; // tokens at most of a CTA that sums their weights over several row tiles
constexpr int kWeighParts = 128; // partitions of a sequence at most

struct WeighParams {
    const void *query;           // [S, q_len, H, D], f16 or bf16
    const void *key_cache;       // of the query's type, or e2m1 codes
    const uint8_t *k_scales;     // codes: [num_blocks, KV, block_size, D / 32]
    const int32_t *block_tables; // [S, max_blocks]
    const int32_t *seq_lens;     // [S]
    int dtype;
    int num_heads;
    int num_kv_heads;
    int group;
    int q_len;
    int cols;                    // G * q_len query rows per KV head
    int col_groups;              // CTAs that split them
    int num_blocks;
    int block_shift;             // log2 of the block size
    int max_blocks;
    int seq_len_cap;
    float scale;
    float decay;
    int part;                    // tokens of a CTA
    int num_parts;
    int num_seqs;
    int sorted;                  // units by size
    int tile;                    // scores computed twice: tokens of a CTA of the second pass
    int num_tiles;
    int tiles_sorted;
    uint32_t group_inv;          // ceil(2^32 / group), group > 1
    long long row_stride;        // tokens between rows of `scores`
    float *scores;               // [S, KV, cols, row_stride], log2 units
    float *maxima;               // [S, KV, cols, kWeighParts]
    float *sums;
    float *weights;              // [num_blocks, KV, block_size]
    int32_t *status;
};
// rows per CTA: 8, 16, 32 or 64; CTAs that registers let share an SM, and their threads.
int weigh_ctas(int rows);
int weigh_threads();
cudaError_t launch_weigh(int head_dim, int rows, const WeighParams &p, int dev, cudaStream_t stream);
// Scores computed twice (no `scores`), 128 rows per CTA (pa_weigh_tc.cu).
int weigh_tc_ctas(int head_dim);
int weigh_tc_threads();
cudaError_t launch_weigh_tc(int head_dim, const WeighParams &p, int dev, cudaStream_t stream);

struct EvictParams {
    void *key_cache, *value_cache;
    uint8_t *k_scales, *v_scales; // or null: 16-bit caches
    float *weights;               // [num_blocks, KV, block_size]
    const int32_t *block_tables;  // [S, max_blocks]
    const int32_t *seq_lens;      // [S]
    const int32_t *dst_tables;    // [S, dst_max_blocks]
    int32_t *kept;                // [S, KV, budget]
    int32_t *new_lens;            // [S]
    int num_seqs;
    int num_kv_heads;
    int row_bytes;                // of a token's keys (or values) in one head
    int scale_bytes;              // of its scales, 0 without
    int num_blocks;
    int block_shift;
    int max_blocks;
    int dst_max_blocks;
    int seq_len_cap;
    int budget, first, recent;
    int select_ways;              // CTAs of a cluster that choose one head's tokens
    int select_held;              // octets whose keys a CTA keeps
    int ways;                     // CTAs of a cluster that move its rows in place
    int32_t *status;
};
cudaError_t launch_evict(const EvictParams &p, int num_sms, int dev, cudaStream_t stream);

} // namespace pa
