// pa_q8.h -- host-side interface of the cache operators (appending to a paged
// cache, attention over an 8-bit cache) between their C entry points
// (pa_q8_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_decode.h"
#include "pa_internal.h"

namespace pa {

// Host helpers of pa_api.cu that the cache operators share with the 16-bit path.
int host_device(int *dev, int *sms);             // current device and its SM count
int host_check_q_len(int num_seqs, int q_len);
// Arguments of the queries for a call's variant and partition size.
int host_check_choose(int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_dim,
                      int max_seq_len, int partition_size);
int host_seq_cap(int max_blocks_per_seq, int block_size, int hint);
bool host_aligned(const void *p, uintptr_t a);
int host_encode_tiled(CUtensorMap *map, CUtensorMapDataType type, uint32_t rank, const void *base,
                      const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
                      CUtensorMapSwizzle swizzle);
void host_tuning(int *warps, int *stages, int *rows_kernel);
int host_merge(const int32_t *seq_lens, int num_seqs, int q_len, int num_heads, int head_dim,
               int max_seq_len, int partition_size, int dtype, const float *tmp_output,
               const float *exp_sums, const float *max_logits, int max_num_partitions, void *out,
               bool single_done, int32_t *status, cudaStream_t stream);

// The 16-bit multi-query attention over copies of K and V (partials at a stride
// of np partitions of `part` tokens, V1 when part is 0), bf16 with V's binary16
// copy as pa_decode_mq uses it (v_half; else v is a cache like k).  Where *flag is
// up the attention does nothing, and what `out` holds then is unspecified.
int host_mq_over_copy(const void *query, const void *k, const void *v, bool v_half,
                      const int32_t *flag, const int32_t *offs, const int32_t *table,
                      const int32_t *seq_lens, int num_seqs, int q_len, int num_heads,
                      int num_kv_heads, int head_dim, int num_blocks, int block_size,
                      int table_width, int cap, float scale, int part, int np, int dtype, void *out,
                      float *tmp_output, float *exp_sums, float *max_logits, int32_t *status,
                      cudaStream_t stream);
// Whether the two-tile kernel takes binary16 rows of these sizes.
bool host_two_tiles(int cols, int head_dim, int cap);
// pa_decode_mq's choice: the partition size of V2, 0 for V1, negative PA_ERR_*.
int host_mq_partition(int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_dim,
                      int max_seq_len, int partition_size);

// ---------------------------------------------------------------- append

// Arguments of both append kernels.  Token row t belongs to the sequence b
// with token_starts[b] <= t < token_starts[b + 1] (or b = t / q_len) and sits
// at position seq_lens[b] - token_starts[b + 1] + t.
struct AppendParams {
    const void *key;             // [num_tokens, KV, D], key_stride elements between tokens
    const void *value;
    const void *query;           // [num_tokens, H, D] or null
    void *query_out;
    long long key_stride, value_stride, query_stride, query_out_stride;
    const float *cos_sin;        // [max_positions, rotary_dim] (cosines, then sines), or null
    int rotary_dim;              // 0 without rotation
    int max_positions;
    int interleaved;
    const int32_t *block_tables; // [S, max_blocks]
    const int32_t *seq_lens;     // [S]
    const int32_t *token_starts; // [S + 1], or null: q_len tokens per sequence
    int num_tokens;
    int num_seqs;
    int q_len;                   // without token_starts
    int num_heads;               // 0 without a query
    int num_kv_heads;
    int head_dim;
    int num_blocks;
    int block_size;
    int max_blocks;
    void *key_cache;
    void *value_cache;
    float *k_scales;             // 8-bit cache: [num_blocks, KV]
    float *v_scales;
    int32_t *status;
};
cudaError_t launch_append(int dtype, const AppendParams &p, cudaStream_t stream);
cudaError_t launch_append_q8(int dtype, const AppendParams &p, int num_sms, cudaStream_t stream);
// CTAs launch_append_q8 needs (its grid is one-dimensional: at most 2^31 - 1).
long long append_q8_ctas(const AppendParams &p);

// ---------------------------------------------------------------- attention

// Arguments of the 8-bit attention kernels.
struct Q8Params {
    const void *query;           // [S, q_len, H, D], f16 or bf16
    const float *k_scales;       // [num_blocks, KV]
    const float *v_scales;
    const int32_t *block_tables; // [S, max_blocks]
    const int32_t *seq_lens;     // [S]
    int dtype;                   // of query and out
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
    int partition_size;          // V2, and V1 over a cluster: tokens of a CTA
    int num_seqs;
    int num_parts;               // V2: partitions per sequence
    uint32_t group_inv;          // ceil(2^32 / group), group > 1
    float class_scale;           // sorted: 32 classes over a whole unit's tokens
    int sorted;                  // units by size (at most kQ8Sorted sequences)
    int ways;                    // V1: CTAs of a cluster that share a row tile's tokens
    int stages;                  // K ring stages
    int v_stages;                // V ring stages
    int max_num_partitions;      // V2: partition capacity of the intermediates
    float *tmp_output;           // V2
    float *exp_sums;
    float *max_logits;
    void *out;                   // V1
    const int32_t *only_if;      // kQ8If: run only if this word is not 0,
    int units;                   // a CTA's share of so many
    int32_t *status;
};

// The 16-bit copy of a call's blocks (pa_q8_copy.cu).
struct Q8CopyParams {
    const void *key_cache, *value_cache;
    const float *k_scales, *v_scales;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    int num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks, seq_len_cap;
    int copy_blocks;             // blocks the copies hold: num_seqs * table_width
    int table_width;             // of the copies' block table
    int32_t *offs;               // [num_seqs + 1], the last the total
    int32_t *flag;
    int32_t *table;              // [num_seqs, table_width]
    void *k_copy, *v_copy;
    int32_t *status;
};
cudaError_t launch_q8_copy(int dtype, bool v_half, const Q8CopyParams &p, int num_sms,
                           cudaStream_t stream);

struct Q8Launch {
    Q8Params p;
    CUtensorMap tmap_k;
    CUtensorMap tmap_v;
    int head_dim;
    int block_size;
    int mode;                    // kQ8V2, ..
    dim3 grid;
    size_t smem_bytes;
};

// The tcgen05 kernels: one per (head_dim, rows per CTA), see pa_q8_tc.cuh.
constexpr int kQ8Tok = 128; // tokens per tile
constexpr int kQ8Sorted = 256; // sequences that a CTA's threads sort
constexpr int kQ8Ways = 8;  // CTAs of a cluster at most (the portable size)
enum { kQ8V2, kQ8V1, kQ8If }; // kQ8If: V1 if a flag is up, any grid
struct Q8TcKernel {
    const void *fn;
    int threads;
    int ctas;                // that share an SM
    size_t fixed_bytes;      // dynamic shared memory but for the rings
};
// rows 8, 16, 32, or (up to head_dim 128) 64; fn null otherwise.
Q8TcKernel q8_tc_d64(int rows, int dtype, int mode);
Q8TcKernel q8_tc_d128(int rows, int dtype, int mode);
Q8TcKernel q8_tc_d256(int rows, int dtype, int mode);

inline Q8TcKernel q8_tc(int head_dim, int rows, int dtype, int mode)
{
    return head_dim == 64    ? q8_tc_d64(rows, dtype, mode)
           : head_dim == 128 ? q8_tc_d128(rows, dtype, mode)
                             : q8_tc_d256(rows, dtype, mode);
}

} // namespace pa
