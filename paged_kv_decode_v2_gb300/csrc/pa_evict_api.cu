// pa_evict_api.cu -- C entry points of pa_kv_weights, pa_kv_weights_q4 and pa_kv_evict,
// declared in include/pa_decode.h.  Host-side validation, workspace layout and sizing.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pa_decode.h"
#include "pa_evict.h"
#include "pa_q4.h"

using namespace pa;

namespace {

int shift_of(int block_size) { return block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6; }

// Floats of a row's scores: whole 128-byte lines, or none where they are not kept.
int64_t score_stride(int q_len, int max_seq_len)
{
    return q_len >= kWeighAgain ? 0 : ((int64_t)max_seq_len + 31) / 32 * 32;
}

int weigh_impl(const void *query, const void *key_cache, const uint8_t *k_scales, bool q4, const int32_t *block_tables,
               const int32_t *seq_lens, int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_dim,
               int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len_hint, float scale, float decay,
               int dtype, float *weights, void *workspace, size_t workspace_bytes, int32_t *status,
               cudaStream_t stream)
{
    int rc = check_cache(key_cache, key_cache, block_tables, seq_lens, num_seqs, num_kv_heads, head_dim, num_blocks,
                         block_size, max_blocks_per_seq, dtype, status);
    if (rc)
        return rc;
    if (!query || !weights || !workspace || num_heads <= 0 || num_heads % num_kv_heads != 0 || !std::isfinite(scale) ||
        !std::isfinite(decay) || (q4 && (!k_scales || !host_aligned(k_scales, 16))))
        return PA_ERR_INVALID_ARG;
    if (!host_aligned(query, 4) || !host_aligned(weights, 16) || !host_aligned(workspace, 16))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (group > kMaxGQA || num_heads > 65535 || (int64_t)max_blocks_per_seq * block_size > INT32_MAX - 65536)
        return PA_ERR_UNSUPPORTED;
    rc = host_check_q_len(num_seqs, q_len);
    if (rc)
        return rc;
    const int cap = host_seq_cap(max_blocks_per_seq, block_size, max_seq_len_hint);
    const size_t need = pa_kv_weights_workspace_bytes(num_seqs, q_len, num_heads, cap);
    if (need == 0)
        return PA_ERR_UNSUPPORTED;
    if (workspace_bytes < need)
        return PA_ERR_WORKSPACE;
    int dev, sms;
    if (host_device(&dev, &sms))
        return PA_ERR_CUDA;
    WeighParams p = {};
    p.query = query;
    p.key_cache = key_cache;
    p.k_scales = k_scales;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.dtype = dtype;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.group_inv = group > 1 ? (uint32_t)(((1ull << 32) + group - 1) / group) : 0;
    p.q_len = q_len;
    p.cols = group * q_len;
    const bool again = q_len >= kWeighAgain;
    const int rows = again ? 128 : p.cols <= 8 ? 8 : p.cols <= 16 ? 16 : p.cols <= 32 ? 32 : 64;
    p.col_groups = (p.cols + rows - 1) / rows;
    p.num_blocks = num_blocks;
    p.block_shift = shift_of(block_size);
    p.max_blocks = max_blocks_per_seq;
    p.seq_len_cap = cap;
    p.scale = scale;
    p.decay = decay;
    // Two waves of CTAs where they are short, of 256 tokens at least; one where each has
    // many rows to prepare.  Waves by registers, although shared memory holds fewer CTAs over
    // 16-bit keys: cut by those, 32 rows of 16 sequences of head_dim 256 take 89 us for 77, 60 rows
    // of 8 sequences 93 for 73, 4 rows of 32 sequences of 128 dims 66 for 65, and only one of
    // 100,000 tokens of 256 dims gains (49 for 51).  Nor does sorting by them change a time.
    const long long groups = (long long)num_seqs * num_kv_heads * p.col_groups;
    const long long slots = (long long)sms * (again ? weigh_tc_ctas(head_dim) : weigh_ctas(rows));
    const int threads = again ? weigh_tc_threads() : weigh_threads();
    const long long most = again ? slots / groups : ((rows <= 16 ? 2 : 1) * slots + groups - 1) / groups;
    const long long parts = std::max(1LL, std::min({most, (cap + 255LL) / 256, (long long)kWeighParts}));
    p.part = (int)(((cap + parts - 1) / parts + 127) / 128 * 128);
    p.num_parts = (int)((cap + (long long)p.part - 1) / p.part);
    p.num_seqs = num_seqs;
    p.sorted = num_seqs > 1 && num_seqs <= threads && groups * p.num_parts > slots;
    const long long heads = (long long)num_seqs * num_kv_heads;
    const long long per = std::max(1LL, slots / heads); // CTAs of a second pass, likewise
    p.tile = (int)std::max(128LL, ((cap + per - 1) / per + 127) / 128 * 128);
    if (p.col_groups > 1)
        p.tile = std::min(p.tile, kWeighTile);
    p.num_tiles = (int)((cap + (long long)p.tile - 1) / p.tile);
    p.tiles_sorted = num_seqs > 1 && num_seqs <= threads && heads * p.num_tiles > slots;
    p.status = status;
    p.row_stride = score_stride(q_len, cap);
    const size_t total = (size_t)num_seqs * num_heads * q_len;
    p.scores = static_cast<float *>(workspace);
    p.maxima = p.scores + total * p.row_stride;
    p.sums = p.maxima + total * kWeighParts;
    p.weights = weights;
    const long long tiles = (cap + 127LL) / 128; // of a second pass at most
    if (cap == 0)
        return PA_OK;
    if (groups * p.num_parts > INT32_MAX || (long long)num_seqs * num_kv_heads * tiles > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    return (again ? launch_weigh_tc(head_dim, p, dev, stream) : launch_weigh(head_dim, rows, p, dev, stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

} // namespace

extern "C" {

PA_API size_t pa_kv_weights_workspace_bytes(int num_seqs, int q_len, int num_heads, int max_seq_len)
{
    if (num_seqs <= 0 || q_len <= 0 || num_heads <= 0 || max_seq_len < 0 || host_check_q_len(num_seqs, q_len))
        return 0;
    const unsigned __int128 bytes = (unsigned __int128)num_seqs * q_len * num_heads *
                                    (uint64_t)(score_stride(q_len, max_seq_len) + 2 * kWeighParts) * 4;
    return bytes > (unsigned __int128)INT64_MAX ? 0 : (size_t)bytes;
}

PA_API int pa_kv_weights(const void *query, const void *key_cache, const int32_t *block_tables,
                         const int32_t *seq_lens, int num_seqs, int q_len, int num_heads, int num_kv_heads,
                         int head_dim, int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len_hint,
                         float scale, float decay, int dtype, float *weights, void *workspace, size_t workspace_bytes,
                         int32_t *status, pa_stream_t stream)
{
    return weigh_impl(query, key_cache, nullptr, false, block_tables, seq_lens, num_seqs, q_len, num_heads,
                      num_kv_heads, head_dim, num_blocks, block_size, max_blocks_per_seq, max_seq_len_hint, scale,
                      decay, dtype, weights, workspace, workspace_bytes, status, (cudaStream_t)stream);
}

PA_API int pa_kv_weights_q4(const void *query, const void *key_cache, const uint8_t *k_scales,
                            const int32_t *block_tables, const int32_t *seq_lens, int num_seqs, int q_len,
                            int num_heads, int num_kv_heads, int head_dim, int num_blocks, int block_size,
                            int max_blocks_per_seq, int max_seq_len_hint, float scale, float decay, int dtype,
                            float *weights, void *workspace, size_t workspace_bytes, int32_t *status,
                            pa_stream_t stream)
{
    return weigh_impl(query, key_cache, k_scales, true, block_tables, seq_lens, num_seqs, q_len, num_heads,
                      num_kv_heads, head_dim, num_blocks, block_size, max_blocks_per_seq, max_seq_len_hint, scale,
                      decay, dtype, weights, workspace, workspace_bytes, status, (cudaStream_t)stream);
}

PA_API int pa_kv_evict(void *key_cache, void *value_cache, uint8_t *k_scales, uint8_t *v_scales, float *weights,
                       const int32_t *block_tables, const int32_t *seq_lens, int num_seqs, int num_kv_heads,
                       int head_dim, int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len_hint,
                       int budget, int first, int recent, const int32_t *dst_tables, int dst_max_blocks,
                       int32_t *kept, int32_t *new_lens, int32_t *status, pa_stream_t stream)
{
    const int rc = check_cache(key_cache, value_cache, block_tables, seq_lens, num_seqs, num_kv_heads, head_dim,
                               num_blocks, block_size, max_blocks_per_seq, PA_F16, status);
    if (rc)
        return rc;
    if (!weights || !dst_tables || !kept || !new_lens || (k_scales != nullptr) != (v_scales != nullptr) ||
        budget <= 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget || dst_max_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!host_aligned(weights, 16) || !host_aligned(dst_tables, 4) || !host_aligned(kept, 4) ||
        !host_aligned(new_lens, 4) || (k_scales && (!host_aligned(k_scales, 16) || !host_aligned(v_scales, 16))))
        return PA_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX - 65536)
        return PA_ERR_UNSUPPORTED;
    const int cap = host_seq_cap(max_blocks_per_seq, block_size, max_seq_len_hint);
    // The tokens that stay have to fit their blocks.
    if ((int64_t)dst_max_blocks * block_size < std::min(budget, cap))
        return PA_ERR_INVALID_ARG;
    if (dst_tables == block_tables && dst_max_blocks != max_blocks_per_seq)
        return PA_ERR_INVALID_ARG;
    int dev, sms;
    if (host_device(&dev, &sms))
        return PA_ERR_CUDA;
    EvictParams p = {};
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.weights = weights;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.dst_tables = dst_tables;
    p.kept = kept;
    p.new_lens = new_lens;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.row_bytes = k_scales ? head_dim / 2 : head_dim * 2;
    p.scale_bytes = k_scales ? head_dim / 32 : 0;
    p.num_blocks = num_blocks;
    p.block_shift = shift_of(block_size);
    p.max_blocks = max_blocks_per_seq;
    p.dst_max_blocks = dst_max_blocks;
    p.seq_len_cap = cap;
    p.budget = budget;
    p.first = first;
    p.recent = recent;
    p.status = status;
    // CTAs: a stretch of at least 16 rows each.
    if ((long long)num_seqs * num_kv_heads * ((std::min(budget, cap) + 15LL) / 16 + 8) > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    return launch_evict(p, sms, dev, (cudaStream_t)stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
