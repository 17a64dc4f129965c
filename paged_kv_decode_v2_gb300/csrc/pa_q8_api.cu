// pa_q8_api.cu -- C entry points of the cache operators declared in
// include/pa_decode.h: appending to a paged cache (16-bit or 8-bit) and
// attention over an 8-bit cache.  Host-side validation, TMA descriptors,
// launch sizing and dispatch.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "pa_decode.h"
#include "pa_q8.h"

using namespace pa;

namespace {

constexpr int kMaxDevices = 64;
// ---- tcgen05 kernels

int rows_per_cta(int cols, int head_dim)
{
    if (cols <= 8)
        return 8;
    if (cols <= 16)
        return 16;
    return cols <= 32 || head_dim == 256 ? 32 : 64;
}

// CTAs of the kernel that share an SM, the same for both types.
int ctas_per_sm(int nr, int head_dim) { return q8_tc(head_dim, nr, PA_F16, kQ8V2).ctas; }

std::atomic<int64_t> g_tc_limit[kMaxDevices][3 * 4 * 2 * 3];

int launch_tc(Q8Launch &L, int dev, int nr, cudaStream_t stream)
{
    const Q8TcKernel k = q8_tc(L.head_dim, nr, L.p.dtype, L.mode);
    if (!k.fn)
        return PA_ERR_UNSUPPORTED;
    const int di = L.head_dim == 64 ? 0 : L.head_dim == 128 ? 1 : 2;
    const int ri = nr == 8 ? 0 : nr == 16 ? 1 : nr == 32 ? 2 : 3;
    std::atomic<int64_t> &cell =
        g_tc_limit[dev][((di * 4 + ri) * 2 + (L.p.dtype == PA_BF16 ? 1 : 0)) * 3 + L.mode];
    // Dynamic limit after the opt-in in the low half, static bytes above.
    int64_t have = cell.load(std::memory_order_acquire);
    if (have == 0) {
        int optin = 0;
        cudaFuncAttributes fa;
        if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
            cudaFuncGetAttributes(&fa, k.fn) != cudaSuccess || (size_t)optin <= fa.sharedSizeBytes)
            return PA_ERR_CUDA;
        const int dyn = optin - (int)fa.sharedSizeBytes;
        if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn) != cudaSuccess)
            return PA_ERR_CUDA;
        have = dyn | (int64_t)fa.sharedSizeBytes << 32;
        cell.store(have, std::memory_order_release);
    }
    const size_t limit = have & 0xffffffff, fixed_static = have >> 32;
    const size_t tile = (size_t)kQ8Tok * L.head_dim;
    int tune_w, tune_s, rows_kernel;
    host_tuning(&tune_w, &tune_s, &rows_kernel);
    // As many CTAs per SM as the kernel is made for, if rings of two stages fit.
    const size_t sm = limit + fixed_static + 1024; // a CTA also takes 1 KB for the system
    size_t per_cta = limit;
    for (int n = k.ctas; n > 1; --n) {
        if (k.fixed_bytes + 4 * tile + fixed_static + 1024 <= sm / n) {
            per_cta = sm / n - 1024 - fixed_static;
            break;
        }
    }
    int ks = 1, vs = 1;
    while (k.fixed_bytes + (ks + vs + 1) * tile <= per_cta && ks + vs < 2 * kMaxStages) {
        if (ks > vs)
            ++vs;
        else
            ++ks;
    }
    if (tune_s > 0)
        ks = vs = tune_s;
    if (tune_w > 0)
        vs = tune_w;
    while (k.fixed_bytes + (ks + vs) * tile > limit && (ks > 1 || vs > 1)) {
        if (ks >= vs)
            --ks;
        else
            --vs;
    }
    L.smem_bytes = k.fixed_bytes + (ks + vs) * tile;
    if (L.smem_bytes > limit)
        return PA_ERR_UNSUPPORTED;
    L.p.stages = ks;
    L.p.v_stages = vs;
    void *args[] = {&L.tmap_k, &L.tmap_v, &L.p};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = L.grid;
    cfg.blockDim = dim3(k.threads);
    cfg.dynamicSmemBytes = L.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)L.p.ways;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.mode == kQ8V1 && L.p.ways > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, k.fn, args) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// 3-D view of an 8-bit cache for the TMA: dims {row bytes of a slice (64 or
// 128), slices, rows = num_blocks * KV * block_size}, swizzled by that width,
// box {slice, 1, block_size}.
int encode_q8_map(CUtensorMap *map, const void *base, int num_blocks, int num_kv_heads,
                  int block_size, int head_dim)
{
    const uint64_t width = head_dim < 128 ? head_dim : 128;
    const uint64_t rows = (uint64_t)num_blocks * num_kv_heads * block_size;
    const uint64_t dims[3] = {width, head_dim / width, rows};
    const uint64_t strides[2] = {width, (uint64_t)head_dim};
    const uint32_t box[3] = {(uint32_t)width, 1, (uint32_t)block_size};
    return host_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box,
                             width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Shape checks shared by the cache operators.  No CUDA call.
int check_cache(const void *key_cache, const void *value_cache, const int32_t *block_tables,
                const int32_t *seq_lens, int num_seqs, int num_kv_heads, int head_dim,
                int num_blocks, int block_size, int max_blocks_per_seq, int dtype,
                const int32_t *status)
{
    if (!key_cache || !value_cache || !block_tables || !seq_lens)
        return PA_ERR_INVALID_ARG;
    if (num_seqs <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0 ||
        max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_F16 && dtype != PA_BF16)
        return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    // TMA row coordinates and token indices are 32-bit.
    if ((int64_t)num_blocks * num_kv_heads * block_size > INT32_MAX ||
        (int64_t)max_blocks_per_seq * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (!host_aligned(key_cache, 16) || !host_aligned(value_cache, 16) ||
        !host_aligned(block_tables, 4) || !host_aligned(seq_lens, 4) ||
        (status && !host_aligned(status, 4)))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

// A strided [num_tokens, heads, head_dim] operand: 16-byte aligned rows that do not overlap.
bool rows_ok(const void *base, int64_t stride, int heads, int head_dim, int num_tokens)
{
    return base && host_aligned(base, 16) && stride % 8 == 0 &&
           (num_tokens <= 1 || stride >= (int64_t)heads * head_dim);
}

int append_impl(const void *key, const void *value, int64_t key_stride, int64_t value_stride,
                const void *query, void *query_out, int64_t query_stride, int64_t query_out_stride,
                const float *cos_sin, int rotary_dim, int max_positions, int interleaved,
                const int32_t *block_tables, const int32_t *seq_lens, const int32_t *token_starts,
                int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                int num_blocks, int block_size, int max_blocks_per_seq, int dtype, void *key_cache,
                void *value_cache, float *k_scales, float *v_scales, bool q8, int32_t *status,
                cudaStream_t stream)
{
    int rc = check_cache(key_cache, value_cache, block_tables, seq_lens, num_seqs, num_kv_heads,
                         head_dim, num_blocks, block_size, max_blocks_per_seq, dtype, status);
    if (rc)
        return rc;
    if (num_tokens < 0 || (query != nullptr) != (query_out != nullptr))
        return PA_ERR_INVALID_ARG;
    if (token_starts ? !host_aligned(token_starts, 4) : num_tokens % num_seqs != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!rows_ok(key, key_stride, num_kv_heads, head_dim, num_tokens) ||
                           !rows_ok(value, value_stride, num_kv_heads, head_dim, num_tokens)))
        return PA_ERR_INVALID_ARG;
    if (query && (num_heads <= 0 || num_heads % num_kv_heads != 0))
        return PA_ERR_INVALID_ARG;
    if (query && num_tokens > 0 &&
        (!rows_ok(query, query_stride, num_heads, head_dim, num_tokens) ||
         !rows_ok(query_out, query_out_stride, num_heads, head_dim, num_tokens)))
        return PA_ERR_INVALID_ARG;
    if (q8 && (!k_scales || !v_scales || !host_aligned(k_scales, 4) || !host_aligned(v_scales, 4)))
        return PA_ERR_INVALID_ARG;
    if (cos_sin) {
        if (!host_aligned(cos_sin, 16) || rotary_dim <= 0 || max_positions <= 0)
            return PA_ERR_INVALID_ARG;
        if (rotary_dim % 16 != 0 || rotary_dim > head_dim)
            return PA_ERR_UNSUPPORTED;
    }
    if (query && num_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    AppendParams p = {};
    p.key = key;
    p.value = value;
    p.query = query;
    p.query_out = query_out;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.query_stride = query_stride;
    p.query_out_stride = query_out_stride;
    p.cos_sin = cos_sin;
    p.rotary_dim = cos_sin ? rotary_dim : 0;
    p.max_positions = max_positions;
    p.interleaved = interleaved != 0;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.token_starts = token_starts;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.q_len = token_starts ? 0 : num_tokens / num_seqs;
    p.num_heads = query ? num_heads : 0;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks = max_blocks_per_seq;
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.status = status;
    if (num_tokens == 0)
        return PA_OK;
    if (q8 && append_q8_ctas(p) > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    int dev, sms;
    if (host_device(&dev, &sms))
        return PA_ERR_CUDA;
    const cudaError_t e =
        q8 ? launch_append_q8(dtype, p, sms, stream) : launch_append(dtype, p, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// CTAs that split the query rows of one KV head.
int row_groups(int cols, int head_dim)
{
    const int nr = rows_per_cta(cols, head_dim);
    return (cols + nr - 1) / nr;
}

// How a call is cut: V2 at `part` tokens, or V1 (part 0) with a cluster of `ways` CTAs
// per group (sequence, KV head, row tile), `per` tokens each.
struct Q8Cut {
    int part, ways, per;
};

// A CTA costs some 5 us beside its tiles, so partitions are long.  One wave of CTAs
// (as many partitions per group as give every place a CTA) if that takes at most
// kWavePart tokens each: one sequence of 100,000 tokens, 4 KV heads: 1408 tokens 21.4
// us, 2048 22.7, 1024 27.2.  Else two waves or more, sorted by size (see the kernel),
// the fewest whose partitions have at most kMaxPart tokens: 32 sequences of up to 8192,
// 8 KV heads: 4096 52 us, 2048 54, 8192 59; 64 of up to 32,768: 8192 74 us, 4096 84,
// 16,384 112; 16 new tokens for 32 of up to 8192: 8192 89 us, 4096 98.
constexpr int kWavePart = 2048, kMaxPart = 8192;
// V1 unless a CTA of its cluster has more tiles than a partition by more than this:
// what the second launch costs (8 groups of 8000 tokens: V2 10.5 us at 4 tiles, V1
// 12.9 at 8; of 4000 tokens both 4 tiles, 9.9 us in either).
constexpr int kJoinTiles = 2;

Q8Cut choose_cut(int num_seqs, int q_len, int group, int num_kv_heads, int head_dim, int max_seq_len,
                 int partition_size, int sms)
{
    const int nr = rows_per_cta(q_len * group, head_dim);
    const long long groups = (long long)num_seqs * num_kv_heads * row_groups(q_len * group, head_dim);
    const long long tiles = ((long long)max_seq_len + kQ8Tok - 1) / kQ8Tok;
    const long long slots = (long long)sms * ctas_per_sm(nr, head_dim);
    Q8Cut cut = {0, 1, 0};
    if (tiles <= 1)
        return cut;
    // Clusters lie inside the GPU's groups of SMs, whose remainders stay empty: of 152
    // SMs with a CTA each, 15 clusters of 8 run at a time, 36 of 4, 76 of 2 (of 3, 5, 6
    // and 7: 46, 28, 23, 15).  48 groups of 4768 tokens (64 rows, fp16) took two waves
    // and 72 us as clusters of 3, 44 as partitions.
    static_assert(kQ8Ways == 8, "the sizes tried");
    const long long most = 8 * groups <= sms * 3 / 4 ? 8 : 4 * groups <= sms * 9 / 10 ? 4 : 2 * groups <= sms ? 2 : 1;
    const long long ways = std::min(most, tiles);
    const long long per = (tiles + ways - 1) / ways;
    cut.ways = (int)((tiles + per - 1) / per);
    cut.per = (int)std::min(per * kQ8Tok, (long long)INT32_MAX);
    auto in_waves = [&](long long k) { // tokens of a partition, k waves
        const long long np = std::max(1LL, k * slots / groups);
        return (tiles + np - 1) / np * kQ8Tok;
    };
    long long part = in_waves(1);
    if (part > kWavePart) {
        part = in_waves(2);
        if (part > kMaxPart) {
            const long long np = (max_seq_len + kMaxPart - 1LL) / kMaxPart; // at least
            part = in_waves((np * groups + slots - 1) / slots);
        }
    }
    part = std::max(part, (long long)partition_size);
    if (part < max_seq_len && per > (part + kQ8Tok - 1) / kQ8Tok + kJoinTiles)
        cut.part = (int)part;
    return cut;
}

// ---- the 16-bit copy for many rows

// From this many query rows per KV head on, the call makes a 16-bit copy of its
// blocks and runs the 16-bit kernels over it, if the intermediates have room (plan_copy;
// sized for partition_size, from about that many rows on) and its scales let the copy be
// exact.  8 KV heads, copy / 8-bit kernel, us: 2 sequences of 9000 tokens 128 rows 56 / 52,
// 256 rows 67 / 82, 1024 rows 116 / 259; 16 of 2000 86 / 76, 99 / 146, 238 / 489.  Where a
// scale is no power of two both run, the copy's attention for nothing but its launch: 2
// sequences of 9216 tokens, 4096 rows 328 -> 829 (fp16 319 -> 1119).
constexpr int kQ8CopyRows = 256;
// And from this many tiles of 128 tokens by 64 rows on: one sequence of 4000 tokens, 256
// rows (992 tiles) 32 / 27, 512 rows (1984) 42 / 40, 2048 rows (7936) 60 / 114; 20,000
// tokens on one KV head, 512 rows (1256) 36 / 30; 4 of 600, 512 rows (1280) 31 / 36.
constexpr long long kQ8CopyTiles = 2048;

struct CopyPlan {
    bool v_half;  // V in binary16 beside a bf16 K, for the two-tile kernel
    int part, np; // pa_decode_mq's choice
};

// Lays the copy out in tmp_output behind the partials the 16-bit call writes
// (256-byte boundaries): the offsets, total and flag, the block table, K, V.
// False when the worst case's blocks do not fit.
bool plan_copy(CopyPlan &plan, Q8CopyParams &c, const Q8Params &p, int partition_size, int num_seqs,
               int block_size, int head_dim)
{
    plan.part = host_mq_partition(num_seqs, p.q_len, p.num_heads, p.num_kv_heads, head_dim,
                                  p.seq_len_cap, partition_size);
    if (plan.part < 0)
        return false;
    plan.np = plan.part ? pa_v2_num_partitions(p.seq_len_cap, plan.part) : 0;
    if (plan.np > p.max_num_partitions)
        return false;
    plan.v_half = p.dtype == PA_BF16 && host_two_tiles(p.cols, head_dim, p.seq_len_cap);
    const long long width = ((long long)p.seq_len_cap + block_size - 1) / block_size;
    const long long blocks = width * num_seqs;
    const long long rows = (long long)p.num_kv_heads * block_size;
    if (width <= 0 || blocks > INT32_MAX / rows)
        return false;
    auto round256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t part_bytes = (size_t)num_seqs * p.q_len * p.num_heads * head_dim * 4;
    const size_t block_bytes = (size_t)rows * head_dim * 2;
    const size_t offs = round256(part_bytes * plan.np);
    const size_t table = offs + round256((size_t)(num_seqs + 2) * 4);
    const size_t k = table + round256((size_t)blocks * 4);
    const size_t v = k + round256((size_t)blocks * block_bytes);
    if (v + (size_t)blocks * block_bytes > part_bytes * p.max_num_partitions)
        return false;
    char *base = reinterpret_cast<char *>(p.tmp_output);
    c.k_scales = p.k_scales;
    c.v_scales = p.v_scales;
    c.block_tables = p.block_tables;
    c.seq_lens = p.seq_lens;
    c.num_seqs = num_seqs;
    c.num_kv_heads = p.num_kv_heads;
    c.head_dim = head_dim;
    c.block_size = block_size;
    c.num_blocks = p.num_blocks;
    c.max_blocks = p.max_blocks;
    c.seq_len_cap = p.seq_len_cap;
    c.copy_blocks = (int)blocks;
    c.table_width = (int)width;
    c.offs = reinterpret_cast<int32_t *>(base + offs);
    c.flag = c.offs + num_seqs + 1;
    c.table = reinterpret_cast<int32_t *>(base + table);
    c.k_copy = base + k;
    c.v_copy = base + v;
    c.status = p.status;
    return true;
}

} // namespace

extern "C" {

PA_API int pa_kv_append(const void *key, const void *value, int64_t key_stride,
                        int64_t value_stride, const void *query, void *query_out,
                        int64_t query_stride, int64_t query_out_stride, const float *cos_sin,
                        int rotary_dim, int max_positions, int interleaved,
                        const int32_t *block_tables, const int32_t *seq_lens,
                        const int32_t *token_starts, int num_tokens, int num_seqs, int num_heads,
                        int num_kv_heads, int head_dim, int num_blocks, int block_size,
                        int max_blocks_per_seq, int dtype, void *key_cache, void *value_cache,
                        int32_t *status, pa_stream_t stream)
{
    return append_impl(key, value, key_stride, value_stride, query, query_out, query_stride,
                       query_out_stride, cos_sin, rotary_dim, max_positions, interleaved,
                       block_tables, seq_lens, token_starts, num_tokens, num_seqs, num_heads,
                       num_kv_heads, head_dim, num_blocks, block_size, max_blocks_per_seq, dtype,
                       key_cache, value_cache, nullptr, nullptr, false, status,
                       (cudaStream_t)stream);
}

PA_API int pa_kv_append_q8(const void *key, const void *value, int64_t key_stride,
                           int64_t value_stride, const void *query, void *query_out,
                           int64_t query_stride, int64_t query_out_stride, const float *cos_sin,
                           int rotary_dim, int max_positions, int interleaved,
                           const int32_t *block_tables, const int32_t *seq_lens,
                           const int32_t *token_starts, int num_tokens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_dim, int num_blocks, int block_size,
                           int max_blocks_per_seq, int dtype, void *key_cache, void *value_cache,
                           float *k_scales, float *v_scales, int32_t *status, pa_stream_t stream)
{
    return append_impl(key, value, key_stride, value_stride, query, query_out, query_stride,
                       query_out_stride, cos_sin, rotary_dim, max_positions, interleaved,
                       block_tables, seq_lens, token_starts, num_tokens, num_seqs, num_heads,
                       num_kv_heads, head_dim, num_blocks, block_size, max_blocks_per_seq, dtype,
                       key_cache, value_cache, k_scales, v_scales, true, status,
                       (cudaStream_t)stream);
}

PA_API int pa_decode_q8_partition(int num_seqs, int q_len, int num_heads, int num_kv_heads,
                                  int head_dim, int max_seq_len, int partition_size)
{
    const int rc = host_check_choose(num_seqs, q_len, num_heads, num_kv_heads, head_dim, max_seq_len,
                                     partition_size);
    if (rc)
        return -rc;
    int dev, sms;
    if (host_device(&dev, &sms))
        return -PA_ERR_CUDA;
    return choose_cut(num_seqs, q_len, num_heads / num_kv_heads, num_kv_heads, head_dim, max_seq_len,
                      partition_size, sms)
        .part;
}

PA_API int pa_decode_q8(const void *query, const void *key_cache, const void *value_cache,
                        const float *k_scales, const float *v_scales, const int32_t *block_tables,
                        const int32_t *seq_lens, int num_seqs, int q_len, int num_heads,
                        int num_kv_heads, int head_dim, int num_blocks, int block_size,
                        int max_blocks_per_seq, int max_seq_len_hint, float scale,
                        int partition_size, int dtype, void *out, float *tmp_output,
                        float *exp_sums, float *max_logits, int max_num_partitions,
                        int32_t *status, pa_stream_t stream)
{
    int rc = check_cache(key_cache, value_cache, block_tables, seq_lens, num_seqs, num_kv_heads,
                         head_dim, num_blocks, block_size, max_blocks_per_seq, dtype, status);
    if (rc)
        return rc;
    if (!query || !k_scales || !v_scales || !out || num_heads <= 0 ||
        num_heads % num_kv_heads != 0 || partition_size <= 0 || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!host_aligned(query, 4) || !host_aligned(out, 4) || !host_aligned(k_scales, 4) ||
        !host_aligned(v_scales, 4))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (group > kMaxGQA || num_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    rc = host_check_q_len(num_seqs, q_len);
    if (rc)
        return rc;
    int dev, sms;
    if (host_device(&dev, &sms))
        return PA_ERR_CUDA;
    const cudaStream_t st = (cudaStream_t)stream;
    const int cap = host_seq_cap(max_blocks_per_seq, block_size, max_seq_len_hint);
    const bool work_ok = tmp_output && exp_sums && max_logits && max_num_partitions > 0 &&
                         host_aligned(tmp_output, 16) && host_aligned(exp_sums, 4) &&
                         host_aligned(max_logits, 4);
    const Q8Cut cut =
        choose_cut(num_seqs, q_len, group, num_kv_heads, head_dim, cap, partition_size, sms);
    const int part = cut.part;
    const int np = part ? pa_v2_num_partitions(cap, part) : 1;
    if (part && !work_ok)
        return PA_ERR_INVALID_ARG;
    if (part && np > max_num_partitions)
        return PA_ERR_WORKSPACE;

    Q8Launch L = {};
    rc = encode_q8_map(&L.tmap_k, key_cache, num_blocks, num_kv_heads, block_size, head_dim);
    if (rc)
        return rc;
    rc = encode_q8_map(&L.tmap_v, value_cache, num_blocks, num_kv_heads, block_size, head_dim);
    if (rc)
        return rc;
    Q8Params &p = L.p;
    p.query = query;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.dtype = dtype;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.group_inv = group > 1 ? (uint32_t)(((1ull << 32) + group - 1) / group) : 0;
    p.q_len = q_len;
    p.cols = group * q_len;
    p.col_groups = row_groups(p.cols, head_dim);
    p.num_blocks = num_blocks;
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    p.max_blocks = max_blocks_per_seq;
    p.seq_len_cap = cap;
    p.scale = scale;
    p.partition_size = part ? part : cut.per;
    p.ways = part ? 1 : cut.ways;
    p.max_num_partitions = max_num_partitions;
    p.tmp_output = tmp_output;
    p.exp_sums = exp_sums;
    p.max_logits = max_logits;
    p.out = out;
    p.status = status;
    L.head_dim = head_dim;
    L.block_size = block_size;
    L.mode = part == 0 ? kQ8V1 : kQ8V2;

    if (work_ok && p.cols >= kQ8CopyRows &&
        (long long)num_seqs * num_kv_heads * ((p.cols + 63) / 64) * ((cap + 127LL) / 128) >= kQ8CopyTiles) {
        Q8CopyParams c = {};
        CopyPlan plan;
        if (plan_copy(plan, c, p, partition_size, num_seqs, block_size, head_dim)) {
            c.key_cache = key_cache;
            c.value_cache = value_cache;
            if (launch_q8_copy(dtype, plan.v_half, c, sms, st) != cudaSuccess)
                return PA_ERR_CUDA;
            rc = host_mq_over_copy(query, c.k_copy, c.v_copy, plan.v_half, c.flag, c.offs, c.table,
                                   seq_lens, num_seqs, q_len, num_heads, num_kv_heads, head_dim,
                                   c.copy_blocks, block_size, c.table_width, cap, scale, plan.part,
                                   plan.np, dtype, out, tmp_output, exp_sums, max_logits, status, st);
            if (rc)
                return rc;
            // Values that 16 bits do not hold exactly: the kernels above have left at once,
            // and the 8-bit one runs after all (V1, which needs no intermediates).
            p.only_if = c.flag;
            L.mode = kQ8If;
            p.ways = 1;
        }
    }
    const long long gx = (long long)num_seqs * num_kv_heads * p.col_groups * (L.mode == kQ8V2 ? np : p.ways);
    if (gx > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    p.units = (int)gx;
    L.grid = dim3((unsigned)(L.mode == kQ8If ? std::min(gx, (long long)sms) : gx));
    // By size where CTAs wait for their turn (the sort costs each some 0.4 us).
    p.num_seqs = num_seqs;
    p.num_parts = np;
    p.class_scale = 32.f / (float)(L.mode == kQ8V2 ? part : cap);
    p.sorted = L.mode != kQ8If && num_seqs > 1 && num_seqs <= kQ8Sorted && p.ways == 1 &&
               gx > (long long)sms * ctas_per_sm(rows_per_cta(p.cols, head_dim), head_dim);
    rc = launch_tc(L, dev, rows_per_cta(p.cols, head_dim), st);
    if (rc || L.mode != kQ8V2)
        return rc;
    return host_merge(seq_lens, num_seqs, q_len, num_heads, head_dim, cap, part, dtype, tmp_output,
                      exp_sums, max_logits, max_num_partitions, out, true, status, st);
}

} // extern "C"
