// pa_evict.cu -- cutting the sequences of a paged cache back to a budget of tokens, by
// the weight that each has accumulated, for every KV head on its own.
//
// Of a longer sequence stay the first `first`, the last `recent` and, of the tokens
// between, the need = budget - first - recent largest (equal weights: the earlier one;
// NaN counts as more than infinity), in the order of their positions.
//
// Pass 1, a CTA per (sequence, KV head), or a cluster of up to 8 that add their
// histograms through distributed shared memory: the weight of the need-th largest by
// radix select over the weights' bits, mapped so that they order as the numbers do (11 +
// 11 + 10 bits, a histogram in shared memory each, as far as it takes to set it apart);
// then one walk in order that gives every token that stays its new place, the ones equal
// to the border by a running count.
// Octets of tokens per thread: they lie in one block, and their keys stay in shared memory
// up to 16,384 tokens a CTA.  Bound by latency: a chain of loads, then some ten barriers.
//
// Pass 2 moves rows.  To other blocks: CTAs stride over tiles of rows, bound by bytes.
// In place: new place <= old place, both increasing, so the CTAs of one cluster walk one
// head's rows in step: all read a stretch of rows into registers, meet, then write it.
// Rows written in a stretch lie below every row read later.
//
// Measured: 32 sequences of up to 8192 tokens (16 bits, 8 heads of 128) cut to 2048 into
// other blocks 92 to 94 us: choosing 17, moving 74 (5.9 TB/s).  One of 100,000 tokens (4 bits,
// 4 heads) cut to 32,768: choosing 28 (a CTA per head 97), moving 12.  The same in place, single
// calls behind a flush of L2 (to other blocks 102 and 44): 199 and 90, by the barriered steps.
#include <cooperative_groups.h>

#include <atomic>

#include "pa_append.cuh"
#include "pa_evict.h"

namespace pa {

namespace {

constexpr int kSelectThreads = 512, kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kHeldOctets = 2048; // whose keys a CTA of pass 1 keeps: 72 KB
constexpr int kMoveRounds = 8; // 16-byte pieces per thread in flight

// Order-preserving bits of a weight: -0 as 0, NaN last.
__device__ __forceinline__ uint32_t order_of(float w)
{
    const uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0xffffffffu;
    if ((u & 0x7fffffffu) == 0u)
        return 0x80000000u;
    return (int)u < 0 ? ~u : u | 0x80000000u;
}

// An octet's weights as bits, of block `id`; a bad one counts as block 0 (and sets the
// status).
__device__ __forceinline__ void octet(const EvictParams &p, int id, int kv, int t, uint32_t (&key)[8])
{
    if (id < 0 || id >= p.num_blocks) {
        set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
        id = 0;
    }
    const float4 *const w = reinterpret_cast<const float4 *>(
        p.weights + (((size_t)id * p.num_kv_heads + kv) << p.block_shift) + (t & ((1 << p.block_shift) - 1)));
    const float4 a = w[0], d = w[1];
    key[0] = order_of(a.x);
    key[1] = order_of(a.y);
    key[2] = order_of(a.z);
    key[3] = order_of(a.w);
    key[4] = order_of(d.x);
    key[5] = order_of(d.y);
    key[6] = order_of(d.z);
    key[7] = order_of(d.w);
}

__device__ __forceinline__ int evict_len(const EvictParams &p, int b, bool report)
{
    const int L = *(volatile const int32_t *)(p.seq_lens + b); // (new_lens may be the same array)
    if (L >= 0 && L <= p.seq_len_cap)
        return L;
    if (report)
        set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
    return L < 0 ? 0 : p.seq_len_cap;
}

// Adds n at `at` in shared memory, or nothing: a predicate, not a branch.
__device__ __forceinline__ void count_if(bool yes, uint32_t at, uint32_t n)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared::cta.add.u32 [%1], %2;\n\t}" ::"r"((uint32_t)yes),
                 "r"(at), "r"(n)
                 : "memory");
}

// Places that n octets' halves take.
__host__ __device__ constexpr int held_places(int n) { return n + n / 8; }

// Exclusive sums of (x, y) over the CTA's threads in order, and the totals; kSelectThreads.
__device__ __forceinline__ void scan2(int &x, int &y, int &tx, int &ty, int (*s_scan)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ix = x, iy = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int vx = __shfl_up_sync(0xffffffffu, ix, off), vy = __shfl_up_sync(0xffffffffu, iy, off);
        ix += lane >= off ? vx : 0;
        iy += lane >= off ? vy : 0;
    }
    __syncthreads();
    if (lane == 31) {
        s_scan[warp][0] = ix;
        s_scan[warp][1] = iy;
    }
    __syncthreads();
    constexpr int kWarps = kSelectThreads / 32;
    const int wx = lane < kWarps ? s_scan[lane][0] : 0, wy = lane < kWarps ? s_scan[lane][1] : 0;
    int sx = wx, sy = wy;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int vx = __shfl_up_sync(0xffffffffu, sx, off), vy = __shfl_up_sync(0xffffffffu, sy, off);
        sx += lane >= off ? vx : 0;
        sy += lane >= off ? vy : 0;
    }
    tx = __shfl_sync(0xffffffffu, sx, 31);
    ty = __shfl_sync(0xffffffffu, sy, 31);
    x = ix - x + __shfl_sync(0xffffffffu, sx - wx, warp);
    y = iy - y + __shfl_sync(0xffffffffu, sy - wy, warp);
}

// The CTAs of a cluster share one (sequence, head)'s octets in order, each a stretch.
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const EvictParams p)
{
    __shared__ __align__(16) int s_bins[kBins];
    __shared__ int s_scan[32][2];
    __shared__ uint32_t s_digit;
    __shared__ int s_above, s_here;
    __shared__ int s_counts[2]; // of this CTA's stretch: above the border, equal to it
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    namespace cg = cooperative_groups;
    const int rank = blockIdx.x % p.select_ways, group = blockIdx.x / p.select_ways;
    const int kv = group % p.num_kv_heads, b = group / p.num_kv_heads;
    const int L = evict_len(p, b, kv == 0 && rank == 0 && threadIdx.x == 0);
    int32_t *const kept = p.kept + ((size_t)b * p.num_kv_heads + kv) * p.budget;
    if (L <= p.budget) {
        for (int t = threadIdx.x + rank * kSelectThreads; t < L; t += kSelectThreads * p.select_ways)
            kept[t] = t;
        return;
    }
    auto together = [&]() {
        if (p.select_ways > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    auto of_rank = [&](int *at, int r) { return p.select_ways > 1 ? cg::this_cluster().map_shared_rank(at, r) : at; };
    const int lo = p.first, hi = L - p.recent; // tokens that weights decide about
    // Octets [begin, end) are this CTA's, thread i's the i-th of each kSelectThreads.
    const int octets = (L + 7) / 8, share = (octets + p.select_ways - 1) / p.select_ways;
    const int begin = min(rank * share, octets), end = min(begin + share, octets);
    const int steps = (share + kSelectThreads - 1) / kSelectThreads;
    // Their keys lie in shared memory, if they are few enough (0: not up for choice; no
    // number's is): halves of octets apart, so that neighbours' loads meet no conflict.
    extern __shared__ uint4 s_keys[]; // [2][held_places(held)]
    const bool held = end - begin <= p.select_held;
    auto block_of = [&](int o) { return __ldg(p.block_tables + (size_t)b * p.max_blocks + (o * 8 >> p.block_shift)); };
    auto load = [&](int o, int id, uint32_t (&key)[8]) { // octet o, of block id
        if (o * 8 + 8 > lo && o * 8 < hi) {
            octet(p, id, kv, o * 8, key);
            if (o * 8 < lo || o * 8 + 8 > hi) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (o * 8 + k < lo || o * 8 + k >= hi)
                        key[k] = 0u;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                key[k] = 0u;
        }
    };
    // (One place of nine stays free: loads of octets beside one another, and of every fourth,
    // meet no conflict.)
    auto held_at = [&](int o) { return o - begin + (o - begin >> 3); };
    const int held_all = held_places(p.select_held);
    auto fetch = [&](int o, uint32_t (&key)[8]) {
        if (!held) {
            load(o, block_of(o), key);
            return;
        }
        const uint4 x = s_keys[held_at(o)], y = s_keys[held_all + held_at(o)];
        key[0] = x.x; key[1] = x.y; key[2] = x.z; key[3] = x.w;
        key[4] = y.x; key[5] = y.y; key[6] = y.z; key[7] = y.w;
    };
    if (held) {
        constexpr int kMany = 4; // octets of a thread under way at a time
        for (int o0 = begin + threadIdx.x; o0 < end; o0 += kMany * kSelectThreads) {
            int id[kMany];
            uint32_t key[kMany][8];
#pragma unroll
            for (int i = 0; i < kMany; ++i)
                id[i] = block_of(min(o0 + i * kSelectThreads, end - 1));
#pragma unroll
            for (int i = 0; i < kMany; ++i)
                load(min(o0 + i * kSelectThreads, end - 1), id[i], key[i]);
#pragma unroll
            for (int i = 0; i < kMany; ++i) {
                const int o = o0 + i * kSelectThreads;
                if (o < end) {
                    s_keys[held_at(o)] = make_uint4(key[i][0], key[i][1], key[i][2], key[i][3]);
                    s_keys[held_all + held_at(o)] = make_uint4(key[i][4], key[i][5], key[i][6], key[i][7]);
                }
            }
        }
    }
    int need = p.budget - p.first - p.recent;  // < hi - lo
    uint32_t border = 0u, above = 0xffffffffu; // keys above it stay (need = 0: none)
    int equal = 0;                             // how many of those equal to it stay
    if (need > 0) {
        // The need-th largest, digit by digit: `prefix` its digits so far, `need` the
        // place that is left among those with the same.
        uint32_t prefix = 0u;
        const uint32_t bins = smem_addr(s_bins);
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            if (pass > 0)
                together(); // everyone has read the last pass's bins
            for (int i = threadIdx.x; i < kBins; i += kSelectThreads)
                s_bins[i] = 0;
            __syncthreads();
            for (int o = begin + threadIdx.x; o < end; o += kSelectThreads) {
                uint32_t key[8];
                fetch(o, key);
                uint32_t other = 0u;
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    other |= key[k] ^ key[0];
                const uint32_t mask = (1u << bits) - 1;
                auto in = [&](uint32_t x) { return pass == 0 ? x != 0u : x >> (shift + bits) == prefix; };
                // (Equal weights would queue at one bin.)
                const bool one = other == 0u;
                count_if(in(key[0]), bins + (key[0] >> shift & mask) * 4, one ? 8u : 1u);
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    count_if(in(key[k]) && !one, bins + (key[k] >> shift & mask) * 4, 1u);
            }
            together();
            // The bin that holds it, from the top: a thread's four bins, then a scan.
            const int top = (1 << bits) - 4 - 4 * (int)threadIdx.x; // larger digits first
            int c[4] = {0, 0, 0, 0};
            if (top >= 0) {
                int4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    v[r] = r < p.select_ways ? *reinterpret_cast<const int4 *>(of_rank(s_bins + top, r)) : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    c[0] += v[r].x;
                    c[1] += v[r].y;
                    c[2] += v[r].z;
                    c[3] += v[r].w;
                }
            }
            int before = c[0] + c[1] + c[2] + c[3], unused = 0, total, unused2;
            scan2(before, unused, total, unused2, s_scan);
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                if (before < need && need <= before + c[k]) {
                    s_digit = top + k;
                    s_above = before;
                    s_here = c[k];
                }
                before += c[k];
            }
            __syncthreads();
            prefix = prefix << bits | s_digit;
            need -= s_above;
            border = prefix << shift;
            if (need == s_here) { // all of the bin stays, often one weight alone: no digits to tell it from
                above = border - 1; // (no number's key begins with zeros alone)
                break;
            }
            above = border; // (the last digit: of those equal to it `need` stay)
            equal = pass == 2 ? need : 0;
        }
    }
    // ---- in order: the place of each token that stays.  Bits of an octet: stays whatever
    // the others do; equal to the border.
    auto bits_of = [&](int o, uint32_t &keep, uint32_t &same) {
        uint32_t key[8];
        fetch(o, key);
        keep = same = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            keep |= (key[k] > above ? 1u : 0u) << k;
            same |= (equal > 0 && key[k] == border ? 1u : 0u) << k;
        }
        if (o * 8 < lo || o * 8 + 8 > hi) { // the first and the last ones stay
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (o * 8 + k < lo || (o * 8 + k >= hi && o * 8 + k < L))
                    keep |= 1u << k;
        }
    };
    // (Here a thread's octets are neighbours, so that one scan gives all their places.  The
    // keys another thread has written are seen: there have been barriers, or are now.)
    const int mine0 = min(begin + (int)threadIdx.x * steps, end), mine1 = min(mine0 + steps, end);
    __syncthreads();
    int eq = 0, sure = 0;
    for (int o = mine0; o < mine1; ++o) {
        uint32_t keep, same;
        bits_of(o, keep, same);
        eq += __popc(same);
        sure += __popc(keep);
    }
    int all_eq, all_sure;
    scan2(eq, sure, all_eq, all_sure, s_scan);
    if (threadIdx.x == 0) {
        s_counts[0] = all_sure;
        s_counts[1] = all_eq;
    }
    together();
#pragma unroll
    for (int r = 0; r < 8; ++r) { // of the CTAs before this one
        sure += r < rank ? *of_rank(s_counts, r) : 0;
        eq += r < rank ? *of_rank(s_counts + 1, r) : 0;
    }
    // Before octet o: `sure` above the border, `eq` equal to it, of which the first `equal`
    // stay.
    for (int o = mine0; o < mine1; ++o) {
        uint32_t keep, same;
        bits_of(o, keep, same);
        const int ahead = min(eq, equal), n_eq = __popc(same), n_sure = __popc(keep);
        const int n_stay = min(eq + n_eq, equal) - ahead;
        for (int k = n_eq; k > n_stay; --k) // the last of them go
            same &= ~(0x80000000u >> __clz(same));
        const uint32_t stay = keep | same;
        int at = sure + ahead;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool stays = stay >> k & 1u;
            if (stays && at < p.budget) // (always, unless the weights change under the call)
                kept[at] = o * 8 + k;
            at += stays;
        }
        sure += n_sure;
        eq += n_eq;
    }
    if (p.select_ways > 1)
        cg::this_cluster().sync(); // the others have read this CTA's counts
}

// Row of token t of (sequence, head) under a table, or -1.
__device__ __forceinline__ long long cache_row(const EvictParams &p, const int32_t *tables, int width, int b, int kv, int t)
{
    const int id = __ldg(tables + (size_t)b * width + (t >> p.block_shift));
    if (id < 0 || id >= p.num_blocks) {
        set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
        return -1;
    }
    return ((long long)id * p.num_kv_heads + kv << p.block_shift) + (t & ((1 << p.block_shift) - 1));
}

// A stretch of rows [j0, j0 + n) of one head in registers: loaded, then stored.
// IN_PLACE: rows that already lie where they go are passed over.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictParams p, int rows, int stretches)
{
    extern __shared__ long long s_rows[]; // [rows][2]: from, to (-1: nothing to do)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // In place: cluster = (sequence, head), its CTAs side by side in each step.
    const int group = IN_PLACE ? blockIdx.x / p.ways : blockIdx.x / stretches;
    const int first_stretch = IN_PLACE ? blockIdx.x % p.ways : blockIdx.x % stretches;
    const int step = IN_PLACE ? p.ways : stretches;
    const int kv = group % p.num_kv_heads, b = group / p.num_kv_heads;
    const int count = min(evict_len(p, b, false), p.budget);
    const int32_t *const kept = p.kept + ((size_t)b * p.num_kv_heads + kv) * p.budget;
    const int pieces = p.row_bytes / 16, lg = __ffs(pieces) - 1; // a power of two
    const uint4 *const kc = static_cast<const uint4 *>(p.key_cache), *const vc = static_cast<const uint4 *>(p.value_cache);
    uint4 *const kd = static_cast<uint4 *>(p.key_cache), *const vd = static_cast<uint4 *>(p.value_cache);
    // In place nothing moves where the last token keeps its place.  (Not by the length: it
    // may have been cut already.)
    const int n_steps = !IN_PLACE ? first_stretch * rows < count
                        : count > 0 && kept[count - 1] != count - 1 ? ((count + rows - 1) / rows + step - 1) / step : 0;
    for (int i = 0; i < n_steps; ++i) {
        const int j0 = (i * step + first_stretch) * rows, n = min(rows, count - j0); // (n < 1: past the end)
        __syncthreads();
        for (int r = threadIdx.x; r < n; r += kMoveThreads) {
            const int j = j0 + r, src = kept[j];
            long long from = -1, to = -1;
            if ((!IN_PLACE || src != j) && src >= 0 && src < p.seq_len_cap) {
                from = cache_row(p, p.block_tables, p.max_blocks, b, kv, src);
                to = cache_row(p, p.dst_tables, p.dst_max_blocks, b, kv, j);
                if (to < 0)
                    from = -1;
            }
            s_rows[2 * r] = from;
            s_rows[2 * r + 1] = to;
        }
        __syncthreads();
        // Keys' pieces, then values'; rows * pieces * 2 = kMoveThreads * kMoveRounds of them.
        uint4 x[kMoveRounds];
#pragma unroll
        for (int u = 0; u < kMoveRounds; ++u) {
            const int at = threadIdx.x + u * kMoveThreads, r = at >> (lg + 1);
            const long long from = r < n ? s_rows[2 * r] : -1;
            if (from >= 0)
                x[u] = ((at >> lg & 1) ? vc : kc)[from * pieces + (at & (pieces - 1))];
        }
        // A thread per row: its weight and scales.
        float w = 0.f;
        uint64_t ks = 0, vs = 0;
        const long long from = (int)threadIdx.x < n ? s_rows[2 * threadIdx.x] : -1;
        if (from >= 0) {
            w = p.weights[from];
            if (p.scale_bytes == 2) {
                ks = reinterpret_cast<const uint16_t *>(p.k_scales)[from];
                vs = reinterpret_cast<const uint16_t *>(p.v_scales)[from];
            } else if (p.scale_bytes == 4) {
                ks = reinterpret_cast<const uint32_t *>(p.k_scales)[from];
                vs = reinterpret_cast<const uint32_t *>(p.v_scales)[from];
            } else if (p.scale_bytes == 8) {
                ks = reinterpret_cast<const uint64_t *>(p.k_scales)[from];
                vs = reinterpret_cast<const uint64_t *>(p.v_scales)[from];
            }
        }
        if (IN_PLACE) { // everyone has read this step's rows
            if (p.ways > 1)
                cooperative_groups::this_cluster().sync();
            else
                __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kMoveRounds; ++u) {
            const int at = threadIdx.x + u * kMoveThreads, r = at >> (lg + 1);
            if (r < n && s_rows[2 * r] >= 0)
                ((at >> lg & 1) ? vd : kd)[s_rows[2 * r + 1] * pieces + (at & (pieces - 1))] = x[u];
        }
        if (from >= 0) {
            const long long dst = s_rows[2 * threadIdx.x + 1];
            p.weights[dst] = w;
            if (p.scale_bytes == 2) {
                reinterpret_cast<uint16_t *>(p.k_scales)[dst] = (uint16_t)ks;
                reinterpret_cast<uint16_t *>(p.v_scales)[dst] = (uint16_t)vs;
            } else if (p.scale_bytes == 4) {
                reinterpret_cast<uint32_t *>(p.k_scales)[dst] = (uint32_t)ks;
                reinterpret_cast<uint32_t *>(p.v_scales)[dst] = (uint32_t)vs;
            } else if (p.scale_bytes == 8) {
                reinterpret_cast<uint64_t *>(p.k_scales)[dst] = ks;
                reinterpret_cast<uint64_t *>(p.v_scales)[dst] = vs;
            }
        }
    }
    // (Any reader of a length that is cut already finds the same count.)
    if (kv == 0 && first_stretch == 0 && threadIdx.x == 0)
        p.new_lens[b] = count;
}

} // namespace

cudaError_t launch_evict(const EvictParams &p0, int num_sms, int dev, cudaStream_t stream)
{
    EvictParams p = p0;
    const long long groups = (long long)p.num_seqs * p.num_kv_heads;
    // CTAs of a cluster: while they have more than an octet per thread and lie side by side.
    p.select_ways = 1;
    while (p.select_ways < 8 && p.seq_len_cap > p.select_ways * kSelectThreads * 8 && groups * 2 * p.select_ways <= num_sms)
        p.select_ways *= 2;
    cudaLaunchConfig_t cfg = {};
    const int share = ((p.seq_len_cap + 7) / 8 + p.select_ways - 1) / p.select_ways;
    p.select_held = share < kHeldOctets ? share : kHeldOctets;
    static std::atomic<int> prepared[64];
    if (prepared[dev].load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   held_places(kHeldOctets) * 32);
        if (e != cudaSuccess)
            return e;
        prepared[dev].store(1, std::memory_order_release);
    }
    cfg.gridDim = dim3((unsigned)(groups * p.select_ways));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = (size_t)held_places(p.select_held) * 32;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.select_ways;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.select_ways > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, p);
    if (e != cudaSuccess)
        return e;
    int rows = kMoveThreads * kMoveRounds / (p.row_bytes / 16 * 2);
    rows = rows < kMoveThreads ? rows : kMoveThreads; // (a thread per row for the rest)
    const int most = p.budget < p.seq_len_cap ? p.budget : p.seq_len_cap;
    int stretches = (most + rows - 1) / rows;
    const bool in_place = p.dst_tables == p.block_tables;
    p.ways = 1;
    while (in_place && p.ways < 8 && 2 * p.ways <= stretches && groups * 2 * p.ways <= 2 * num_sms)
        p.ways *= 2;
    cfg.gridDim = dim3((unsigned)(groups * (in_place ? p.ways : stretches)));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = (size_t)rows * 16;
    attr[1].val.clusterDim.x = (unsigned)p.ways;
    cfg.numAttrs = in_place && p.ways > 1 ? 2 : 1;
    return in_place ? cudaLaunchKernelEx(&cfg, move_kernel<true>, p, rows, stretches)
                    : cudaLaunchKernelEx(&cfg, move_kernel<false>, p, rows, stretches);
}

} // namespace pa
