// pa_q8_copy.cu -- a 16-bit copy of the blocks one multi-query call reads from
// an 8-bit cache, for calls with many query rows per KV head (chunked prefill):
// there each value read serves hundreds of rows, the copy's bytes are a few
// percent of the call, and the 16-bit tcgen05 kernels, whose rows run on one
// thread each, compute faster than the 8-bit one.
//
// The sequences' blocks lie packed, sequence s's logical block j at index
// offs[s] + j (offs the exclusive prefix sum of ceil(L_s / block_size)), rows
// past a sequence's end zero:
//   K  [copy_blocks][KV][block_size][D] in the query's type, a cache of its own
//      with the block table the pass writes;
//   V  the same for binary16 queries; for bf16 ones binary16 in the layout
//      [KV][copy_blocks][block_size][D] that the two-tile kernel's binary16
//      P.V reads.
// value = code * scale, exactly: the scales that the append writes are powers of two, and
// what the 16-bit types hold under them is what the 8-bit kernel multiplies.  A nonzero
// code under any other scale -- one that is no power of two, or so large or small that
// the type does not hold every code's value under it (see exact_under) -- sets the flag:
// the 16-bit attention behind then returns at once and the call runs the 8-bit kernel,
// so that a result's precision depends neither on the number of rows nor on the
// workspace.
//
// Bound by its bytes and the chain that finds a block: one read of the codes, two bytes
// written for each; 24 us alone for 36 MB of codes (66% of the measured copy
// bandwidth), before 293 of attention.
#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_q8.h"

namespace pa {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyRounds = 4; // 16-byte pieces per thread in flight

__device__ __forceinline__ int clamp_len(int L, int cap) { return L < 0 ? 0 : L > cap ? cap : L; }

// One CTA: the offsets, and the flag cleared.
__global__ void __launch_bounds__(kScanThreads) q8_offsets_kernel(const Q8CopyParams p)
{
    __shared__ long long part[kScanThreads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int per = (p.num_seqs + kScanThreads - 1) / kScanThreads;
    const int s0 = threadIdx.x * per, s1 = min(s0 + per, p.num_seqs);
    auto nblocks = [&](int s) {
        return (long long)((clamp_len(__ldg(p.seq_lens + s), p.seq_len_cap) + p.block_size - 1) /
                           p.block_size);
    };
    long long sum = 0;
    for (int s = s0; s < s1; ++s)
        sum += nblocks(s);
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int d = 1; d < kScanThreads; d <<= 1) { // inclusive scan
        const long long v = threadIdx.x >= d ? part[threadIdx.x - d] : 0;
        __syncthreads();
        part[threadIdx.x] += v;
        __syncthreads();
    }
    long long run = part[threadIdx.x] - sum;
    for (int s = s0; s < s1; ++s) {
        p.offs[s] = (int32_t)run;
        run += nblocks(s);
    }
    if (threadIdx.x == kScanThreads - 1) {
        p.offs[p.num_seqs] = (int32_t)part[threadIdx.x];
        *p.flag = 0;
    }
}

// Whether T holds every code times s: e4m3 has 4 significant bits and values from 2^-9 to
// 448 = 1.75 * 2^8.  binary16 holds multiples of 2^-24 and up to 65504.  bf16 would hold
// them from 2^-117 to 2^119, but there a sum of products with a query can leave fp32's
// range where the 8-bit kernel's, of codes, does not: far within it, 2^-60 to 2^60.
template <typename T>
__device__ __forceinline__ bool exact_under(float s)
{
    const float lo = Elem<T>::kSplitP ? 8.673617379884035e-19f : 3.0517578125e-5f; // 2^-60, 2^-15
    const float hi = Elem<T>::kSplitP ? 1.152921504606847e18f : 128.f;             // 2^60, 2^7
    return s == 0.f || ((__float_as_uint(s) & 0x7fffffu) == 0u && s >= lo && s <= hi);
}

template <typename T>
__device__ __forceinline__ void widen(const uint4 &v, float scale, uint4 (&out)[2])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[k >> 1] >> ((k & 1) * 16)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        r[k] = Elem<T>::pack(f.x * scale, f.y * scale);
    }
    out[0] = make_uint4(r[0], r[1], r[2], r[3]);
    out[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// CTAs stride over the K and the V of packed blocks; a thread moves 16 codes at a
// time.  T: the type of K and, unless VH, of V.
template <typename T, bool VH>
__global__ void __launch_bounds__(kCopyThreads) q8_copy_kernel(const Q8CopyParams p)
{
    __shared__ int s_id, s_rows;
    asm volatile("griddepcontrol.wait;" ::: "memory"); // the offsets, and the flag cleared
    const int total = __ldg(p.offs + p.num_seqs);
    const int per_row = p.head_dim / 16;             // pieces of a row (a power of two)
    const int per_head = p.block_size * per_row;     // of one head of a block (a power of two)
    const int lg_row = __ffs(per_row) - 1, lg_head = __ffs(per_head) - 1;
    const int pieces = p.num_kv_heads * per_head;
    const uint4 *kc = static_cast<const uint4 *>(p.key_cache);
    const uint4 *vc = static_cast<const uint4 *>(p.value_cache);
    bool odd = false;
    for (long long item = blockIdx.x; item < 2LL * total; item += gridDim.x) {
        const int q = (int)(item >> 1), which = (int)(item & 1);
        __syncthreads();
        if (threadIdx.x == 0) {
            int lo = 0, hi = p.num_seqs - 1; // the last s with offs[s] <= q
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(p.offs + mid) <= q)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int j = q - __ldg(p.offs + lo);
            int id = __ldg(p.block_tables + (size_t)lo * p.max_blocks + j);
            if (id < 0 || id >= p.num_blocks) {
                if (which == 0)
                    set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                id = 0; // read a valid block instead of memory outside the cache
            }
            s_id = id;
            s_rows = min(p.block_size,
                         clamp_len(__ldg(p.seq_lens + lo), p.seq_len_cap) - j * p.block_size);
            if (which == 0)
                p.table[(size_t)lo * p.table_width + j] = q;
        }
        __syncthreads();
        const int id = s_id, rows = s_rows;
        const size_t src = (size_t)id * pieces;
        const uint4 *in = (which ? vc : kc) + src;
        const float *scales = (which ? p.v_scales : p.k_scales) + (size_t)id * p.num_kv_heads;
        uint4 *out = static_cast<uint4 *>(which ? p.v_copy : p.k_copy);
        for (int base = threadIdx.x; base < pieces; base += kCopyRounds * kCopyThreads) {
            uint4 x[kCopyRounds];
#pragma unroll
            for (int u = 0; u < kCopyRounds; ++u) {
                const int i = base + u * kCopyThreads;
                const bool in_row = i < pieces && ((i & (per_head - 1)) >> lg_row) < rows;
                x[u] = in_row ? __ldg(in + i) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kCopyRounds; ++u) {
                const int i = base + u * kCopyThreads;
                if (i >= pieces)
                    continue;
                const int h = i >> lg_head;
                float s = __ldg(scales + h);
                if (which && !(s >= 0.f && s <= 3.4028234663852886e38f))
                    s = NAN; // as in the 8-bit kernel
                // Codes but for their signs.
                const uint32_t any = (x[u].x | x[u].y | x[u].z | x[u].w) & 0x7f7f7f7fu;
                if (any != 0u && !(VH && which == 1 ? exact_under<__half>(s) : exact_under<T>(s)))
                    odd = true;
                uint4 y[2];
                if (VH && which == 1)
                    widen<__half>(x[u], s, y);
                else
                    widen<T>(x[u], s, y);
                const size_t at = VH && which == 1
                                      ? ((size_t)h * p.copy_blocks + q) * per_head + (i & (per_head - 1))
                                      : (size_t)q * pieces + i;
                out[2 * at] = y[0];
                out[2 * at + 1] = y[1];
            }
        }
    }
    if (__syncthreads_or(odd) && threadIdx.x == 0)
        atomicOr(p.flag, 1);
}

} // namespace

cudaError_t launch_q8_copy(int dtype, bool v_half, const Q8CopyParams &p, int num_sms,
                           cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, q8_offsets_kernel, p);
    if (e != cudaSuccess)
        return e;
    const long long most = 2LL * p.num_seqs * ((p.seq_len_cap + p.block_size - 1) / p.block_size);
    const long long slots = 8LL * num_sms;
    const unsigned grid = (unsigned)(most < slots ? (most > 0 ? most : 1) : slots);
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kCopyThreads);
    return v_half              ? cudaLaunchKernelEx(&cfg, q8_copy_kernel<__nv_bfloat16, true>, p)
           : dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, q8_copy_kernel<__nv_bfloat16, false>, p)
                              : cudaLaunchKernelEx(&cfg, q8_copy_kernel<__half, false>, p);
}

} // namespace pa
