// pa_append.cuh -- what the appends to 16-, 8- and 4-bit caches share: which sequence
// and position a token row has, and the rotation of its heads (see pa_append.cu).
#pragma once

#include "pa_device.cuh"
#include "pa_q8.h"

namespace pa {

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    using E = Elem<T>;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = E::lo(w[k]);
        x[2 * k + 1] = E::hi(w[k]);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    using E = Elem<T>;
    return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]),
                      E::pack(x[6], x[7]));
}

// A sequence of a ragged batch: its token rows [begin, end) and its length.
struct Seq {
    int b, begin, end, len;
};

// The last sequence b < n whose key(b) <= at, key increasing with b: from its first
// token row (key = starts[b]) or its first block item.  False when there is none.
// The warp probes 32 entries at a time, and fetches the rows' ends and the lengths
// along with the last probes: one chain link for up to 31 sequences, two for about
// a thousand.
template <typename Key>
__device__ __forceinline__ bool find_seq(const AppendParams &p, long long at, int lane, Key key, Seq &s)
{
    const int n = p.num_seqs;
    int lo = 0, hi = n; // how many have key <= at: in [lo, hi]
    while (hi - lo > 30) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + (lane + 1) * step - 1;
        const bool le = i < hi && key(i, __ldg(p.token_starts + i)) <= at;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        const int next = min(lo + c * step, hi);
        hi = max(min(hi, lo + (c + 1) * step - 1), next);
        lo = next;
    }
    // Lane l holds entry first + l, first .. hi (at most 32 of them).
    const int first = lo > 0 ? lo - 1 : 0;
    const int i = first + lane;
    const int start = i <= n && i <= hi ? __ldg(p.token_starts + i) : 0;
    const int len = i < n && i <= hi ? __ldg(p.seq_lens + i) : 0;
    const bool le = i < n && i < hi && key(i, start) <= at;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1; // among these
    if (k < 0)
        return false;
    s.b = first + k;
    s.begin = __shfl_sync(0xffffffffu, start, k);
    s.end = __shfl_sync(0xffffffffu, start, k + 1);
    s.len = __shfl_sync(0xffffffffu, len, k);
    return true;
}

// Which two 8-dim chunks of a row item u (of head_dim / 16) covers, and
// whether it is rotated.  Neighbouring halves: chunk u and the one r / 2 dims
// up; the dims past rotary_dim, and interleaved rows, chunk by chunk.
struct Item {
    int c0, c1;
    bool rot0, rot1; // interleaved: per chunk; else both or none
};

__device__ __forceinline__ Item item_of(int u, int rotary_dim, bool interleaved, bool rotate)
{
    Item it;
    const int half = rotary_dim / 16; // chunks of one half
    if (rotate && !interleaved && u < half) {
        it.c0 = u;
        it.c1 = u + half;
        it.rot0 = it.rot1 = true;
    } else {
        it.c0 = 2 * u;
        it.c1 = 2 * u + 1;
        it.rot0 = rotate && interleaved && it.c0 * 8 < rotary_dim;
        it.rot1 = rotate && interleaved && it.c1 * 8 < rotary_dim;
    }
    return it;
}

// The 16 cosines and sines item u needs: neighbouring halves cos[8], sin[8];
// interleaved 4 cosines and 4 sines for each chunk.
__device__ __forceinline__ void load_angles(const float *row, const Item &it, int rotary_dim,
                                            bool interleaved, float (&c)[8], float (&s)[8])
{
    const int half = rotary_dim / 2;
    const int o0 = interleaved ? it.c0 * 4 : it.c0 * 8;
    const int o1 = interleaved ? it.c1 * 4 : it.c0 * 8 + 4;
    const bool r1 = interleaved ? it.rot1 : it.rot0;
    const float4 z = make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 a = it.rot0 ? __ldg(reinterpret_cast<const float4 *>(row + o0)) : z;
    const float4 b = r1 ? __ldg(reinterpret_cast<const float4 *>(row + o1)) : z;
    const float4 d = it.rot0 ? __ldg(reinterpret_cast<const float4 *>(row + half + o0)) : z;
    const float4 e = r1 ? __ldg(reinterpret_cast<const float4 *>(row + half + o1)) : z;
    c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
    c[4] = b.x; c[5] = b.y; c[6] = b.z; c[7] = b.w;
    s[0] = d.x; s[1] = d.y; s[2] = d.z; s[3] = d.w;
    s[4] = e.x; s[5] = e.y; s[6] = e.z; s[7] = e.w;
}

// Products and their difference are rounded one by one (no contraction), as
// the formula is written.
__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s)
{
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
    b = y;
}

__device__ __forceinline__ void rotate_item(float (&x0)[8], float (&x1)[8], const Item &it,
                                            bool interleaved, const float (&c)[8],
                                            const float (&s)[8])
{
    if (interleaved) {
        if (it.rot0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rotate_pair(x0[2 * k], x0[2 * k + 1], c[k], s[k]);
        }
        if (it.rot1) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rotate_pair(x1[2 * k], x1[2 * k + 1], c[4 + k], s[4 + k]);
        }
    } else if (it.rot0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            rotate_pair(x0[k], x1[k], c[k], s[k]);
    }
}

// Where token row t goes.  Returns false (and sets the status bit) for a row
// that belongs to no sequence or has no valid position.  *angle: the position it is
// rotated by.  OFFSETS: the call may have offsets of positions (the 8-bit append has none:
// asking took two chunks of 2048 tokens from 14.1 to 14.4 us).
template <bool OFFSETS = true>
__device__ __forceinline__ bool place_of(const AppendParams &p, int t, int lane, bool reporter,
                                         int *seq, int *pos, int *angle, Seq *of = nullptr)
{
    Seq q;
    if (p.token_starts) {
        if (!find_seq(p, t, lane, [](int, int start) { return (long long)start; }, q) || t >= q.end)
            return false; // before the first sequence's rows or behind the last one's
        if (q.end > p.num_tokens) {
            if (reporter)
                set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
            return false;
        }
    } else {
        q.b = t / p.q_len;
        q.end = (q.b + 1) * p.q_len;
        q.len = __ldg(p.seq_lens + q.b);
    }
    const int L = q.len;
    const long long at = (long long)L - q.end + t;
    if (at < 0 || L > p.max_blocks * p.block_size) {
        if (reporter)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        if (at < 0 || at >= (long long)p.max_blocks * p.block_size)
            return false;
    }
    const long long turn = OFFSETS && p.pos_offsets ? at + __ldg(p.pos_offsets + q.b) : at;
    if (p.rotary_dim && (turn < 0 || turn >= p.max_positions)) {
        if (reporter)
            set_status(p.status, PA_STATUS_BAD_POSITION);
        return false;
    }
    if (of)
        *of = q;
    *seq = q.b;
    *pos = (int)at;
    *angle = (int)turn;
    return true;
}

template <typename F>
inline cudaError_t launch_pdl(F *fn, unsigned grid, unsigned threads, cudaStream_t stream, void **args, size_t smem = 0)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(fn), args);
}

} // namespace pa
