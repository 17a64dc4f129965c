// pa_append.cu -- appending the keys and values of new tokens to a paged
// cache, the position rotation applied on the way, and (optionally) rotating
// their queries in the same launch.
//
// Rotation of a row x at position n, over its first r = rotary_dim dims, by
// the angles whose cosines c_i and sines s_i the caller tabulates:
//     x'_a = x_a c_i - x_b s_i,   x'_b = x_b c_i + x_a s_i,   i < r / 2,
// with (a, b) = (i, i + r / 2), or (2i, 2i + 1) when interleaved; the other
// dims pass unchanged.  It is computed in fp32 and rounded once, to the
// storage type (or straight to 8 bits).
//
// Measured on a GB300 (us a call, share of the measured copy bandwidth): 64 prompts
// of up to 2048 tokens, 64 heads on 8, 128 dims, blocks of 32: 410 (98%), to 8 bits 404
// (94%; blocks of 8 405, of 64 460, 83%); 32 such prompts of 256 dims 399 (100%), to 8
// bits 446 (85%) at blocks of 32 and 468 (81%) of 64, whose wide CTAs of several heads
// spill; 64 of 64 dims 242 (83%), to 8 bits 244 (78%).  Two chunks of 2048 tokens, 32
// heads on 8, to 8 bits: 18.7 (74%); 32 single tokens to 8 bits 3.4, one token 2.7
// (latency and launch).
//
// 16-bit caches: a pure copy with three operations per value, bound by bytes
// on prompts and by its chain of dependent loads (starts -> length -> block
// id -> store) on single tokens.  One CTA per token: a thread keeps one pair
// of 8-dim chunks for the heads it visits, so the token's cosines and sines
// are read once per thread, and the row loads are issued before anything
// that depends on the token's place.
//
// 8-bit caches (e4m3): the rows of one block and KV head share a scale,
//     s = the smallest power of two with amax <= 448 s,
// amax over the block's new rows, and never below the scale the block already
// has when it holds earlier tokens.  A grown scale re-quantises those rows:
// between powers of two that only moves exponents (exact, but for values that
// fall into e4m3's subnormals), so rounding does not build up as a block is
// filled token by token.  One CTA owns one (block, KV head) -- its rows times
// pairs of chunks are its threads -- so the maximum is a reduction inside the
// CTA and no two CTAs write one scale.  Splitting K and V over CTAs, and four
// rows per thread in flight, were slower.
#include <cuda_fp8.h>

#include <type_traits>

#include "pa_append.cuh"

namespace pa {

namespace {

constexpr int kAppendThreads = 128;
// Rows per thread in flight and CTAs per SM: prompts 410 us, 420 with four rows.
constexpr int kAppendRounds = 2;
constexpr int kAppendCtas = 8;

// One CTA per token row; rows of heads: query, then key, then value.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) append_kernel(const AppendParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int items = p.head_dim / 16;                 // per row: 4, 8 or 16
    const int u = threadIdx.x % items;
    const int row0 = threadIdx.x / items;
    const int step = kAppendThreads / items;           // rows the CTA covers at once
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const bool interleaved = p.interleaved != 0;
    const Item rot = item_of(u, p.rotary_dim, interleaved, true);
    const Item raw = item_of(u, 0, false, false);

    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) +
                                                     t * p.query_stride);
    const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key) +
                                                     t * p.key_stride);
    const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.value) +
                                                     t * p.value_stride);
    uint4 *qo = reinterpret_cast<uint4 *>(static_cast<T *>(p.query_out) + t * p.query_out_stride);
    const int chunks = p.head_dim / 8;

    int b = 0, pos = 0, angle = 0;
    bool ok = false, have_place = false;
    int32_t block = -1;
    float c[8], s[8];
    for (int base = row0; base - row0 < rows; base += kAppendRounds * step) {
        uint4 x0[kAppendRounds], x1[kAppendRounds];
#pragma unroll
        for (int i = 0; i < kAppendRounds; ++i) {
            const int h = base + i * step;
            if (h < rows) {
                const bool is_v = h >= p.num_heads + p.num_kv_heads;
                const Item &it = is_v ? raw : rot;
                // Plain loads: the query may be rotated in place.
                const uint4 *src = h < p.num_heads ? q + h * chunks
                                   : !is_v         ? k + (h - p.num_heads) * chunks
                                                   : v + (h - p.num_heads - p.num_kv_heads) * chunks;
                x0[i] = src[it.c0];
                x1[i] = src[it.c1];
            }
        }
        if (!have_place) {
            have_place = true;
            ok = place_of(p, t, lane, threadIdx.x == 0, &b, &pos, &angle);
            if (ok) {
                block = __ldg(p.block_tables + (size_t)b * p.max_blocks + pos / p.block_size);
                if (block < 0 || block >= p.num_blocks) {
                    if (threadIdx.x == 0)
                        set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                    block = -1;
                }
                if (p.rotary_dim)
                    load_angles(p.cos_sin + (size_t)angle * p.rotary_dim, rot, p.rotary_dim,
                                interleaved, c, s);
            }
        }
        if (!ok)
            return;
#pragma unroll
        for (int i = 0; i < kAppendRounds; ++i) {
            const int h = base + i * step;
            if (h >= rows)
                continue;
            const bool is_v = h >= p.num_heads + p.num_kv_heads;
            if (!is_v && (rot.rot0 || rot.rot1)) {
                float a[8], d[8];
                unpack8<T>(x0[i], a);
                unpack8<T>(x1[i], d);
                rotate_item(a, d, rot, interleaved, c, s);
                x0[i] = pack8<T>(a);
                x1[i] = pack8<T>(d);
            }
            const Item &it = is_v ? raw : rot;
            uint4 *dst;
            if (h < p.num_heads) {
                dst = qo + h * chunks;
            } else {
                if (block < 0)
                    continue;
                const int kv = is_v ? h - p.num_heads - p.num_kv_heads : h - p.num_heads;
                dst = static_cast<uint4 *>(is_v ? p.value_cache : p.key_cache) +
                      (((size_t)block * p.num_kv_heads + kv) * p.block_size + pos % p.block_size) *
                          chunks;
            }
            dst[it.c0] = x0[i];
            dst[it.c1] = x1[i];
        }
    }
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8),
// from amax's bits.
__device__ __forceinline__ float scale_of(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Four values -> four e4m3 codes (NaN stays NaN; infinities saturate).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint2 to_e4m3x8(const float (&x)[8], float f)
{
    return make_uint2(to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                      to_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
}

__device__ __forceinline__ void divide8(float (&x)[8], float s)
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        x[k] = __fdiv_rn(x[k], s);
}

__device__ __forceinline__ void from_e4m3x8(uint2 v, float (&x)[8])
{
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[k >> 1] >> ((k & 1) * 16)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}

// Largest magnitude; NaN when there is one.
__device__ __forceinline__ float amax8(const float (&x)[8], float m)
{
#pragma unroll
    for (int k = 0; k < 8; k += 2)
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x[k]), "f"(x[k + 1]));
    return m;
}

// The same of eight 16-bit values, as the bits of the widened value's magnitude, larger
// than any finite one's for infinities and NaN.
template <typename T>
__device__ __forceinline__ uint32_t amax8_bits(const uint4 &v, uint32_t m)
{
    m = __vmaxu2(m, v.x & 0x7fff7fffu);
    m = __vmaxu2(m, v.y & 0x7fff7fffu);
    m = __vmaxu2(m, v.z & 0x7fff7fffu);
    return __vmaxu2(m, v.w & 0x7fff7fffu);
}

// Values that are not finite -> NaN; the largest magnitude of the others.
__device__ __forceinline__ float clean8(float (&x)[8], float m)
{
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (fabsf(x[k]) <= 3.4028234663852886e38f)
            m = fmaxf(m, fabsf(x[k]));
        else
            x[k] = NAN;
    }
    return m;
}

// Items of the 8-bit append: a sequence's new tokens touch at most n / bs + 2
// blocks; with token_starts the items of sequence b are numbered from
// starts[b] / bs + 2 b (strictly increasing, and far enough apart for those
// blocks: floor(x + n) - floor(x) >= floor(n)), else per sequence alike.
__host__ __device__ inline int items_per_seq(int q_len, int bs) { return (q_len + bs - 2) / bs + 1; }

// 16 codes of an earlier token's row, from scale `old` to scale `now`.
__device__ __forceinline__ void requantise(uint2 *at, float old, float now)
{
    if (now == old)
        return;
    uint4 *const q = reinterpret_cast<uint4 *>(at);
    const uint4 v = *q;
    const float f = old / now;
    float x[8];
    from_e4m3x8(make_uint2(v.x, v.y), x);
    const uint2 a = to_e4m3x8(x, f);
    from_e4m3x8(make_uint2(v.z, v.w), x);
    const uint2 b = to_e4m3x8(x, f);
    *q = make_uint4(a.x, a.y, b.x, b.y);
}

// One CTA per item and `heads` KV heads, block_size * head_dim / 16 threads: thread
// = (row of the block, pair of chunks).  CTAs past those rotate one token's query
// rows each.  Several heads a CTA (MANY) save the chain of loads that finds the block
// (and the angles): prompts run 8 at a time, the next head's rows loaded while this
// one's maxima are found; few tokens one head, so that their CTAs fill the GPU (see
// launch_append_q8).
template <typename T, bool WIDE, bool MANY>
__global__ void __launch_bounds__(WIDE ? 1024 : 256, WIDE ? 1 : MANY ? 3 : 4)
    append_q8_kernel(const AppendParams p, int kv_ctas, int heads, int block_shift, int item_shift)
{
    using E = Elem<T>;
    __shared__ float s_max[2][64];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31;
    const int u = threadIdx.x & ((1 << item_shift) - 1);
    const int row = threadIdx.x >> item_shift;
    const bool interleaved = p.interleaved != 0;
    const Item rot = item_of(u, p.rotary_dim, interleaved, true);
    const int chunks = p.head_dim / 8;
    float c[8] = {}, s[8] = {};

    if ((int)blockIdx.x >= kv_ctas) {
        // ---- one token's query rows
        const int t = blockIdx.x - kv_ctas;
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) +
                                                         t * p.query_stride);
        uint4 *qo = reinterpret_cast<uint4 *>(static_cast<T *>(p.query_out) +
                                              t * p.query_out_stride);
        const int step = blockDim.x >> item_shift;
        bool placed = false;
        for (int base = row; base - row < p.num_heads; base += 2 * step) {
            uint4 x0[2], x1[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (base + i * step < p.num_heads) {
                    x0[i] = q[(base + i * step) * chunks + rot.c0];
                    x1[i] = q[(base + i * step) * chunks + rot.c1];
                }
            if (!placed) {
                placed = true;
                int b, pos, angle;
                if (!place_of<false>(p, t, lane, false, &b, &pos, &angle))
                    return;
                if (p.rotary_dim)
                    load_angles(p.cos_sin + (size_t)angle * p.rotary_dim, rot, p.rotary_dim,
                                interleaved, c, s);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (base + i * step < p.num_heads) {
                    if (rot.rot0 || rot.rot1) {
                        float a[8], d[8];
                        unpack8<T>(x0[i], a);
                        unpack8<T>(x1[i], d);
                        rotate_item(a, d, rot, interleaved, c, s);
                        x0[i] = pack8<T>(a);
                        x1[i] = pack8<T>(d);
                    }
                    qo[(base + i * step) * chunks + rot.c0] = x0[i];
                    qo[(base + i * step) * chunks + rot.c1] = x1[i];
                }
        }
        return;
    }

    // ---- one block of `heads` KV heads, one after another
    const int splits = MANY ? (p.num_kv_heads + heads - 1) / heads : p.num_kv_heads;
    const int item = blockIdx.x / splits;
    const int kv0 = ((int)blockIdx.x - item * splits) * (MANY ? heads : 1);
    const int kv1 = MANY ? min(kv0 + heads, p.num_kv_heads) : kv0 + 1;
    const int bs = 1 << block_shift;
    Seq q;
    int j;
    if (p.token_starts) {
        auto first_item = [&](int i, int start) { // (as start / bs + 2 i, for any start)
            return (long long)(start < 0 ? -(-start >> block_shift) : start >> block_shift) + 2LL * i;
        };
        if (!find_seq(p, item, lane, first_item, q))
            return;
        j = item - (int)first_item(q.b, q.begin);
    } else {
        const int per = items_per_seq(p.q_len, bs);
        q.b = item / per;
        j = item - q.b * per;
        q.begin = q.b * p.q_len;
        q.end = q.begin + p.q_len;
        q.len = __ldg(p.seq_lens + q.b);
    }
    const int b = q.b, begin = q.begin, end = q.end;
    if (begin >= end || j < 0)
        return;
    const bool reporter = threadIdx.x == 0 && kv0 == 0;
    if (begin < 0 || end > p.num_tokens) {
        if (reporter)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        return;
    }
    // Positions fit 32 bits (a table's do), end - begin is at most num_tokens.
    const int L = q.len;
    const int cap = p.max_blocks << block_shift;
    const long long first = (long long)L - (end - begin); // position of the first new token
    if (first < 0 || L > cap) {
        if (reporter && j == 0)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
    }
    // Positions written: from `first` (0 when negative) up to L, the table's
    // and the rotation table's ends.
    const int lo_pos = first < 0 ? 0 : (int)first;
    int hi_pos = min(L, cap);
    if (p.rotary_dim && hi_pos > p.max_positions) {
        if (reporter && j == 0)
            set_status(p.status, PA_STATUS_BAD_POSITION);
        hi_pos = p.max_positions;
    }
    const int blk = (lo_pos >> block_shift) + j; // logical block
    if (lo_pos >= hi_pos || blk > (hi_pos - 1) >> block_shift)
        return;
    const int p0 = blk << block_shift;           // its first position
    const int new_lo = max(lo_pos - p0, 0);      // rows [new_lo, new_hi) are new
    const int new_hi = min(hi_pos - p0, bs);
    const int32_t block = __ldg(p.block_tables + (size_t)b * p.max_blocks + blk);
    if (block < 0 || block >= p.num_blocks) {
        if (reporter)
            set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
        return;
    }
    const bool is_new = row >= new_lo && row < new_hi;
    const size_t slot0 = (size_t)block * p.num_kv_heads;
    // This thread's two chunks of K and of V.
    const Item raw = item_of(u, 0, false, false);
    const uint4 *ksrc = nullptr, *vsrc = nullptr;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    if (is_new) {
        const int t = begin + (int)(p0 + row - first);
        ksrc = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key) + t * p.key_stride) + kv0 * chunks;
        vsrc = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.value) + t * p.value_stride) +
               kv0 * chunks;
        k0 = __ldcs(ksrc + rot.c0);
        k1 = __ldcs(ksrc + rot.c1);
        v0 = __ldcs(vsrc + raw.c0);
        v1 = __ldcs(vsrc + raw.c1);
        if (p.rotary_dim)
            load_angles(p.cos_sin + (size_t)(p0 + row) * p.rotary_dim, rot, p.rotary_dim,
                        interleaved, c, s);
    }
    const int warps = blockDim.x >> 5;
    for (int kv = kv0; kv < kv1; ++kv) {
        const size_t slot = slot0 + kv;
        // Rows below new_lo hold earlier tokens: their scale is a floor.  Plain loads, which
        // stay before the barrier behind which thread 0 writes the slot.
        const float old_k = new_lo > 0 ? p.k_scales[slot] : 0.f;
        const float old_v = new_lo > 0 ? p.v_scales[slot] : 0.f;
        float a[8], d[8];
        unpack8<T>(k0, a);
        unpack8<T>(k1, d);
        if (rot.rot0 || rot.rot1)
            rotate_item(a, d, rot, interleaved, c, s);
        const uint4 w0 = v0, w1 = v1;
        if (MANY && is_new && kv + 1 < kv1) {
            ksrc += chunks;
            vsrc += chunks;
            k0 = __ldcs(ksrc + rot.c0);
            k1 = __ldcs(ksrc + rot.c1);
            v0 = __ldcs(vsrc + raw.c0);
            v1 = __ldcs(vsrc + raw.c1);
        }
        float mk = amax8(d, amax8(a, 0.f));
        const uint32_t vb = amax8_bits<T>(w1, amax8_bits<T>(w0, 0u));
        // (an infinity or NaN widens to one)
        float mv = E::lo(max(vb & 0xffffu, vb >> 16));
        float *const sm = s_max[kv & 1]; // the head before may still be reading the other half
        // The CTA's maxima; magnitudes order as their bits, NaN last.
        auto over_cta = [&]() {
            mk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(mk))));
            mv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(mv))));
            if (lane == 0) {
                sm[threadIdx.x >> 5] = mk;
                sm[32 + (threadIdx.x >> 5)] = mv;
            }
            __syncthreads();
            mk = lane < warps ? sm[lane] : 0.f;
            mv = lane < warps ? sm[32 + lane] : 0.f;
            mk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mk)));
            mv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mv)));
        };
        over_cta();
        float x[8], y[8];
        unpack8<T>(w0, x);
        unpack8<T>(w1, y);
        if (!(mk <= 3.4028234663852886e38f && mv <= 3.4028234663852886e38f)) {
            // Some value is not finite: it becomes e4m3's NaN, beside the scale of the others.
            mk = clean8(d, clean8(a, 0.f));
            mv = clean8(y, clean8(x, 0.f));
            __syncthreads(); // everyone has read the maxima
            over_cta();
        }
        const float sk = fmaxf(scale_of(mk), old_k), sv = fmaxf(scale_of(mv), old_v);
        if (threadIdx.x == 0) {
            p.k_scales[slot] = sk;
            p.v_scales[slot] = sv;
        }
        const size_t at = ((slot << block_shift) + row) * p.head_dim;
        uint2 *kd = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.key_cache) + at);
        uint2 *vd = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.value_cache) + at);
        if (is_new) {
            // x / s is x times an exact power of two for the scales this writes; under an
            // old one that is none, the reciprocal's rounding would decide ties.
            float fk = 1.f / sk, fv = 1.f / sv;
            if (((__float_as_uint(sk) | __float_as_uint(sv)) & 0x7fffffu) != 0u) {
                divide8(a, sk);
                divide8(d, sk);
                divide8(x, sv);
                divide8(y, sv);
                fk = fv = 1.f;
            }
            kd[rot.c0] = to_e4m3x8(a, fk);
            kd[rot.c1] = to_e4m3x8(d, fk);
            const uint2 e = to_e4m3x8(x, fv), f = to_e4m3x8(y, fv);
            *reinterpret_cast<uint4 *>(vd + raw.c0) = make_uint4(e.x, e.y, f.x, f.y);
        } else if (row < new_lo) {
            requantise(kd + raw.c0, old_k, sk);
            requantise(vd + raw.c0, old_v, sv);
        }
    }
}

} // namespace

cudaError_t launch_append(int dtype, const AppendParams &p, cudaStream_t stream)
{
    void *args[] = {const_cast<AppendParams *>(&p)};
    return dtype == PA_BF16 ? launch_pdl(&append_kernel<__nv_bfloat16>, (unsigned)p.num_tokens,
                                         kAppendThreads, stream, args)
                            : launch_pdl(&append_kernel<__half>, (unsigned)p.num_tokens,
                                         kAppendThreads, stream, args);
}

static long long append_q8_items(const AppendParams &p)
{
    return p.token_starts ? (long long)p.num_tokens / p.block_size + 2LL * p.num_seqs
                          : (long long)p.num_seqs * items_per_seq(p.q_len, p.block_size);
}

long long append_q8_ctas(const AppendParams &p)
{
    return append_q8_items(p) * p.num_kv_heads + (p.num_heads ? p.num_tokens : 0);
}

constexpr int kMaxHeads = 8; // KV heads of a CTA at most
// Tokens per SM from which queries get their own launch: prompts (some 430 per SM) 404
// us, 445 in one launch; two chunks (27 per SM) 24.4 us, 18.7 in one launch.
constexpr int kApartTokens = 60;

static int log2_of(int x) // of a power of two
{
    int n = 0;
    while (1 << n < x)
        ++n;
    return n;
}

cudaError_t launch_append_q8(int dtype, const AppendParams &p, int num_sms, cudaStream_t stream)
{
    // KV heads of a CTA: as many as leave some eight CTAs per SM (counting the items
    // that hold tokens: at most every block of a prompt, and one per sequence).
    const long long items = append_q8_items(p);
    const long long used = (long long)p.num_tokens / p.block_size + p.num_seqs;
    int heads = (int)(used * p.num_kv_heads / (8LL * num_sms));
    heads = heads < 1 ? 1 : heads > kMaxHeads ? kMaxHeads : heads;
    heads = heads > p.num_kv_heads ? p.num_kv_heads : heads;
    const int splits = (p.num_kv_heads + heads - 1) / heads;
    // Many tokens' queries go to the 16-bit kernel behind this one (more of them in
    // flight); few share this launch.
    const bool apart = p.num_heads && p.num_tokens >= kApartTokens * num_sms;
    int kv_ctas = (int)(items * splits);
    int block_shift = log2_of(p.block_size), item_shift = log2_of(p.head_dim / 16);
    void *args[] = {const_cast<AppendParams *>(&p), &kv_ctas, &heads, &block_shift, &item_shift};
    const unsigned threads = (unsigned)(p.block_size * p.head_dim / 16);
    const unsigned grid = (unsigned)(kv_ctas + (p.num_heads && !apart ? p.num_tokens : 0));
    auto launch = [&](auto wide, auto many) {
        return dtype == PA_BF16
                   ? launch_pdl(&append_q8_kernel<__nv_bfloat16, wide.value, many.value>, grid, threads, stream, args)
                   : launch_pdl(&append_q8_kernel<__half, wide.value, many.value>, grid, threads, stream, args);
    };
    const std::true_type yes;
    const std::false_type no;
    const cudaError_t e = threads <= 256 ? heads > 1 ? launch(no, yes) : launch(no, no)
                          : heads > 1    ? launch(yes, yes)
                                         : launch(yes, no);
    if (e != cudaSuccess || !apart)
        return e;
    AppendParams q = p;
    q.num_kv_heads = 0;
    return launch_append(dtype, q, stream);
}

} // namespace pa
