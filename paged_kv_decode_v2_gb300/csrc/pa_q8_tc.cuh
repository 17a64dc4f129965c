// pa_q8_tc.cuh -- attention over a paged cache held in 8 bits (e4m3) with one
// fp32 scale per (block, KV head) for K and for V, on the tcgen05 tensor
// cores: phase 1 of split-K decode ("V2") and the single-pass form ("V1"),
// for one new token or many.
//
//     s_t = scale * ks[blk(t)] * <q, kq_t>,    out = sum_t softmax(s)_t vs[blk(t)] vq_t
//
// Bound by reading the cache up to about a hundred query rows per KV head, at
// half the bytes of a 16-bit one.  The codes go into the tensor cores as they
// are (kind::f8f6f4): nothing is converted, and the arithmetic per cache byte
// is the query rows' alone.  Tokens are the M side, NR query rows of one KV
// head the N side, 128 tokens a tile:
//
//   S[token, (k, row)]   = K_tile Q_k^T     A = K tile as TMA writes it; B = Q in
//                          PL e4m3 parts, part k in its own NR columns
//   P                    = one thread per token: s from its parts' columns,
//                          scaled by its own block's ks, exponentiated, split
//                          into four e5m2 parts, written as its row of B
//   O[dim, (k, row)]    += V_tile^T P_k     A = V tile (M = dims: MN-major),
//                          B = P (MN-major), part k in its own NR columns
//
// Since a thread owns a token, its scales and its mask are its own registers,
// no reduction crosses lanes in the loop, and l is summed once at the end.
//
// Parts.  A query row is scaled by the power of two that brings its largest
// value to [2^7, 2^8) and held as x = x_0 + x_1 / 16 + x_2 / 256, x_k the e4m3
// rounding of 16 times what x_(k-1) left: two parts hold bf16's 8 significant
// bits, three binary16's 11, exactly down to 2^-6 of that scale (and to 2^-14,
// 2^-18 absolute below); the parts' products meet in fp32.  A weight is rounded
// to binary16 (2^-11 of itself) and then split without error, w = w_0 + w_1 / 8 +
// w_2 / 64 + w_3 / 512: e5m2 is binary16's upper byte, so each of the four parts is
// the upper byte of 8 times what the part before it left (3 + 3 + 3 + 2 bits; what a
// part leaves is below a quarter of its power of two, so that 8 times it stays within
// the weights' bound of 2^15, and e5m2's smallest step, 2^-16, is 2^-25 of w_3).  Weights
// of 1 are stored as 2^11: those below 2^-25 of them are binary16's subnormals, off by at
// most 2^-36.
//
// V's scales go into the softmax's exponent.  With r the largest V scale of the
// CTA's range and lv_t = log2(vs_t / r), floored at -60,
//     w_t = 2^(s_t + lv_t - M),   O = sum w_t vq_t,   l = sum w_t 2^(-lv_t),
// s in log2 units: O / l * r is the output.  M bounds the weighted exponents, so
// P's rounding is relative to the largest contribution, whatever the blocks'
// scales.  M moves only when a weight would pass 2^4 (the first tile always);
// O is rescaled in tensor memory only then.  l and M are a valid pair for the
// merge: l = sum 2^(s_t - M).
//
// Warp roles: warpgroups of softmax warps (16 rows each at most; thread = token
// = TMEM lane, and dim in the epilogue), one warp that issues the MMAs of S (and
// owns the tensor memory), one that issues those of P.V, two or four that issue
// the TMA loads.  S and P have two buffers where tensor memory allows (else one):
// S of tile t + 2 is issued once the softmax has read S of tile t.
//
// Rows beyond NR go to more CTAs, tokens are cut into partitions (V2) or over a
// cluster (V1, joined through distributed shared memory).  Where CTAs queue they
// take units of work in order of size.
//
// Measured on a GB300 (us a call, and its bytes as a share of the measured copy
// bandwidth): 32 sequences of up to 8192 tokens, 32 heads on 8: 45-49 (82%); one of
// 100,000 tokens on 4 KV heads: 22.6 (67%); 64 of up to 32,768, 64 heads on 8: 71-80
// (its own 497 MB in 73: 100%); 8 of 131,072: 321-324 (98%); one of 1000: 6.7, latency.
// 16 new tokens for 32 sequences: 83-86 (48%), bound by the softmax warps: some 400
// instructions a warp and tile, about 160 of them arithmetic, more than half of that the
// parts of P and Q (the factors between P's parts 2-3% of the time).
//
// Built and measured slower: the same work on mma.sync (16 new tokens 278); equal
// stretches of tiles over a fixed grid (16 new tokens 166 where partitions took
// 121, ragged 96 and 89); 32 rows a softmax warpgroup (100 and 92); two CTAs of 32
// rows for 64 (107 and 92); waits that spin, or suspend at the first try (96 and 92).
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_q8.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr float kQ8Ln2 = 0.69314718055994531f;
// M before a row has seen a token: the lowest finite value, so that any score moves it.
constexpr float kQ8NoMax = -3.4028234663852886e38f;
constexpr float kQ8Grow = 4.f;     // weights stay <= 2^4,
constexpr float kQ8Unit = 11.f;    // stored times 2^11: <= 2^15 (e5m2's largest is 1.75 * 2^15)
constexpr float kQ8Floor = -60.f;  // of log2(vs / r)

// ---------------------------------------------------------------- primitives

// Two e4m3 codes (the low half of x) -> two binary16 values.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t x)
{
    uint32_t y;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t h2_times8(uint32_t a)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x48004800u));
    return r;
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float fast_log2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Shared-memory matrix descriptor with 128-, 64- or 32-byte swizzle (see
// smem_desc_sw128; the mode field is 2, 4 or 6, and an atom 8 rows of that width).
template <int WIDTH>
__device__ __forceinline__ uint64_t smem_desc_sw(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    uint64_t d = (uint64_t)((addr >> 4) & 0x3fffu);
    d |= (uint64_t)((lbo >> 4) & 0x3fffu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3fffu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(WIDTH == 128 ? 2 : WIDTH == 64 ? 4 : 6) << 61;
    return d;
}

// Instruction descriptor of kind::f8f6f4 with an fp32 accumulator, A e4m3
// (format 0) and B e4m3 or e5m2 (format 1); fields as in idesc_f16, bit 15 = A
// MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, bool b_e5m2, bool mn_major)
{
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((mn_major ? 3u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem], 8-bit operands, K = 32; one thread issues it.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// 8 or 16 consecutive columns of this thread's TMEM lane; valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld(uint32_t ta, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(ta)
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t ta, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t ta, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(ta)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// Waits for this thread's tcgen05.ld; the array is an operand so that no use
// of its values moves before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7])::"memory");
}

__device__ __forceinline__ void mbar_inval(uint32_t bar)
{
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// mbar_wait_abortable for a warp: true in all lanes or in none.  The loop is a function
// of its own: a copy at every wait crowded the instruction cache (16 new tokens 91.7
// us, 89.1 without).
static __device__ __noinline__ bool warp_wait_loop(uint32_t bar, uint32_t parity, const volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait_abortable(bar, parity, abort));
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int *abort)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    return warp_wait_loop(bar, parity, abort);
}

// Barrier over `count` threads (a multiple of the warp size), and one that
// also ORs a predicate over them.
__device__ __forceinline__ void bar_sync(int id, int count)
{
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_any(int id, int count, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(count), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

// ---- thread-block clusters: all threads of all CTAs meet; a peer's shared memory
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// An int whose order is the float's (no NaN), and back.
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i)
{
    return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff);
}

// 2^k and 2^-k for the power of two that brings a row whose largest magnitude
// is amax to [2^7, 2^8) (k limited to keep both finite).
__device__ __forceinline__ void q_row_scale(float amax, float &f, float &inv)
{
    const int e = (int)(__float_as_uint(amax) >> 23); // biased exponent
    const int fe = amax > 0.f ? min(127 + 7 - (e - 127), 253) : 127;
    f = __uint_as_float((uint32_t)fe << 23);
    inv = __uint_as_float((uint32_t)(254 - fe) << 23);
}

// V1 over a cluster: the CTAs' partials of the same rows (o normalised, l, M in log2
// units; M = -inf, l = 0 without a token) -> out.  `o_sm` [NR][D] and `ml` [2][NR] in
// every CTA's shared memory; each CTA joins every ways-th four values.  All threads
// of the CTA call it, its partial written and synchronised.
template <int D, int NR, typename T, typename RowOf>
__device__ __forceinline__ void join_cluster(uint32_t o_sm, uint32_t ml, int rank, int ways, int nrows,
                                             T *out, RowOf row_of)
{
    using E = Elem<T>;
    cluster_sync();
    for (int i = threadIdx.x * ways + rank; i < nrows * (D / 4); i += blockDim.x * ways) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float m[kQ8Ways], l[kQ8Ways], top = -INFINITY;
        float4 o[kQ8Ways];
#pragma unroll
        for (int w = 0; w < kQ8Ways; ++w) {
            const int from = w < ways ? w : rank;
            m[w] = ld_peer(peer_addr(ml + 4 * r, from));
            l[w] = w < ways ? ld_peer(peer_addr(ml + 4 * (NR + r), from)) : 0.f;
            o[w] = ld_peer4(peer_addr(o_sm + (r * D + d) * 4, from));
            top = fmaxf(top, m[w]);
        }
        float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kQ8Ways; ++w) {
            if (!(l[w] == 0.f)) { // (an empty one's o may be anything)
                const float f = l[w] * fast_exp2(m[w] - top);
                sum += f;
                x[0] += f * o[w].x;
                x[1] += f * o[w].y;
                x[2] += f * o[w].z;
                x[3] += f * o[w].w;
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint32_t *const dst = reinterpret_cast<uint32_t *>(out + row_of(r) * D + d);
        dst[0] = E::pack(x[0] * inv, x[1] * inv);
        dst[1] = E::pack(x[2] * inv, x[3] * inv);
    }
    cluster_sync(); // the peers have read this CTA's part
}

// ---------------------------------------------------------------- shape

template <int D, int NR, int PL>
struct Q8Cfg {
    static constexpr int kRB = D < 128 ? D : 128;                 // bytes of a K/V row in one slice
    static constexpr int kSlices = D / kRB;
    static constexpr uint32_t kSlice = kQ8Tok * kRB;              // one slice of a K or V tile
    static constexpr uint32_t kTile = kQ8Tok * D;
    static constexpr int kSN = (NR * PL + 15) / 16 * 16;          // columns of S (N of its MMA)
    static constexpr int kPN = NR * 4;                            // of P, and of O per 128 dims
    static constexpr int kMB = D == 256 ? 2 : 1;                  // 128-dim halves of O
    // TMEM columns, in regions of 32: O's halves, then the S buffers.
    static constexpr int kOReg = (kPN + 31) / 32 * 32;
    static constexpr int kSReg = (kSN + 31) / 32 * 32;
    // CTAs that share an SM: registers (by the launch bounds), tensor memory (below) and
    // shared memory (launch_tc's rings) are each cut to it.  32 binary16 rows: one S buffer
    // for two CTAs, batch decode lengths 70 us, one CTA with two buffers 74 (100,000 tokens
    // 41 and 50; 300 sequences of up to 700 41 and 52; 32 rows of one new token over 100,000
    // 77 and 72).
    static constexpr int kCtas = NR <= 32 && D <= 128 ? 2 : 1;
    static constexpr int kBuf = kOReg * kMB + 2 * kSReg <= 512 / kCtas ? 2 : 1; // S and P buffers
    static constexpr int kNeed = kOReg * kMB + kBuf * kSReg;
    static constexpr uint32_t kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static constexpr uint32_t kSCol = kOReg * kMB;
    static_assert(kCtas * kCols <= 512, "the CTAs of an SM exceed its tensor memory");
    static_assert(NR * D * 4 <= 2 * kTile, "a cluster's partials lie in the smallest rings");
    static constexpr int kPW = kPN <= 32 ? 32 : kPN <= 64 ? 64 : 128; // bytes of P's rows, and
    static constexpr int kPGroups = (kPN + kPW - 1) / kPW;        // groups of that many columns
    static constexpr uint32_t kPGroup = kQ8Tok * kPW;
    static constexpr uint32_t kPBytes = kPGroups * kPGroup;
    static constexpr uint32_t kQBytes = kSN * D;
    static constexpr int kRW = NR < 16 ? NR : 16;                 // rows of a softmax warpgroup
    static constexpr int kWG = NR / kRW;
    static constexpr int kChap = kWG * 128 < 256 ? 256 : kWG * 128; // blocks whose scales are held at a time
    static constexpr int kSoft = kWG * 128;
    // Producer warps: two for K and two for V, or one each from 16 rows on, where a tile
    // lasts longer and the softmax warps want the registers (16 new tokens 104 us, 121
    // with four; at 8 rows 100k tokens 22.0, 22.7 with two).
    static constexpr int kLoad = NR <= 8 ? 4 : 2;
    static constexpr int kThreads = kSoft + 64 + 32 * kLoad;
    static constexpr uint32_t kFixed = 1024 + kBuf * kPBytes + kQBytes;
};

// The work of CTA `bid` of the grid that p describes; false after a wait that gave up.
// LOOP: one of several that a CTA takes, its barriers gone at the end.
template <int D, int NR, int PL, bool V1, bool LOOP>
__device__ __forceinline__ bool q8_unit(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                                        const Q8Params &p, int bid)
{
    using C = Q8Cfg<D, NR, PL>;
    using T = typename std::conditional<PL == 2, __nv_bfloat16, __half>::type;
    using E = Elem<T>;
    constexpr int kRW = C::kRW;
    constexpr int kMmaWarp = C::kSoft / 32, kTmaWarp = kMmaWarp + 2;

    __shared__ uint64_t k_full[kMaxStages], v_full[kMaxStages], k_empty[kMaxStages],
        v_empty[kMaxStages];
    __shared__ uint64_t s_full[2], p_full[2], o_done[2], drained[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ __align__(16) float s_cf[NR];   // a row's raw products -> log2 units (but for ks)
    __shared__ __align__(16) float s_nm[NR];   // kQ8Unit - M
    __shared__ float s_al[NR];                 // 2^(M_old - M_new)
    __shared__ float s_inv[NR];                // r / l
    __shared__ size_t s_row[NR];               // rows of out, or slots of the intermediates
    __shared__ float s_ml[2 * NR];             // a cluster's join: M and l
    __shared__ int s_red[C::kSoft / 32][kRW];
    __shared__ float s_part[C::kSoft / 32][kRW];
    __shared__ float s_vref[C::kSoft / 32];
    __shared__ float s_ks[C::kChap], s_lv[C::kChap], s_rl[C::kChap]; // a chapter's ks, lv, 2^-lv
    extern __shared__ uint8_t dyn_smem[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // bid = ((unit * KV + KV head) * row tiles + row tile) * ways + rank: units are
    // partitions of sequences (V1: sequences, the `ways` CTAs of a cluster their
    // partitions); row tiles of one KV head are neighbours, so that their reads meet
    // in L2.
    const int ways = V1 ? p.ways : 1;
    int unit = V1 ? bid / ways : bid;
    int part = V1 ? bid % ways : 0;
    int rt = 0;
    if (p.col_groups > 1) {
        rt = unit % p.col_groups;
        unit /= p.col_groups;
    }
    const int kv = unit % p.num_kv_heads;
    unit /= p.num_kv_heads;
    const bool reporter = kv == 0 && rt == 0 && (!V1 || part == 0);
    auto length = [&](int at, bool report) -> int {
        const int len = __ldg(p.seq_lens + at);
        if (len >= 0 && len <= p.seq_len_cap)
            return len;
        if (report)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        return len < 0 ? 0 : p.seq_len_cap;
    };
    int b, L;
    if (p.sorted) {
        // Units by the tokens they hold, whole partitions first, then the rest of each
        // sequence (V1: each sequence) in 32 classes of size, so that no long one is
        // left for the end.  Every CTA sorts: thread = sequence.
        constexpr int kWarps = C::kThreads / 32;
        static_assert(C::kThreads >= kQ8Sorted, "a thread holds one sequence");
        __shared__ int s_count[kWarps][32]; // sequences of each class, by warp
        __shared__ int s_whole[kWarps];     // whole partitions
        __shared__ int s_pick[3];
        const int at = threadIdx.x;
        const int len = at < p.num_seqs ? length(at, reporter && unit == 0) : 0;
        const int size = V1 ? p.seq_len_cap : p.partition_size;
        const int parts = V1 ? 0 : len / size; // whole ones
        const int rest = len - parts * size;
        int cls = -1; // 0 (largest) to 31; none without a unit
        if (V1 ? at < p.num_seqs : rest > 0)
            cls = min((int)((float)(size - rest) * p.class_scale), 31);
        s_count[warp][lane] = 0;
        if (threadIdx.x == 0)
            s_pick[0] = -1;
        __syncwarp();
        const uint32_t peers = __match_any_sync(0xffffffffu, cls);
        const int ahead = __popc(peers & ((1u << lane) - 1u));
        if (cls >= 0 && ahead == 0)
            s_count[warp][cls] = __popc(peers);
        int run = parts; // inclusive scan
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, off);
            run += lane >= off ? v : 0;
        }
        if (lane == 31)
            s_whole[warp] = run;
        __syncthreads();
        const int used = (p.num_seqs + 31) / 32; // warps that hold sequences
        int total = 0, start = run - parts, count = 0, before = 0;
        for (int w = 0; w < used; ++w) {
            const int n = s_whole[w], c = s_count[w][lane];
            total += n;
            start += w < warp ? n : 0;
            count += c;
            before += w < warp ? c : 0;
        }
        int up = count; // of this lane's class and those ahead of it
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, up, off);
            up += lane >= off ? v : 0;
        }
        const int first = __shfl_sync(0xffffffffu, total + up - count + before, cls & 31) + ahead;
        const bool in_whole = unit >= start && unit - start < parts;
        if (in_whole || (cls >= 0 && unit == first)) {
            s_pick[0] = at;
            s_pick[1] = in_whole ? unit - start : parts;
            s_pick[2] = len;
        }
        __syncthreads();
        b = s_pick[0];
        if (b < 0)
            return true; // past the last unit
        part = s_pick[1];
        L = s_pick[2];
    } else if (V1) {
        b = unit;
    } else {
        b = unit / p.num_parts;
        part = unit - b * p.num_parts;
    }

    const int tokA = part * p.partition_size;
    const int sh = p.block_shift, bs = 1 << sh; // block size
    const int bpt = kQ8Tok >> sh;               // blocks per tile: 2 to 16
    const int blk0 = tokA >> sh;
    const int32_t *bt = p.block_tables + (size_t)b * p.max_blocks + blk0;
    // A producer warp loads all or half the blocks of every K or V tile: one warp
    // issuing all of a tile's TMA loads (16 at 16-token blocks, 40-80 clocks each)
    // would bound the loop of few rows.
    constexpr int kSplit = C::kLoad / 2; // producer warps of one tile
    const int pw = warp - kTmaWarp;
    const bool is_k = pw < kSplit;
    const int p_num = bpt / kSplit, p_first = pw % kSplit * p_num; // its blocks of a tile
    // The table's first entries, loaded beside the length: block threadIdx.x of a
    // softmax thread, a producer lane's block of the first tile.
    int32_t id_first = 0;
    const int at_first = warp < kTmaWarp ? (int)threadIdx.x : p_first + lane;
    if ((warp < kMmaWarp || (warp >= kTmaWarp && lane < p_num)) && blk0 + at_first < p.max_blocks)
        id_first = __ldg(bt + at_first);
    if (!p.sorted)
        L = length(b, reporter && part == 0 && threadIdx.x == 0);
    if (!V1 && tokA >= L)
        return true; // partition past the end of the sequence: nothing to write
    const bool whole = V1 || L <= p.partition_size; // the output itself, no partials

    // Rows [c0, c0 + nrows) of the KV head's cols = q_len * group rows.
    const int c0 = rt * NR;
    const int nrows = min(NR, p.cols - c0);
    // c / group: c < 2^18 and group <= 64, so that the multiplier's excess stays below 1.
    auto new_token = [&](int c) -> int {
        return p.group == 1 ? c : (int)__umulhi((uint32_t)c, p.group_inv);
    };
    const int i_last = p.q_len == 1 ? 0 : new_token(c0 + nrows - 1);
    auto row_of = [&](int r) -> size_t { // row of [S * q_len * H] of local row r
        const int c = c0 + r;
        const int i = p.q_len == 1 ? 0 : new_token(c);
        return (size_t)(b * p.q_len + i) * p.num_heads + (kv * p.group + c - i * p.group);
    };
    // Tokens the CTA needs: [tokA, tokE), the range cut by the causal limit of
    // its last new token (new token i sees positions <= L - q_len + i).
    long long e = ways == 1 && V1 ? (long long)L : min((long long)L, (long long)tokA + p.partition_size);
    e = min(e, (long long)L - p.q_len + i_last + 1);
    const int tokE = (int)e;
    const int tok0 = blk0 << sh;
    const int ntiles = tokE > tokA ? (tokE - tok0 + kQ8Tok - 1) / kQ8Tok : 0;
    const int nblk = tokE > tokA ? (tokE - tok0 + bs - 1) >> sh : 0;

    const uint32_t smem0 = (smem_addr(dyn_smem) + 1023u) & ~1023u;
    if (ntiles == 0) {
        // No row sees a token of the range: an empty partition (m = -inf,
        // l = 0, o = 0), or a zero output.
        if (V1 && ways > 1) {
            if (threadIdx.x < NR) {
                s_ml[threadIdx.x] = -INFINITY;
                s_ml[NR + threadIdx.x] = 0.f;
            }
            __syncthreads();
            join_cluster<D, NR>(smem0, smem_addr(s_ml), part, ways, nrows, static_cast<T *>(p.out), row_of);
            return true;
        }
        for (int idx = threadIdx.x; idx < nrows * D; idx += C::kThreads) {
            const size_t row = row_of(idx / D);
            if (whole) {
                static_cast<T *>(p.out)[row * D + idx % D] = E::from_float(0.f);
            } else {
                const size_t slot = row * p.max_num_partitions + part;
                p.tmp_output[slot * D + idx % D] = 0.f;
                if (idx % D == 0) {
                    p.exp_sums[slot] = 0.f;
                    p.max_logits[slot] = -INFINITY;
                }
            }
        }
        return true;
    }

    const int kst = p.stages;   // K ring stages
    const int vst = p.v_stages; // V ring stages
    const uint32_t k_sm = smem0;
    const uint32_t v_sm = k_sm + (uint32_t)kst * C::kTile;
    const uint32_t p_sm = v_sm + (uint32_t)vst * C::kTile;
    const uint32_t q_sm = p_sm + C::kBuf * C::kPBytes;
    const uint32_t b_k_full = smem_addr(k_full), b_v_full = smem_addr(v_full);
    const uint32_t b_k_empty = smem_addr(k_empty), b_v_empty = smem_addr(v_empty);
    const uint32_t b_s_full = smem_addr(s_full), b_p_full = smem_addr(p_full);
    const uint32_t b_o_done = smem_addr(o_done), b_drained = smem_addr(drained);
    volatile int *abort_flag = &abort_sh;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&tmem_base_sh), C::kCols);
        if (!LOOP)
            tmem_relinquish();
    }
    int32_t status_bits = 0;
    const int p_stages = is_k ? kst : vst;
    const uint32_t p_full_bar = is_k ? b_k_full : b_v_full, p_empty_bar = is_k ? b_k_empty : b_v_empty;
    const uint32_t p_ring = is_k ? k_sm : v_sm;
    const CUtensorMap *p_map = is_k ? &tmap_k : &tmap_v;
    const uint64_t policy = p.col_groups == 1 ? l2_evict_first_policy() : l2_evict_normal_policy();
    auto fetch_id = [&](int t) -> int32_t { // this lane's block of tile t
        const int i = t * bpt + p_first + lane;
        return lane < p_num && i < nblk ? __ldg(bt + i) : 0;
    };
    auto load_tile = [&](int s, int t, int32_t id) {
        const int nb = min(max(nblk - t * bpt - p_first, 0), p_num);
        if (id < 0 || id >= p.num_blocks) {
            status_bits |= PA_STATUS_BAD_BLOCK_ID;
            id = 0; // read a valid block instead of memory outside the cache
        }
        const uint32_t bar = p_full_bar + 8 * s;
        const uint32_t dst = p_ring + (uint32_t)s * C::kTile + p_first * bs * C::kRB;
        if (lane == 0)
            mbar_arrive_expect_tx(bar, (uint32_t)nb * bs * D);
        const int row = (id * p.num_kv_heads + kv) << sh; // (all rows number less than 2^31)
        for (int i = 0; i < nb; ++i) {
            const int at = __shfl_sync(0xffffffffu, row, i);
            if (lane == 0) {
#pragma unroll
                for (int sl = 0; sl < C::kSlices; ++sl)
                    tma_load_3d(dst + sl * C::kSlice + i * bs * C::kRB, p_map, 0, sl, at, bar, policy);
            }
        }
    };
    if (threadIdx.x == kTmaWarp * 32) {
        for (int s = 0; s < kst; ++s) {
            mbar_init(b_k_full + 8 * s, kSplit);
            mbar_init(b_k_empty + 8 * s, 1);
        }
        for (int s = 0; s < vst; ++s) {
            mbar_init(b_v_full + 8 * s, kSplit);
            mbar_init(b_v_empty + 8 * s, 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(b_s_full + 8 * j, 1);
            mbar_init(b_p_full + 8 * j, C::kSoft);
            mbar_init(b_o_done + 8 * j, 1);
        }
        mbar_init(b_drained, 1);
        mbar_init(b_drained + 8, 1);
        abort_sh = 0;
        mbar_init_fence();
    }
    int issued = 0;          // tiles this producer has issued
    int32_t id_next = 0;     // this lane's block of the next one, fetched ahead of its stage
    if (warp >= kTmaWarp) {
        // The first tiles, before the rest of the set-up.
        bar_sync(15, 32 * C::kLoad); // the barriers are initialised
        id_next = lane < p_num && p_first + lane < nblk ? id_first : 0;
        while (issued < ntiles && issued < p_stages) {
            const int32_t id = id_next;
            id_next = fetch_id(issued + 1);
            load_tile(issued, issued, id);
            ++issued;
        }
    }
    // A block's id, or 0 (a valid block) when out of range.
    auto valid_id = [&](int32_t id) -> int32_t { return id < 0 || id >= p.num_blocks ? 0 : id; };

    float vref = 0.f;                     // the range's largest V scale
    float ks_first = 0.f, vs_first = 0.f; // scales of block threadIdx.x
    if (warp < kMmaWarp) {
        // Q rows -> shared memory in PL parts, K-major, swizzled (16-byte chunk c of
        // row n at c ^ (n & 7), of 64-byte rows c ^ (n >> 1 & 3)); a warp per row.
        constexpr int kDL = D / 32;                 // consecutive dims of a lane: 2, 4 or 8
        constexpr int kRows = NR / (C::kSoft / 32); // rows of a warp
        uint32_t q_raw[kRows][kDL / 2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = warp + i * (C::kSoft / 32);
            const uint32_t *q32 = static_cast<const uint32_t *>(p.query) +
                                  row_of(r < nrows ? r : 0) * (D / 2) + lane * (kDL / 2);
#pragma unroll
            for (int k = 0; k < kDL / 2; ++k)
                q_raw[i][k] = r < nrows ? __ldg(q32 + k) : 0u;
        }
        if ((int)threadIdx.x < nblk) {
            const size_t at = (size_t)valid_id(id_first) * p.num_kv_heads + kv;
            ks_first = __ldg(p.k_scales + at);
            vs_first = __ldg(p.v_scales + at);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = warp + i * (C::kSoft / 32);
            float x[kDL], m = 0.f;
#pragma unroll
            for (int k = 0; k < kDL / 2; ++k) {
                x[2 * k] = E::lo(q_raw[i][k]);
                x[2 * k + 1] = E::hi(q_raw[i][k]);
                m = fmaxf(m, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            float f, inv;
            q_row_scale(m, f, inv);
            if (lane == 0) {
                s_cf[r] = p.scale * inv * kLog2e;
                s_nm[r] = -kQ8NoMax;
                const size_t row = row_of(r < nrows ? r : 0);
                s_row[r] = whole ? row : row * p.max_num_partitions + part;
            }
#pragma unroll
            for (int k = 0; k < kDL; ++k) // a value that is not finite becomes NaN
                x[k] = fabsf(x[k]) <= 3.4028234663852886e38f ? x[k] * f : NAN;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                const int n = k * NR + r;
                const int d = lane * kDL;          // first dim
                const int c = (d % C::kRB) >> 4;   // 16-byte chunk
                const int sw = C::kRB == 128 ? c ^ (n & 7) : c ^ ((n >> 1) & 3);
                const uint32_t dst = q_sm + (d / C::kRB) * (C::kSN * C::kRB) + n * C::kRB +
                                     (sw << 4) + (d & 15);
#pragma unroll
                for (int h = 0; h < kDL / 2; ++h) {
                    const uint32_t code = __nv_cvt_float2_to_fp8x2(
                        make_float2(x[2 * h], x[2 * h + 1]), __NV_SATFINITE, __NV_E4M3);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + 2 * h), "h"((unsigned short)code)
                                 : "memory");
                    const uint32_t back = e4m3_to_f16(code);
                    x[2 * h] = (x[2 * h] - Elem<__half>::lo(back)) * 16.f;
                    x[2 * h + 1] = (x[2 * h + 1] - Elem<__half>::hi(back)) * 16.f;
                }
            }
        }
        fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp >= kTmaWarp) {
        // ---------------------------------------------------------- producers
        int s = 0;
        uint32_t ph = 0u;
        for (; issued < ntiles; ++issued) {
            if (!warp_wait(p_empty_bar + 8 * s, ph, abort_flag)) {
                status_bits |= PA_STATUS_TIMEOUT;
                *abort_flag = 1;
                break;
            }
            load_tile(s, issued, id_next);
            id_next = fetch_id(issued + 1);
            if (++s == p_stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        // Let copies still in flight land before the shared memory is released
        // (normally consumed long ago; bounded).
        for (int t = max(0, issued - p_stages); t < issued; ++t)
            mbar_wait_bounded(p_full_bar + 8 * (t % p_stages), (uint32_t)(t / p_stages) & 1u, kWaitLimitNs);
        __syncwarp();
    } else if (warp >= kMmaWarp) {
        // ---------------------------------------------------------- MMA issuers
        // One warp issues the S MMAs, one the P.V MMAs, each as its operands
        // arrive (an issue takes tens of clocks and a wait a hundred: together
        // they would bound the loop).  Control flow is warp-uniform and one
        // elected lane issues, so that descriptors stay in uniform registers.
        const bool is_s = warp == kMmaWarp;
        // K-major operands: 8-row groups 8 * kRB bytes apart.
        const uint64_t qd = smem_desc_sw<C::kRB>(q_sm, 16, 8 * C::kRB);
        const uint64_t kd = smem_desc_sw<C::kRB>(k_sm, 16, 8 * C::kRB);
        // MN-major: 8-token groups 8 * row bytes apart, P's column groups a
        // tile of rows apart.  head_dim 64: M = 128 spans two 64-dim groups; the
        // second one reads 8 tokens on, into lanes that nothing reads.
        const uint64_t vd = smem_desc_sw<C::kRB>(v_sm, 8 * C::kRB, 8 * C::kRB);
        const uint64_t pd = smem_desc_sw<C::kPW>(p_sm, C::kPGroup, 8 * C::kPW);
        bool ok = true;
        int s = 0; // ring stage of tile t
        uint32_t ph = 0u;
        for (int t = 0; t < ntiles; ++t) {
            const int j = C::kBuf == 2 ? t & 1 : 0;
            if (is_s) {
                // S(t) once K tile t has landed and softmax(t - kBuf) has read the buffer.
                ok = warp_wait(b_k_full + 8 * s, ph, abort_flag) &&
                     (t < C::kBuf || warp_wait(b_p_full + 8 * ((t - C::kBuf) & 1),
                                               (uint32_t)((t - C::kBuf) >> 1) & 1u, abort_flag));
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    constexpr uint32_t idesc = idesc_f8(128, C::kSN, false, false);
                    const uint64_t kb = kd + (((uint32_t)s * C::kTile) >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks) {
                        constexpr int kPer = C::kRB / 32;
                        const uint32_t off_k = (ks / kPer) * C::kSlice + (ks % kPer) * 32;
                        const uint32_t off_q = (ks / kPer) * (C::kSN * C::kRB) + (ks % kPer) * 32;
                        tc_mma_f8(tmem + C::kSCol + j * C::kSReg, kb + (off_k >> 4), qd + (off_q >> 4),
                                  idesc, ks > 0);
                    }
                    tc_commit(b_s_full + 8 * (t & 1));
                    tc_commit(b_k_empty + 8 * s);
                }
                __syncwarp();
                if (++s == kst) {
                    s = 0;
                    ph ^= 1u;
                }
            } else {
                // P.V(t) once P(t) is written and V tile t has landed.
                ok = warp_wait(b_v_full + 8 * s, ph, abort_flag) &&
                     warp_wait(b_p_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    constexpr uint32_t idesc = idesc_f8(128, C::kPN, true, true);
                    const uint64_t vb = vd + (((uint32_t)s * C::kTile) >> 4);
                    const uint64_t pb = pd + ((j * C::kPBytes) >> 4);
#pragma unroll
                    for (int h = 0; h < C::kMB; ++h)
#pragma unroll
                        for (int kt = 0; kt < kQ8Tok / 32; ++kt)
                            tc_mma_f8(tmem + h * C::kOReg, vb + ((h * C::kSlice + kt * 32 * C::kRB) >> 4),
                                      pb + ((kt * 32 * C::kPW) >> 4), idesc,
                                      kt > 0 ? 1u : (t > 0 ? 1u : 0u));
                    tc_commit(b_o_done + 8 * (t & 1));
                    tc_commit(b_v_empty + 8 * s);
                }
                __syncwarp();
                if (++s == vst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) {
            status_bits |= PA_STATUS_TIMEOUT;
            *abort_flag = 1;
        }
        // Every MMA this warp issued has completed once this commit arrives.
        const uint32_t bar = b_drained + (is_s ? 0 : 8);
        if (elect_one())
            tc_commit(bar);
        __syncwarp();
        mbar_wait_bounded(bar, 0, kWaitLimitNs);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        const int wg = warp >> 2;             // rows [wg * kRW, wg * kRW + kRW)
        const int row0 = wg * kRW;
        const int tk = threadIdx.x & 127;     // token of the tile, TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // The range's scales (the first S runs meanwhile): the largest V scale of
        // all, and the first chapter into shared memory.
        auto usable = [](float v) { return v >= 0.f && v <= 3.4028234663852886e38f; };
        vref = fmaxf(vref, usable(vs_first) ? vs_first : 0.f);
        for (int j = threadIdx.x + C::kSoft; j < nblk; j += C::kSoft) {
            const float v = __ldg(p.v_scales + (size_t)valid_id(__ldg(bt + j)) * p.num_kv_heads + kv);
            vref = fmaxf(vref, usable(v) ? v : 0.f);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            vref = fmaxf(vref, __shfl_xor_sync(0xffffffffu, vref, off));
        if (lane == 0)
            s_vref[warp] = vref;
        bar_sync(1, C::kSoft);
#pragma unroll
        for (int w = 0; w < C::kSoft / 32; ++w)
            vref = fmaxf(vref, s_vref[w]);
        const float vref_lg = fast_log2(fmaxf(vref, 1.1754943508222875e-38f)); // (2^-126)
        // Blocks that are not there get ks = 0 and any lv.
        // A V scale that is negative or not finite: weights of NaN for who sees the block.
        auto put_scales = [&](int i, float k, float v) {
            const bool good = usable(v);
            const float lv = good ? fmaxf(fast_log2(v) - vref_lg, kQ8Floor) : NAN;
            s_ks[i] = k;
            s_lv[i] = lv;
            s_rl[i] = good ? fast_exp2(-lv) : 1.f;
        };
        auto load_chapter = [&](int j0, int i0) { // blocks j0 + i, i >= i0
            for (int i = i0 + threadIdx.x; i < C::kChap; i += C::kSoft) {
                float k = 0.f, v = 0.f;
                if (j0 + i < nblk) {
                    const size_t at = (size_t)valid_id(__ldg(bt + j0 + i)) * p.num_kv_heads + kv;
                    k = __ldg(p.k_scales + at);
                    v = __ldg(p.v_scales + at);
                }
                put_scales(i, k, v);
                if (j0 + i >= nblk + bpt)
                    break; // past the last tile
            }
        };
        put_scales(threadIdx.x, ks_first, vs_first);
        load_chapter(0, C::kSoft);
        bar_sync(1, C::kSoft);
        // Rows r >= r_min(token) see the token; a tile that every row sees whole
        // (and that lies inside the range) skips the test.  Positions from tok0
        // (a range is less than 2^31 - 128 tokens long: its tiles' ends fit 32 bits).
        const int rel_a = tokA - tok0, rel_e = tokE - tok0;
        const int rel_q = L - p.q_len - tok0;
        const int rel_all = min(rel_e, rel_q + (p.q_len == 1 ? 0 : new_token(c0)) + 1);
        // Tiles [full_lo, full_hi) are seen whole by every row.
        const int full_lo = (rel_a + kQ8Tok - 1) / kQ8Tok, full_hi = rel_all < 0 ? 0 : rel_all / kQ8Tok;
        uint64_t l2[kRW / 2]; // pairs of rows
#pragma unroll
        for (int r = 0; r < kRW / 2; ++r)
            l2[r] = 0;
        // Where this thread's row of P begins, in the first buffer: 16-byte chunk c of a
        // row lies where the swizzle places it; part k's chunk differs in its own bits.
        constexpr int kPLg = C::kPW == 128 ? 0 : C::kPW == 64 ? 1 : 2;
        const uint32_t prow = p_sm + tk * C::kPW + (((row0 / 16) ^ ((tk >> kPLg) & (C::kPW / 16 - 1))) << 4);
        bool ok = true;
        for (int t = 0; t < ntiles; ++t) {
            const int j = C::kBuf == 2 ? t & 1 : 0;
            if (t > 0 && (t * bpt) % C::kChap == 0) {
                // The next chapter of scales (ranges of more than kChap blocks).
                bar_sync(1, C::kSoft);
                load_chapter(t * bpt, 0);
                bar_sync(1, C::kSoft);
            }
            const int at = (t * bpt + (tk >> sh)) & (C::kChap - 1); // this token's block
            const float ks = s_ks[at], lv = s_lv[at], rl = s_rl[at];
            const bool full = t >= full_lo && t < full_hi;
            // First visible row of this thread's token: new token i = (c0 + r) /
            // group sees it when i >= pos - (L - q_len).
            int r_min = 0;
            if (!full) {
                const int pos = t * kQ8Tok + tk; // from tok0
                const int i0 = pos - rel_q;
                const long long r0 = i0 > 0 ? (long long)i0 * p.group - c0 : 0;
                r_min = pos < rel_a || pos >= rel_e || r0 > NR ? NR : (int)(r0 < 0 ? 0 : r0);
            }

            if (!warp_wait(b_s_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1u, abort_flag))
                ok = false;
            tc_fence_after();
            const uint32_t sc = lane_base + C::kSCol + (uint32_t)j * C::kSReg + row0;
            // Exponents of the stored weights, s + lv + (11 - M); with raw, s + lv.
            uint64_t x[kRW / 2]; // pairs of rows
            auto exponents = [&](bool raw) -> float {
                float top = -INFINITY;
                uint32_t sr[PL][kRW];
#pragma unroll
                for (int k = 0; k < PL; ++k)
                    tmem_ld(sc + k * NR, sr[k]);
#pragma unroll
                for (int k = 0; k < PL; ++k)
                    tmem_wait_ld(sr[k]);
                const uint64_t ks2 = f2_pack(ks, ks), lv2 = f2_pack(lv, lv);
#pragma unroll
                for (int r = 0; r < kRW; r += 4) {
                    const float4 cf = *reinterpret_cast<const float4 *>(s_cf + row0 + r);
                    const float4 nm = *reinterpret_cast<const float4 *>(s_nm + row0 + r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int i = r + 2 * h;
                        uint64_t s = f2_pack(__uint_as_float(sr[PL - 1][i]),
                                             __uint_as_float(sr[PL - 1][i + 1]));
#pragma unroll
                        for (int k = PL - 2; k >= 0; --k)
                            s = f2_fma(s, f2_pack(0.0625f, 0.0625f),
                                       f2_pack(__uint_as_float(sr[k][i]), __uint_as_float(sr[k][i + 1])));
                        const uint64_t add =
                            raw ? lv2 : f2_add(lv2, h ? f2_pack(nm.z, nm.w) : f2_pack(nm.x, nm.y));
                        x[i / 2] = f2_fma(s, f2_mul(ks2, h ? f2_pack(cf.z, cf.w) : f2_pack(cf.x, cf.y)), add);
                    }
                }
                if (!full) {
#pragma unroll
                    for (int r = 0; r < kRW; r += 2) {
                        float x0, x1;
                        f2_unpack(x[r / 2], x0, x1);
                        x[r / 2] = f2_pack(row0 + r >= r_min ? x0 : -INFINITY,
                                           row0 + r + 1 >= r_min ? x1 : -INFINITY);
                    }
                }
#pragma unroll
                for (int r = 0; r < kRW; r += 2) {
                    float x0, x1;
                    f2_unpack(x[r / 2], x0, x1);
                    top = fmax3(top, x0, x1);
                }
                return top;
            };
            if (t == 0 || bar_any(2 + wg, 128, exponents(false) > kQ8Unit + kQ8Grow)) {
                // A weight passes 2^4 in some row: M moves to the rows' maxima over
                // the tile.
                exponents(true);
#pragma unroll
                for (int r = 0; r < kRW; r += 2) {
                    float x0, x1;
                    f2_unpack(x[r / 2], x0, x1);
                    const int m0 = __reduce_max_sync(0xffffffffu, ordered(x0));
                    const int m1 = __reduce_max_sync(0xffffffffu, ordered(x1));
                    if (lane == 0) {
                        s_red[warp][r] = m0;
                        s_red[warp][r + 1] = m1;
                    }
                }
                bar_sync(2 + wg, 128);
                if (tk < kRW) {
                    int m = s_red[wg * 4][tk];
#pragma unroll
                    for (int w = 1; w < 4; ++w)
                        m = max(m, s_red[wg * 4 + w][tk]);
                    const float old = s_nm[row0 + tk];
                    const float now = fminf(old, kQ8Unit - unordered(m));
                    s_nm[row0 + tk] = now;
                    s_al[row0 + tk] = fast_exp2(now - old);
                }
                bar_sync(2 + wg, 128);
                if (t > 0) {
                    // P.V(t - 1) has to land before O is rescaled (tile 0 has no O yet).
                    if (!warp_wait(b_o_done + 8 * ((t - 1) & 1), (uint32_t)((t - 1) >> 1) & 1u, abort_flag))
                        ok = false;
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < 4 * C::kMB; ++k) {
                        const uint32_t oc = lane_base + (k >> 2) * C::kOReg + (k & 3) * NR + row0;
#pragma unroll
                        for (int r8 = 0; r8 < kRW; r8 += 8) {
                            uint32_t o[8];
                            tmem_ld(oc + r8, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                o[r] = __float_as_uint(__uint_as_float(o[r]) * s_al[row0 + r8 + r]);
                            tmem_st(oc + r8, o);
                        }
                    }
                    tmem_st_wait();
                }
#pragma unroll
                for (int r = 0; r < kRW; r += 2)
                    x[r / 2] = f2_add(x[r / 2], f2_pack(s_nm[row0 + r], s_nm[row0 + r + 1]));
#pragma unroll
                for (int r = 0; r < kRW; r += 2)
                    l2[r / 2] = f2_mul(l2[r / 2], f2_pack(s_al[row0 + r], s_al[row0 + r + 1]));
            }

            // ---- weights, their sums, and their four parts -> this token's row of P,
            // once P.V(t - kBuf) has read the buffer
            if (t >= C::kBuf &&
                !warp_wait(b_o_done + 8 * ((t - C::kBuf) & 1), (uint32_t)((t - C::kBuf) >> 1) & 1u, abort_flag))
                ok = false;
            uint32_t w[4][kRW / 4]; // part k of rows 4 i .. 4 i + 3
            const uint64_t rl2 = f2_pack(rl, rl);
#pragma unroll
            for (int r = 0; r < kRW; r += 4) {
                uint32_t h[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float x0, x1;
                    f2_unpack(x[r / 2 + q], x0, x1);
                    const float w0 = fast_exp2(x0), w1 = fast_exp2(x1);
                    l2[r / 2 + q] = f2_fma(f2_pack(w0, w1), rl2, l2[r / 2 + q]);
                    h[q] = Elem<__half>::pack(w0, w1);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[k][r / 4] = __byte_perm(h[0], h[1], 0x7531); // upper bytes
                    if (k < 3) {
                        h[0] = h2_times8(h2_sub(h[0], h[0] & 0xff00ff00u));
                        h[1] = h2_times8(h2_sub(h[1], h[1] & 0xff00ff00u));
                    }
                }
            }
            const uint32_t pj = prow + (uint32_t)j * C::kPBytes;
            if constexpr (kRW == 16) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     (pj ^ (k * NR % C::kPW)) + k * NR / C::kPW * C::kPGroup),
                                 "r"(w[k][0]), "r"(w[k][1]), "r"(w[k][2]), "r"(w[k][3])
                                 : "memory");
            } else {
#pragma unroll
                for (int k = 0; k < 4; k += 2)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(pj ^ (k * 8)), "r"(w[k][0]),
                                 "r"(w[k][1]), "r"(w[k + 1][0]), "r"(w[k + 1][1])
                                 : "memory");
            }
            if (t == ntiles - 1) {
                // Tile rows past the range (unloaded blocks, slots past the sequence
                // end) may hold anything: zero them in V so that 0 * NaN cannot reach O.
                const int vt = tokE - (tok0 + t * kQ8Tok);
                if (vt < kQ8Tok) {
                    const int s = t % vst;
                    // The parity wait is unambiguous once the stage's previous fill has
                    // landed, which P.V(t - kBuf), done by now, says for a ring of kBuf
                    // stages or more; a shorter one waits for P.V(t - 1) first.
                    if (vst < C::kBuf && t > 0 &&
                        !warp_wait(b_o_done + 8 * ((t - 1) & 1), (uint32_t)((t - 1) >> 1) & 1u, abort_flag))
                        ok = false;
                    if (!warp_wait(b_v_full + 8 * s, (uint32_t)(t / vst) & 1u, abort_flag))
                        ok = false;
                    const uint32_t vb = v_sm + (uint32_t)s * C::kTile;
                    constexpr int kChunks = C::kRB / 16;
                    const int n = (kQ8Tok - vt) * kChunks * C::kSlices;
                    for (int idx = threadIdx.x; idx < n; idx += C::kSoft) {
                        const int rest = idx / C::kSlices;
                        st_shared_zero16(vb + (idx % C::kSlices) * C::kSlice +
                                         (vt + rest / kChunks) * C::kRB + (rest % kChunks) * 16);
                    }
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(b_p_full + 8 * (t & 1));
        }
        // ---- l over the tokens while the last P.V runs.  In a warp: lanes trade
        // halves of their rows until each holds one row's sum over a group of
        // lanes, then those groups meet; warps meet in shared memory.
        constexpr int kLg = kRW == 16 ? 4 : 3;
        float l_run[kRW];
#pragma unroll
        for (int r = 0; r < kRW; r += 2)
            f2_unpack(l2[r / 2], l_run[r], l_run[r + 1]);
#pragma unroll
        for (int i = 0; i < kLg; ++i) {
            const int half = kRW >> (i + 1), off = 16 >> i;
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int r = 0; r < half; ++r) {
                const float give = up ? l_run[r] : l_run[r + half];
                const float keep = up ? l_run[r + half] : l_run[r];
                l_run[r] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
#pragma unroll
        for (int off = 16 >> kLg; off > 0; off >>= 1)
            l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], off);
        // Lane bits 4, 3, .. chose the halves: its row is lane >> (5 - kLg).
        if ((lane & ((32 >> kLg) - 1)) == 0)
            s_part[warp][lane >> (5 - kLg)] = l_run[0];
        bar_sync(2 + wg, 128);
        if (tk < kRW) {
            float sum = s_part[wg * 4][tk];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                sum += s_part[wg * 4 + w][tk];
            const int r = row0 + tk;
            s_inv[r] = sum == 0.f ? 0.f : vref / sum; // O and l hold weights in the same unit
            if (V1) {
                s_ml[r] = sum > 0.f ? kQ8Unit - s_nm[r] : -INFINITY;
                s_ml[NR + r] = sum;
            } else if (!whole && r < nrows) {
                p.exp_sums[s_row[r]] = sum * 4.8828125e-4f; // 2^-11
                p.max_logits[s_row[r]] = sum > 0.f ? (kQ8Unit - s_nm[r]) * kQ8Ln2 : -INFINITY;
            }
        }
        bar_sync(2 + wg, 128);
        // P.V(ntiles - 1), the last MMA.
        if (!warp_wait(b_o_done + 8 * ((ntiles - 1) & 1), (uint32_t)((ntiles - 1) >> 1) & 1u, abort_flag))
            ok = false;
        tc_fence_after();
        if (!ok) {
            status_bits |= PA_STATUS_TIMEOUT;
            *abort_flag = 1;
        }

        // ---- epilogue: thread = dim, O of its rows from the four parts
        if (ok && tk < D) {
#pragma unroll 1
            for (int h = 0; h < C::kMB; ++h) {
                const int d = h * 128 + tk;
#pragma unroll 1
                for (int r8 = 0; r8 < kRW; r8 += 8) {
                    uint32_t o[4][8];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tmem_ld(lane_base + h * C::kOReg + k * NR + row0 + r8, o[k]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tmem_wait_ld(o[k]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = row0 + r8 + i;
                        if (r < nrows) {
                            float v = __uint_as_float(o[3][i]);
#pragma unroll
                            for (int k = 2; k >= 0; --k)
                                v = fmaf(v, 0.125f, __uint_as_float(o[k][i]));
                            v *= s_inv[r];
                            if (V1 && ways > 1) // every tile of the rings is read by now
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem0 + (r * D + d) * 4), "f"(v)
                                             : "memory");
                            else if (whole)
                                static_cast<T *>(p.out)[s_row[r] * D + d] = E::from_float(v);
                            else
                                p.tmp_output[s_row[r] * D + d] = v;
                        }
                    }
                }
            }
        }
    }

    if (status_bits)
        set_status(p.status, status_bits);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
    if (V1 && ways > 1)
        join_cluster<D, NR>(smem0, smem_addr(s_ml), part, ways, nrows, static_cast<T *>(p.out), row_of);
    if (LOOP && threadIdx.x == 0) {
        for (int s = 0; s < kst; ++s) {
            mbar_inval(b_k_full + 8 * s);
            mbar_inval(b_k_empty + 8 * s);
        }
        for (int s = 0; s < vst; ++s) {
            mbar_inval(b_v_full + 8 * s);
            mbar_inval(b_v_empty + 8 * s);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_inval(b_s_full + 8 * j);
            mbar_inval(b_p_full + 8 * j);
            mbar_inval(b_o_done + 8 * j);
            mbar_inval(b_drained + 8 * j);
        }
    }
    return !LOOP || abort_sh == 0;
}

// Before anything global is touched the previous grid in the stream has completed
// (programmatic stream serialisation).
__device__ __forceinline__ void q8_begin(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v)
{
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

// (Registers are handed out to warps by fours: launch bounds of a multiple of 128
// threads let two CTAs share an SM.)
template <int D, int NR, int PL, bool V1>
__global__ void __launch_bounds__((Q8Cfg<D, NR, PL>::kThreads + 127) / 128 * 128, Q8Cfg<D, NR, PL>::kCtas)
    q8_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const Q8Params p)
{
    q8_begin(tmap_k, tmap_v);
    q8_unit<D, NR, PL, V1, false>(tmap_k, tmap_v, p, blockIdx.x);
}

// V1 after the 16-bit copy's attention: runs only if the copy's flag is up, mostly not,
// so a CTA per SM takes all the work (two chunks of 1024 new tokens then 308 us, 314 with a
// CTA for each unit, the wide CTAs leaving wave by wave; 31 of 390 on 3 heads 263, 282).
template <int D, int NR, int PL>
__global__ void __launch_bounds__((Q8Cfg<D, NR, PL>::kThreads + 127) / 128 * 128, Q8Cfg<D, NR, PL>::kCtas)
    q8_tc_if_kernel(const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const Q8Params p)
{
    q8_begin(tmap_k, tmap_v);
    if (__ldcg(p.only_if) == 0)
        return;
    for (int bid = blockIdx.x; bid < p.units; bid += gridDim.x) {
        if (!q8_unit<D, NR, PL, true, true>(tmap_k, tmap_v, p, bid))
            break;
        fence_proxy_async(); // the next unit's tiles land where this one's lay
        __syncthreads();
    }
}

// Kernel and shared memory of one head_dim for NR = 8, 16, 32 or 64 rows (64 up to head_dim
// 128); the conditional one for the widest NR, which calls of many rows use.
template <int D, int NR, int PL>
static Q8TcKernel q8_tc_pick_parts(int mode)
{
    using C = Q8Cfg<D, NR, PL>;
    const void *fn = mode == kQ8V1   ? reinterpret_cast<const void *>(&q8_tc_kernel<D, NR, PL, true>)
                     : mode == kQ8V2 ? reinterpret_cast<const void *>(&q8_tc_kernel<D, NR, PL, false>)
                                     : nullptr;
    if constexpr (NR == (D == 256 ? 32 : 64)) {
        if (mode == kQ8If)
            fn = reinterpret_cast<const void *>(&q8_tc_if_kernel<D, NR, PL>);
    }
    return {fn, C::kThreads, C::kCtas, C::kFixed};
}
template <int D, int NR>
static Q8TcKernel q8_tc_pick(int dtype, int mode)
{
    // (a call is cut before its type is known: pa_decode_q8_partition)
    static_assert(Q8Cfg<D, NR, 2>::kCtas == Q8Cfg<D, NR, 3>::kCtas, "one plan for both types");
    return dtype == PA_BF16 ? q8_tc_pick_parts<D, NR, 2>(mode) : q8_tc_pick_parts<D, NR, 3>(mode);
}

} // namespace pa
