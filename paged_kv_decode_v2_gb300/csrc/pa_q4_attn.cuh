// pa_q4_attn.cuh -- attention over a paged cache held in 4 bits (e2m1 codes, one e8m0
// scale per token, KV head and 32 dims) for few query rows per KV head: phase 1 of
// split-K decode ("V2") and the single-pass form ("V1").
//
//     s_t = scale * sum_g 2^(ke_tg) <q, kq_t>_g,     g: groups of 32 dims
//     out_d = sum_t softmax(s)_t 2^(ve_tg(d)) vq_td
//
// Bound by reading the cache up to some tens of query rows per KV head, at little more
// than a quarter of the bytes of a 16-bit one, so what counts is how few instructions a
// code takes on its way from memory into the tensor cores.  The codes go from shared
// memory into registers and there, two at a time, to binary16 (exactly), straight into
// the A fragments of mma.sync: nothing is written back.  Tokens (S = K Q^T) and then
// dims (O = V^T P) are the M side, 8 query rows an N tile, so that eight rows waste
// nothing.
//
//   S   A = K: a lane's word of a row holds 8 consecutive dims of group g; they take
//       the places of two K-steps' fragments (a dim's place is the lane's choice, Q is
//       laid out alike), so that a product of the MMAs lies within one group and its
//       scale multiplies the fp32 sum of its 32 dims.
//   P   weights in binary16, transposed in registers (movmatrix).
//   O   A = V^T: a pair of binary16 holds one dim of two tokens.  Interleaving the
//       nibbles of the two tokens' words (one shift and one logic operation for four
//       pairs) makes bytes that convert to such pairs.  Their tokens' scales, relative
//       to the largest V scale so far (e_ref, which moves rarely, as the softmax's
//       maximum does), multiply them in binary16: exact while a scale is at least
//       2^-26 of the largest, 0 below.
//
// Q in binary16, a row scaled by the power of two that brings its largest value to
// [2^14, 2^15): exact for binary16 values down to 2^-38 of the largest, for bf16's to
// 2^-32.  A weight is rounded to binary16 (2^-11 of itself), stored times 2^11: those
// below 2^-25 of the largest are binary16's subnormals, off by at most 2^-36.  Sums,
// maxima and accumulators are fp32.  M moves only when a weight would pass 2^4.
//
// Each warp walks its own tiles (4 KB of codes and their scales) through a ring of its
// own that cp.async fills (rows of 16-byte pieces, XORed so that both fragments' loads
// are free of bank conflicts): no barrier in the loop.  Warps join in shared memory, the
// CTAs of a sequence through the merge pass (V2) or distributed shared memory (V1 over a
// cluster).
//
// Measured (head_dim 128): 32 sequences of up to 8192 tokens, 32 heads on 8, 39 to 43 us a
// call by their lengths (143 MB: 3.5 TB/s); 64 ragged ones, 64 heads on 8, 56 to 68 us (3.2 to
// 3.9 TB/s); one of 100,000 tokens, 32 on 4, 22 us; one of 1000 tokens 6 us.  16 rows per KV
// head of such 32 sequences 60 us, 17 rows 93, 32 rows 97 (the 8-bit attention: 52, 59 and 60).  The loop issues in 56 to 59% of its
// slots, 330 warp instructions for 16 tokens: conversions, scales and their products, not
// DRAM, are what is left, and where calls are short some 5 us of set-up, merge and launches.
#pragma once

#include <type_traits>

#include "pa_q4.cuh"
#include "pa_tcgen05.cuh"
#include "pa_units.cuh"

namespace pa {

constexpr float kQ4Ln2 = 0.69314718055994531f;
constexpr float kQ4NoMax = -3.4028234663852886e38f; // M before a row has seen a token
constexpr float kQ4Grow = 4.f;  // weights stay <= 2^4,
constexpr float kQ4Unit = 11.f; // stored times 2^11
constexpr int kQ4VUnit = 13;    // V's values times 2^13 at the largest scale: <= 6 * 2^13

template <int D, int NT>
struct Q4Cfg {
    static constexpr int kTok = 4096 / D;            // tokens of a tile
    static constexpr int kRB = D / 2;                // bytes of a row's codes
    static constexpr int kSB = D / kQ4Group;         // of its scales
    static constexpr int kPieces = kRB / 16;         // 16-byte pieces of a row: one group each
    static constexpr uint32_t kCodes = kTok * kRB;   // of a tile's K or V
    static constexpr uint32_t kScales = kTok * kSB;
    static constexpr uint32_t kStage = 2 * (kCodes + kScales);
    static constexpr int kRows = 8 * NT;
    static constexpr int kAcc = D / 16 * NT * 4;     // registers of O
    static constexpr int kWarps = kAcc <= 32 ? 8 : 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kCtas = kAcc <= 32 ? 2 : kAcc <= 64 ? 3 : 2; // that share an SM
    static constexpr int kStages = kWarps == 8 ? 3 : kCtas == 3 ? 4 : 5;
    static constexpr int kSub = NT == 1 ? 2 : 1;     // 16-token steps computed side by side
    static constexpr int kQRow = D * 2 + 64;         // bytes of a Q row: neighbours in other banks
    static constexpr uint32_t kRing = kWarps * kStages * kStage;
    static constexpr uint32_t kSmem = kRing + kRows * kQRow;
    static_assert(kWarps * kRows * D * 4 <= kRing, "the warps' O lie in the rings at the end");
    static_assert(kTok % (16 * kSub) == 0 || kTok == 16, "whole steps");
    static constexpr int kSteps = kTok == 16 ? 1 : kSub; // (head_dim 256: one step per tile)
};

// Bits of a where m is set, else of b.
__device__ __forceinline__ uint32_t bits_of(uint32_t a, uint32_t b, uint32_t m)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
    return r;
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Places in shared memory.  Row r's piece i lies at piece i ^ q4_swizzle(r); K's loads
// take 8 rows of one piece, V's 4 rows of part of a row, each in all 32 banks.
template <int D>
__device__ __forceinline__ int q4_swizzle(int r)
{
    return D == 64 ? (r >> 2) & 1 : D == 128 ? (r >> 1) & 3 : r & 7;
}
// The row, of 8, at MMA place 2 c + j: bits of c where the banks of V's loads differ.
template <int D>
__device__ __forceinline__ int q4_row(int c, int j)
{
    return D == 64 ? c | j << 2 : D == 128 ? (c & 1) | j << 1 | (c >> 1) << 2 : c << 1 | j;
}

// The work of CTA `bid` of the grid that p describes.
template <int D, int NT, bool V1>
__device__ __forceinline__ void q4_unit(const Q4Params &p, int bid)
{
    using C = Q4Cfg<D, NT>;
    using H = Elem<__half>;
    constexpr int kW = C::kWarps, kR = C::kRows, kG = D / kQ4Group, kVW = D / 64;
    __shared__ float s_cf[kR];         // a row's raw products -> log2 units
    __shared__ size_t s_row[kR];       // rows of out, or slots of the intermediates
    __shared__ float s_m[kW][kR], s_l[kW][kR];
    __shared__ int s_e[kW];
    __shared__ float s_f[kW][kR];      // what a warp's O counts by
    __shared__ float s_inv[kR], s_unit; // an O's share of l, and V's largest scale
    __shared__ float s_ml[2 * kR];     // a cluster's join: M and l
    extern __shared__ __align__(16) uint8_t dyn_smem[];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 3, g8 = lane >> 2;

    // bid = ((unit * KV + KV head) * row tiles + row tile) * ways + rank, units as in
    // pick_by_size.
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
        if (!pick_by_size<V1, C::kThreads>(p.num_seqs, V1 ? p.seq_len_cap : p.partition_size, p.class_scale, unit,
                                           [&](int at) { return length(at, reporter && unit == 0); }, b, part, L))
            return;
    } else {
        b = V1 ? unit : unit / p.num_parts;
        if (!V1)
            part = unit - b * p.num_parts;
        L = length(b, reporter && part == 0 && threadIdx.x == 0);
    }
    const int tokA = part * p.partition_size;
    if (!V1 && tokA >= L)
        return; // partition past the end of the sequence: nothing to write
    const bool whole = V1 || L <= p.partition_size; // the output itself, no partials

    // Rows [c0, c0 + nrows) of the KV head's cols = q_len * group rows.
    const int c0 = rt * kR;
    const int nrows = min(kR, p.cols - c0);
    auto new_token = [&](int r) -> int { // r / group (r < 2^18, group <= 64)
        return p.group == 1 ? r : (int)__umulhi((uint32_t)r, p.group_inv);
    };
    const int i_last = p.q_len == 1 ? 0 : new_token(c0 + nrows - 1);
    auto row_of = [&](int r) -> size_t { // row of [S * q_len * H] of local row r
        const int x = c0 + r;
        const int i = p.q_len == 1 ? 0 : new_token(x);
        return (size_t)(b * p.q_len + i) * p.num_heads + (kv * p.group + x - i * p.group);
    };
    // Tokens the CTA needs: [tokA, tokE), the range cut by the causal limit of its last
    // new token (new token i sees positions <= L - q_len + i).
    long long e = ways == 1 && V1 ? (long long)L : min((long long)L, (long long)tokA + p.partition_size);
    e = min(e, (long long)L - p.q_len + i_last + 1);
    const int tokE = (int)e;
    const int tok0 = tokA & ~7;
    const int ntiles = tokE > tokA ? (tokE - tok0 + C::kTok - 1) / C::kTok : 0;
    const uint32_t smem0 = smem_addr(dyn_smem);
    auto join = [&]() {
        if (p.dtype == PA_BF16)
            join_cluster<D, kR>(smem0, smem_addr(s_ml), part, ways, nrows, static_cast<__nv_bfloat16 *>(p.out), row_of);
        else
            join_cluster<D, kR>(smem0, smem_addr(s_ml), part, ways, nrows, static_cast<__half *>(p.out), row_of);
    };
    auto put_out = [&](size_t at, float x) {
        if (p.dtype == PA_BF16)
            static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
        else
            static_cast<__half *>(p.out)[at] = __float2half_rn(x);
    };
    if (ntiles == 0) {
        // No row sees a token of the range: an empty partition (m = -inf, l = 0, o = 0),
        // or a zero output.
        if (V1 && ways > 1) {
            if (threadIdx.x < kR) {
                s_ml[threadIdx.x] = -INFINITY;
                s_ml[kR + threadIdx.x] = 0.f;
            }
            __syncthreads();
            join();
            return;
        }
        for (int idx = threadIdx.x; idx < nrows * D; idx += C::kThreads) {
            const size_t row = row_of(idx / D);
            if (whole) {
                put_out(row * D + idx % D, 0.f);
            } else {
                const size_t slot = row * p.max_num_partitions + part;
                p.tmp_output[slot * D + idx % D] = 0.f;
                if (idx % D == 0) {
                    p.exp_sums[slot] = 0.f;
                    p.max_logits[slot] = -INFINITY;
                }
            }
        }
        return;
    }

    // ---- this warp's tiles: warp, warp + kW, ..
    const int mine = warp < ntiles ? (ntiles - warp + kW - 1) / kW : 0;
    const int sh = p.block_shift, in_block = (1 << sh) - 1;
    const int32_t *bt = p.block_tables + (size_t)b * p.max_blocks;
    const uint32_t ring = smem0 + warp * C::kStages * C::kStage;
    const int t_first = tok0 + warp * C::kTok; // its first tile's first token
    // Lane l holds the cache row of 8 tokens, l % kOct of tile base + l / kOct, kPer tiles
    // at a time, the next ones' ahead.
    constexpr int kOct = C::kTok / 8, kPer = 32 / kOct;
    auto fetch_rows = [&](int base) -> int {
        const int i = base + lane / kOct;
        const int tok = t_first + i * (kW * C::kTok) + lane % kOct * 8;
        if (i >= mine || tok >= tokE)
            return 0;
        int id = __ldg(bt + (tok >> sh));
        if (id < 0 || id >= p.num_blocks) {
            set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
            id = 0; // read a valid block instead of memory outside the cache
        }
        return ((id * p.num_kv_heads + kv) << sh) + (tok & in_block); // (all rows number less than 2^31)
    };
    int rows_now = fetch_rows(0), rows_next = 0;
    // Copy q of a tile's four: row q * 32 / kPieces + lane / kPieces, its piece lane % kPieces.
    const int l_row = lane / C::kPieces, l_piece = lane % C::kPieces;
    const uint8_t *const k_src = p.key_cache + l_row % 8 * C::kRB + l_piece * 16;
    const uint8_t *const v_src = p.value_cache + l_row % 8 * C::kRB + l_piece * 16;
    const int l_scale = (lane & 7) * (16 / C::kSB); // the first row of its piece of scales
    const uint8_t *const s_src = (lane < 8 ? p.k_scales : p.v_scales) + l_scale % 8 * C::kSB;
    int issued = 0, t_issue = t_first;
    uint32_t st_issue = ring;
    auto issue = [&]() { // the next tile of this warp into its stage
        if (issued < mine) {
            const int at = issued % kPer;
            if (at == 0) {
                if (issued > 0)
                    rows_now = rows_next;
                rows_next = fetch_rows(issued + kPer);
            }
            auto copies = [&](auto inside) { // (a tile that lies in the range as a whole asks nothing)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // (head_dim 256: four rows a copy, of one octet two copies)
                constexpr int kHalf = C::kPieces == 8 ? 4 : 0;
                const int more = q & 1 ? kHalf : 0;
                const int oct = C::kPieces == 8 ? q / 2 : C::kPieces == 4 ? q : 2 * q + (lane >> 4);
                const uint32_t r = (uint32_t)__shfl_sync(0xffffffffu, rows_now, at * kOct + oct) + more;
                const uint32_t dst = st_issue + q * 512 + l_row * C::kRB + ((l_piece ^ q4_swizzle<D>(l_row + more)) << 4);
                const int row = q * (32 / C::kPieces) + l_row;
                const uint32_t n = decltype(inside)::value || t_issue + row < tokE ? 16u : 0u;
                q4_copy16(dst, row_at<C::kRB>(k_src, r), n);
                q4_copy16(dst + C::kCodes, row_at<C::kRB>(v_src, r), n);
            }
            // Scales: 128 bytes of K's, 128 of V's, a piece's tokens in one octet.
            const uint32_t r = (uint32_t)__shfl_sync(0xffffffffu, rows_now, at * kOct + l_scale / 8);
            if (lane < 16) {
                const int n = decltype(inside)::value ? 16 : min(max((tokE - t_issue - l_scale) * C::kSB, 0), 16);
                q4_copy16(st_issue + 2 * C::kCodes + lane * 16, row_at<C::kSB>(s_src, r), n);
            }
            };
            if (t_issue + C::kTok <= tokE)
                copies(std::true_type());
            else
                copies(std::false_type());
            ++issued;
            t_issue += kW * C::kTok;
            st_issue += C::kStage;
            if (st_issue == ring + C::kStages * C::kStage)
                st_issue = ring;
        }
        q4_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i)
        issue();

    // ---- Q rows -> binary16 in shared memory; a warp per row
    const uint32_t q_sm = smem0 + C::kRing;
    for (int r = warp; r < kR; r += kW) {
        constexpr int kDL = D / 32; // consecutive dims of a lane: 2, 4 or 8
        const uint32_t *q32 = static_cast<const uint32_t *>(p.query) + row_of(r < nrows ? r : 0) * (D / 2) +
                              lane * (kDL / 2);
        float x[kDL], m = 0.f;
#pragma unroll
        for (int k = 0; k < kDL / 2; ++k) {
            const uint32_t w = r < nrows ? __ldg(q32 + k) : 0u;
            x[2 * k] = p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::lo(w) : H::lo(w);
            x[2 * k + 1] = p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::hi(w) : H::hi(w);
            m = fmaxf(m, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float f, inv;
        q4_row_scale(m, f, inv);
        if (lane == 0) {
            s_cf[r] = p.scale * inv * kLog2e;
            const size_t row = row_of(r < nrows ? r : 0);
            s_row[r] = whole ? row : row * p.max_num_partitions + part;
        }
#pragma unroll
        for (int k = 0; k < kDL / 2; ++k)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(q_sm + r * C::kQRow + lane * (kDL * 2) + k * 4),
                         "r"(H::pack(q4_scaled(x[2 * k], f), q4_scaled(x[2 * k + 1], f)))
                         : "memory");
    }
    __syncthreads();

    // B fragments of Q: row nt * 8 + g8, dims 32 g + 8 c .. + 7.
    const uint32_t q_at = q_sm + g8 * C::kQRow + c * 16;
    uint32_t qf[NT == 1 ? kG : 1][4];
    if constexpr (NT == 1) {
#pragma unroll
        for (int g = 0; g < kG; ++g)
            lds_words(q_at + g * 64, qf[g]);
    }
    // Rows n * 8 + 2 c + j: what a raw product counts by, kQ4Unit - M, and l.
    float cf[NT][2], nm[NT][2], l[NT][2];
    float o[D / 16][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            cf[n][j] = s_cf[n * 8 + 2 * c + j];
            nm[n][j] = -kQ4NoMax;
            l[n][j] = 0.f;
        }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[i][n][k] = 0.f;
    int e_ref = 0;
    // Tiles that lie in [tokA, tok_all) are seen whole by every row.
    const int rel = L - p.q_len; // new token i sees positions <= rel + i
    const int tok_all = (int)min((long long)tokE, (long long)rel + (p.q_len == 1 ? 0 : new_token(c0)) + 1);
    // This lane's places in a tile: its K row of 8 (and 8 on), the groups' words in it;
    // its V rows 2 c + j of 8 (and 8 on), its dims' words in them.  Swizzles repeat
    // after 8 rows.
    const int rk = q4_row<D>(g8 >> 1, g8 & 1);
    uint32_t k_at[kG], v_at[2];
#pragma unroll
    for (int g = 0; g < kG; ++g)
        k_at[g] = rk * C::kRB + ((g ^ q4_swizzle<D>(rk)) << 4) + c * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = q4_row<D>(c, j), byte = g8 * kVW * 4;
        v_at[j] = C::kCodes + row * C::kRB + (((byte >> 4) ^ q4_swizzle<D>(row)) << 4) + (byte & 15);
    }
    constexpr int kJ = (D == 64 ? 4 : D == 128 ? 2 : 1) * C::kSB; // from a V row's scales to its neighbour's (j)
    const uint32_t ks_at = 2 * C::kCodes + rk * C::kSB;
    const uint32_t vs_at = 2 * C::kCodes + C::kScales + q4_row<D>(c, 0) * C::kSB + (g8 * kG >> 3);

    uint32_t st = ring;
    int t0 = t_first;
    for (int i = 0; i < mine; ++i, t0 += kW * C::kTok) {
        q4_wait<C::kStages - 2>();
        __syncwarp();
        issue(); // into the stage that tile i - 1 has left
        const bool full = t0 >= tokA && t0 + C::kTok <= tok_all;
#pragma unroll 1
        for (int u0 = 0; u0 < C::kTok; u0 += 16 * C::kSteps, st += 16 * C::kSteps * C::kRB) {
            // (st: the stage, advanced by the rows of codes behind; the scales' rows are shorter)
            const uint32_t sc_st = st - u0 * (C::kRB - C::kSB);
            // ---- raw products of 16-token steps: rows rk and 8 + rk, columns 2 c + j
            float s[C::kSteps][NT][4];
#pragma unroll
            for (int u = 0; u < C::kSteps; ++u) {
                float sc0[kG], sc1[kG];
                q4_scales<kG>(sc_st + ks_at + u * 16 * C::kSB, sc0);
                q4_scales<kG>(sc_st + ks_at + (u * 16 + 8) * C::kSB, sc1);
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                    uint32_t x0[4], x1[4];
                    e2m1x8(lds32(st + k_at[g] + u * 16 * C::kRB), x0);
                    e2m1x8(lds32(st + k_at[g] + (u * 16 + 8) * C::kRB), x1);
                    const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t q[4];
                        if constexpr (NT == 1) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                q[k] = qf[g][k];
                        } else {
                            lds_words(q_at + n * 8 * C::kQRow + g * 64, q);
                        }
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        H::mma(acc, a0, q[0], q[1]);
                        H::mma(acc, a1, q[2], q[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float f = k < 2 ? sc0[g] : sc1[g];
                            s[u][n][k] = g == 0 ? acc[k] * f : fmaf(acc[k], f, s[u][n][k]);
                        }
                    }
                }
            }
            // ---- exponents of the stored weights
            float x[C::kSteps][NT][4], top = -INFINITY;
#pragma unroll
            for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[u][n][k] = fmaf(s[u][n][k], cf[n][k & 1], nm[n][k & 1]);
            if (!full) {
                // First visible row of a token: new token i = (c0 + r) / group sees it when
                // i >= pos - rel.
#pragma unroll
                for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int pos = t0 + u0 + u * 16 + h * 8 + rk;
                        const long long i0 = (long long)pos - rel;
                        const long long first = i0 > 0 ? i0 * p.group - c0 : 0;
                        const int r_min = pos < tokA || pos >= tokE || first > kR ? kR : (int)max(first, 0ll);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (n * 8 + 2 * c + j < r_min)
                                    x[u][n][2 * h + j] = -INFINITY;
                    }
            }
#pragma unroll
            for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    top = fmax3(top, x[u][n][0], x[u][n][1]);
                    top = fmax3(top, x[u][n][2], x[u][n][3]);
                }
            // ---- V's scales of this lane's four tokens a step (of its dims' group), as
            // 2^(13 + e - e_ref) in binary16 pairs: exponent field 28 + e - e_ref.
            uint32_t ve[C::kSteps][2], f[C::kSteps][2]; // two tokens' bytes, and factors
            auto factors = [&]() {
#pragma unroll
                for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t down = min_u16x2((uint32_t)e_ref * 0x10001u - ve[u][h], (15 + kQ4VUnit) * 0x10001u);
                        f[u][h] = (15 + kQ4VUnit) * 0x4000400u - down * 0x400u;
                    }
            };
            uint32_t ve_top = 0;
#pragma unroll
            for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t at = sc_st + vs_at + (u * 16 + h * 8) * C::kSB;
                    ve[u][h] = lds8(at) + lds8(at + kJ) * 0x10000u;
                    ve_top = max_u16x2(ve_top, ve[u][h]);
                }
            const bool grow = top > kQ4Unit + kQ4Grow || min_u16x2(ve_top, (uint32_t)e_ref * 0x10001u) != ve_top;
            factors();
            if (__any_sync(0xffffffffu, grow)) {
                // M moves to the rows' maxima, e_ref to the largest scale; O follows.
                float al[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float most = -INFINITY;
#pragma unroll
                        for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float &v = x[u][n][2 * h + j];
                                v = v == -INFINITY ? v : s[u][n][2 * h + j] * cf[n][j];
                                most = fmaxf(most, v);
                            }
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                        const float now = fminf(nm[n][j], kQ4Unit - most);
                        al[n][j] = fast_exp2(now - nm[n][j]);
                        nm[n][j] = now;
                        l[n][j] *= al[n][j];
#pragma unroll
                        for (int u = 0; u < C::kSteps; ++u) {
                            x[u][n][j] += now;
                            x[u][n][2 + j] += now;
                        }
                    }
                uint32_t most = 0, nan_of[C::kSteps][2];
#pragma unroll
                for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool n0 = (ve[u][h] & 0xffffu) == 255u, n1 = ve[u][h] >> 16 == 255u;
                        nan_of[u][h] = (n0 ? 0x7fffu : 0u) | (n1 ? 0x7fff0000u : 0u);
                        ve[u][h] &= (n0 ? 0u : 0xffffu) | (n1 ? 0u : 0xffff0000u);
                        most = max(most, max(ve[u][h] & 0xffffu, ve[u][h] >> 16));
                    }
                // (One more than the largest so far: the next larger one, a power of two away
                // and likely in a small tile's successors, costs nothing then.)
                const int top_e = (int)__reduce_max_sync(0xffffffffu, most);
                const int now = top_e > e_ref ? min(top_e + 1, 254) : e_ref;
                const float back = fast_exp2((float)(e_ref - now));
                e_ref = now;
                factors();
#pragma unroll
                for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        f[u][h] |= nan_of[u][h];
                if (i > 0 || u0 > 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        al[n][0] *= back;
                        al[n][1] *= back;
                    }
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                o[d][n][k] *= al[n][k & 1];
                }
            }
#pragma unroll
            for (int u = 0; u < C::kSteps; ++u) {
                // ---- weights, their sums, and the B fragments of P
                uint32_t pb[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[k] = fast_exp2(x[u][n][k]);
                        l[n][k & 1] += w[k];
                    }
                    pb[n][0] = movmatrix_trans(H::pack(w[0], w[1]));
                    pb[n][1] = movmatrix_trans(H::pack(w[2], w[3]));
                }
                // ---- V: words of the lane's dims for tokens 2 c, 2 c + 1 (and + 8) of P
                uint32_t vw[4][kVW];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    lds_words(st + v_at[k & 1] + (u * 16 + (k >> 1) * 8) * C::kRB, vw[k]);
#pragma unroll
                for (int w = 0; w < kVW; ++w) {
                    uint32_t a[4][4]; // [fragment register][byte]
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w0 = vw[2 * h][w], w1 = vw[2 * h + 1][w];
                        e2m1x8(bits_of(w0, w1 * 16u, 0x0f0f0f0fu), a[2 * h]);     // even dims
                        e2m1x8(bits_of(w0 >> 4, w1, 0x0f0f0f0fu), a[2 * h + 1]); // odd dims
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t av[4] = {h2_mul(a[0][k], f[u][0]), h2_mul(a[1][k], f[u][0]), h2_mul(a[2][k], f[u][1]),
                                                h2_mul(a[3][k], f[u][1])};
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            H::mma(o[w * 4 + k][n], av, pb[n][0], pb[n][1]);
                    }
                }
            }
        }
        st += C::kStage - C::kCodes; // (kTok rows of codes are kCodes)
        if (st == ring + C::kStages * C::kStage)
            st = ring;
    }
    q4_wait<0>();

    // ---- the warps join.  O's lane: dims g8 * D / 8 + 2 i (+ 1), rows n * 8 + 2 c + j.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
            if (g8 == 0) {
                s_m[warp][n * 8 + 2 * c + j] = kQ4Unit - nm[n][j];
                s_l[warp][n * 8 + 2 * c + j] = l[n][j];
            }
        }
    if (lane == 0)
        s_e[warp] = e_ref;
    __syncthreads(); // (and every warp is done with its ring)
    if (threadIdx.x < kR) {
        const int r = threadIdx.x;
        float top = s_m[0][r], sum = 0.f;
        int most = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            top = fmaxf(top, s_m[w][r]);
            most = max(most, s_e[w]);
        }
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const float f = fast_exp2(s_m[w][r] - top);
            sum += s_l[w][r] * f;
            s_f[w][r] = f * fast_exp2((float)(s_e[w] - most));
        }
        const bool seen = !(sum == 0.f);
        s_inv[r] = seen ? 1.f / ((float)(1 << kQ4VUnit) * sum) : 0.f;
        if (r == 0)
            s_unit = __uint_as_float(most ? (uint32_t)most << 23 : 1u << 22); // 2^(most - 127)
        if (V1) {
            s_ml[r] = seen ? top : -INFINITY;
            s_ml[kR + r] = sum;
        } else if (!whole && r < nrows) {
            p.exp_sums[s_row[r]] = sum * 4.8828125e-4f; // 2^-11
            p.max_logits[s_row[r]] = seen ? top * kQ4Ln2 : -INFINITY;
        }
    }
    float *const o_sm = reinterpret_cast<float *>(dyn_smem); // [warp][row][dim]
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float2 *>(o_sm + (size_t)((warp * kR + n * 8 + 2 * c + j) * D + g8 * (D / 8) + 2 * i)) =
                    make_float2(o[i][n][j], o[i][n][2 + j]);
    __syncthreads();
    for (int at = threadIdx.x; at < nrows * (D / 2); at += C::kThreads) {
        const int r = at / (D / 2), d = at % (D / 2) * 2;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const float2 v = *reinterpret_cast<const float2 *>(o_sm + (w * kR + r) * D + d);
            x = fmaf(v.x, s_f[w][r], x);
            y = fmaf(v.y, s_f[w][r], y);
        }
        const float inv = s_inv[r];
        x = inv == 0.f ? 0.f : x * inv * s_unit; // (a row that sees nothing: 0, whatever its O holds)
        y = inv == 0.f ? 0.f : y * inv * s_unit;
        if (V1 && ways > 1) {
            *reinterpret_cast<float2 *>(o_sm + r * D + d) = make_float2(x, y);
        } else if (whole) {
            static_cast<uint32_t *>(p.out)[(s_row[r] * D + d) / 2] =
                p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::pack(x, y) : H::pack(x, y);
        } else {
            *reinterpret_cast<float2 *>(p.tmp_output + s_row[r] * D + d) = make_float2(x, y);
        }
    }
    if (V1 && ways > 1) {
        __syncthreads();
        join();
    }
}

// Before anything global is touched the previous grid in the stream has completed
// (programmatic stream serialisation).
template <int D, int NT, bool V1>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::kThreads, Q4Cfg<D, NT>::kCtas) q4_attn_kernel(const Q4Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    q4_unit<D, NT, V1>(p, blockIdx.x);
}

// V1 after the 16-bit copy's attention: runs only if the copy's flag is up, mostly not.
template <int D, int NT>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::kThreads, Q4Cfg<D, NT>::kCtas) q4_attn_if_kernel(const Q4Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (__ldcg(p.only_if) == 0)
        return;
    for (int bid = blockIdx.x; bid < p.units; bid += gridDim.x) {
        q4_unit<D, NT, true>(p, bid);
        __syncthreads(); // the next unit's tiles land where this one's lay
    }
}

template <int D, int NT>
static Q4Kernel q4_attn_pick(int mode)
{
    using C = Q4Cfg<D, NT>;
    const void *fn = mode == kQ8V1   ? reinterpret_cast<const void *>(&q4_attn_kernel<D, NT, true>)
                     : mode == kQ8V2 ? reinterpret_cast<const void *>(&q4_attn_kernel<D, NT, false>)
                                     : nullptr;
    if constexpr (NT == (D == 256 ? 2 : 4)) {
        if (mode == kQ8If)
            fn = reinterpret_cast<const void *>(&q4_attn_if_kernel<D, NT>);
    }
    return {fn, C::kThreads, C::kCtas, C::kSmem};
}

} // namespace pa
