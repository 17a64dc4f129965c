// pa_q4_tc.cuh -- attention over a paged cache held in 4 bits for many query rows per KV
// head, on the tcgen05 tensor cores: phase 1 of split-K decode ("V2") and the single-pass
// form ("V1").
//
//   S   = Q K_t^T       M = 128 query rows, N = 64 tokens, K = D
//   P   = exp(S - M)    one thread per row, over S in tensor memory
//   O  += P V_t         M = 128, N = D, K = 64 tokens; A = P in tensor memory
//
// as the 16-bit kernel (pa_tc.cuh) has it, but that the K and V tiles come from four
// converter warps instead of the TMA: they read codes a tile ahead into registers, turn
// them into binary16 (exactly, two instructions for two values) and write them where the
// TMA would have, in 128-byte swizzled rows.  A code is converted
// once per 128 rows, a quarter of the softmax's work there.  Everything is binary16,
// whatever the query's type:
//
//   Q   a row times the power of two that brings its largest value to [2^14, 2^15);
//   K   times 2^13 at the largest scale of the tile's 64 tokens, whose power of two the
//       rows multiply their scores by: exact while a scale is at least 2^-27 of that
//       one, 0 below;
//   V   likewise at a reference that only grows, one step above the largest scale so far;
//       O follows where it moves;
//   P   in units of 2^-7 of e^(s - M), rounded once (2^-11 of itself, or by at most 2^-32
//       of a row's largest).  M moves when a weight would pass 2^8.
//
// Warp roles: 0-3 rows (softmax, epilogue), 4 issues the MMAs and owns the tensor memory,
// 5-8 convert.  Rows take half a tile's row at a time, and compute weights under the M they
// have while they look for a larger one, so that two CTAs share an SM.  A KV head of at most 64
// rows stores only those of Q (see pa_tc.cuh), and its other row warps sleep.
//
// Measured (head_dim 128, 8 KV heads): 16 new tokens of 4 heads each for 32 sequences of up
// to 8192 tokens 102 to 112 us by their lengths (143 MB at 1.4 TB/s; mma.sync 165; the 8-bit
// attention 79), 128 rows per KV head 128 (298).
// Some 2770 warp instructions for a tile of 64 tokens, two fifths of them the converters',
// at 44% of the issue slots: a tile takes its CTA some 2800 clocks, of which the converters
// work some 2200, and the thread that issues MMAs 1200.  Tried and slower: codes through a
// ring that cp.async fills (127 us) or bulk copies of eight tokens do (112), lanes side by
// side on a row's codes (109), eight converter warps for up to 64 rows (119).
#pragma once

#include <type_traits>

#include "pa_q4.cuh"
#include "pa_tcgen05.cuh"
#include "pa_units.cuh"

namespace pa {

constexpr float kQ4TcGrow = 8.f; // weights stay <= 2^8,
constexpr float kQ4TcUnit = 7.f; // stored times 2^7
constexpr int kQ4TcKv = 13;      // K and V times 2^13 at their largest scale
constexpr int kQ4TcThreads = 288;
constexpr int kQ4TcAhead = 5; // tiles: how far ahead codes are brought into L2

template <int D>
struct Q4TcCfg {
    static constexpr int kSlices = D / 64;                 // 128-byte swizzled column slices
    static constexpr uint32_t kQSlice = kTcRows * 128;     // bytes of one Q slice
    static constexpr uint32_t kKVSlice = kTcTok * 128;     // bytes of one K or V slice
    static constexpr uint32_t kQBytes = kQSlice * kSlices;
    static constexpr uint32_t kKVBytes = kKVSlice * kSlices;
    // TMEM columns: O at [0, D), S/P buffer j at [D + 64 j, D + 64 j + 64).
    static constexpr uint32_t kSCol = D;
    static constexpr uint32_t kCols = D + 2 * kTcTok <= 256 ? 256 : 512;
    static constexpr int kCtas = D <= 128 ? 2 : 1;         // that share an SM
    static constexpr int kPieces = D / 64;                 // 32-dim pieces of a converter thread's K or V
    static constexpr int kRB = D / 2, kSB = D / 32;        // bytes of a row's codes and scales
};

// Codes and scale bytes of one converter thread's pieces of K or V.
template <int N>
struct Q4Piece {
    uint4 codes[N];
    uint32_t scales; // N bytes
    bool in;         // (K's) the token lies in the range
};

// (Registers are handed out to warps by fours: launch bounds of a multiple of 128 threads
// let two CTAs share an SM.)
template <int D, bool V1>
__global__ void __launch_bounds__((kQ4TcThreads + 127) / 128 * 128, Q4TcCfg<D>::kCtas) q4_tc_kernel(const Q4Params p)
{
    using C = Q4TcCfg<D>;
    using H = Elem<__half>;
    constexpr int kMmaWarp = 4, kConvWarp = 5;
    __shared__ uint64_t k_full[kMaxStages], v_full[kMaxStages], k_empty[kMaxStages], v_empty[kMaxStages];
    __shared__ uint64_t q_full, s_full[2], p_full[2], o_done[2], drained;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ int2 s_e[2 * kMaxStages];  // of tile t: K's largest scale byte, V's reference
    __shared__ __align__(16) uint32_t s_most[2][4]; // of tile t: each converter warp's largest bytes
    __shared__ float s_cf[kTcRows];       // what undoes Q rows' scales
    extern __shared__ uint8_t dyn_smem[];

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blockIdx.x = (unit * KV + KV head) * row tiles + row tile, units as in pick_by_size;
    // row tiles of one KV head are neighbours, so that their reads meet in L2.
    int unit = blockIdx.x;
    const int rt = unit % p.col_groups;
    unit /= p.col_groups;
    const int kv = unit % p.num_kv_heads;
    unit /= p.num_kv_heads;
    const bool reporter = kv == 0 && rt == 0;
    auto length = [&](int at, bool report) -> int {
        const int len = __ldg(p.seq_lens + at);
        if (len >= 0 && len <= p.seq_len_cap)
            return len;
        if (report)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        return len < 0 ? 0 : p.seq_len_cap;
    };
    int b, part = 0, L;
    if (p.sorted) {
        if (!pick_by_size<V1, kQ4TcThreads>(p.num_seqs, V1 ? p.seq_len_cap : p.partition_size, p.class_scale, unit,
                                            [&](int at) { return length(at, reporter && unit == 0); }, b, part, L))
            return;
    } else {
        b = V1 ? unit : unit / p.num_parts;
        part = V1 ? 0 : unit - b * p.num_parts;
        L = length(b, reporter && part == 0 && threadIdx.x == 0);
    }
    const int tokA = V1 ? 0 : part * p.partition_size;
    if (!V1 && tokA >= L)
        return; // partition past the end of the sequence: nothing to write
    const bool whole = V1 || L <= p.partition_size; // the output itself, no partials

    // Rows [c0, c0 + nrows) of the KV head's cols = q_len * group rows.
    const int c0 = rt * kTcRows;
    const int nrows = min(kTcRows, p.cols - c0);
    auto new_token = [&](int r) -> int { // r / group (r < 2^18, group <= 64)
        return p.group == 1 ? r : (int)__umulhi((uint32_t)r, p.group_inv);
    };
    const int i_last = new_token(c0 + nrows - 1);
    // Tokens the CTA needs: [tokA, tokE), the range cut by the causal limit of its last
    // new token (new token i sees positions <= L - q_len + i).
    long long e = V1 ? (long long)L : min((long long)L, (long long)tokA + p.partition_size);
    e = min(e, (long long)L - p.q_len + i_last + 1);
    const int tokE = (int)e;
    const int tok0 = tokA & ~7;
    const int ntiles = tokE > tokA ? (tokE - tok0 + kTcTok - 1) / kTcTok : 0;

    // This thread's row (warps 0-3).  A tile of fewer than 128 rows puts them in the
    // highest of these warps.
    const int roff = kTcRows - (nrows + 31) / 32 * 32;
    const int r = threadIdx.x;
    const bool row_ok = r < kTcRows && r >= roff && r - roff < nrows;
    const int ci = c0 + (row_ok ? r - roff : 0);
    const int qi = new_token(ci);
    const size_t qrow = (size_t)(b * p.q_len + qi) * p.num_heads + kv * p.group + ci - qi * p.group;
    auto put_pair = [&](uint32_t *out, float x, float y) {
        *out = p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::pack(x, y) : H::pack(x, y);
    };
    if (ntiles == 0) {
        // No row sees a token of the range: an empty partition (m = -inf, l = 0, o = 0),
        // or a zero output.
        if (row_ok) {
            if (whole) {
                uint32_t *const out = static_cast<uint32_t *>(p.out) + qrow * (D / 2);
                for (int d = 0; d < D / 2; ++d)
                    out[d] = 0u;
            } else {
                const size_t slot = qrow * p.max_num_partitions + part;
                float4 *const tmp = reinterpret_cast<float4 *>(p.tmp_output + slot * D);
                for (int d = 0; d < D / 4; ++d)
                    tmp[d] = make_float4(0.f, 0.f, 0.f, 0.f);
                p.exp_sums[slot] = 0.f;
                p.max_logits[slot] = -INFINITY;
            }
        }
        return;
    }

    const int kst = p.stages, vst = p.v_stages;
    const uint32_t smem0 = (smem_addr(dyn_smem) + 1023u) & ~1023u;
    // [Q | K ring | V ring], or with a half Q tile [K ring | Q | V ring], the K ring then
    // holding the 8 KB that the first slice's padding rows alias.
    const bool q_half = p.cols <= kTcRows / 2;
    const uint32_t q_slice = q_half ? C::kQSlice / 2 : C::kQSlice;
    const uint32_t k_sm = q_half ? smem0 : smem0 + C::kQBytes;
    const uint32_t q_sm = q_half ? k_sm + (uint32_t)kst * C::kKVBytes : smem0;
    const uint32_t v_sm = q_half ? q_sm + C::kQBytes / 2 : k_sm + (uint32_t)kst * C::kKVBytes;
    const uint32_t b_k_full = smem_addr(k_full), b_v_full = smem_addr(v_full);
    const uint32_t b_k_empty = smem_addr(k_empty), b_v_empty = smem_addr(v_empty);
    const uint32_t b_q_full = smem_addr(&q_full), b_s_full = smem_addr(s_full);
    const uint32_t b_p_full = smem_addr(p_full), b_o_done = smem_addr(o_done);
    const uint32_t b_drained = smem_addr(&drained);
    volatile int *abort_flag = &abort_sh;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&tmem_base_sh), C::kCols);
        tmem_relinquish();
    }
    if (threadIdx.x == kConvWarp * 32) {
        for (int s = 0; s < kst; ++s) {
            mbar_init(b_k_full + 8 * s, 128);
            mbar_init(b_k_empty + 8 * s, 1);
        }
        for (int s = 0; s < vst; ++s) {
            mbar_init(b_v_full + 8 * s, 128);
            mbar_init(b_v_empty + 8 * s, 1);
        }
        mbar_init(b_q_full, kTcRows);
        for (int j = 0; j < 2; ++j) {
            mbar_init(b_s_full + 8 * j, 1);
            mbar_init(b_p_full + 8 * j, kTcRows - roff); // (warps of padding rows only stay away)
            mbar_init(b_o_done + 8 * j, 1);
        }
        mbar_init(b_drained, 1);
        abort_sh = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    int32_t status_bits = 0;

    if (warp >= kConvWarp) {
        // ---------------------------------------------------------- converters
        // Thread = token of the tile (two warps of 32) and half of its dims.  Codes of the
        // next tile are on their way while this one's are converted.
        const int cw = warp - kConvWarp;
        const int token = (cw & 1) * 32 + lane, half = cw >> 1;
        const int sh = p.block_shift, in_block = (1 << sh) - 1;
        const int32_t *const bt = p.block_tables + (size_t)b * p.max_blocks;
        using Piece = Q4Piece<C::kPieces>;
        const uint8_t *const k_src = p.key_cache + half * C::kPieces * 16, *const v_src = p.value_cache + half * C::kPieces * 16;
        const uint8_t *const ks_src = p.k_scales + half * C::kPieces, *const vs_src = p.v_scales + half * C::kPieces;
        int tok = tok0 + token; // of the tile asked for next
        // The block of token tok + ahead, or -1 where the range has ended.
        auto fetch_id = [&](int ahead) -> int32_t { return tok + ahead < tokE ? __ldg(bt + ((tok + ahead) >> sh)) : -1; };
        auto load = [&](int32_t id, Piece &k, Piece &v) {
            const bool in = tok < tokE; // (behind the range any row's codes, times 0)
            if (in && (id < 0 || id >= p.num_blocks)) {
                status_bits |= PA_STATUS_BAD_BLOCK_ID;
                id = 0; // read a valid block instead of memory outside the cache
            }
            const uint32_t row = in ? (uint32_t)(((id * p.num_kv_heads + kv) << sh) + (tok & in_block)) : 0u;
            k.in = in;
            const uint4 *const kc = reinterpret_cast<const uint4 *>(row_at<C::kRB>(k_src, row));
            const uint4 *const vc = reinterpret_cast<const uint4 *>(row_at<C::kRB>(v_src, row));
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                k.codes[i] = __ldg(kc + i);
                v.codes[i] = __ldg(vc + i);
            }
            const uint8_t *const ks = row_at<C::kSB>(ks_src, row), *const vs = row_at<C::kSB>(vs_src, row);
            if constexpr (C::kPieces == 1) {
                k.scales = __ldg(ks);
                v.scales = __ldg(vs);
            } else if constexpr (C::kPieces == 2) {
                k.scales = __ldg(reinterpret_cast<const uint16_t *>(ks));
                v.scales = __ldg(reinterpret_cast<const uint16_t *>(vs));
            } else {
                k.scales = __ldg(reinterpret_cast<const uint32_t *>(ks));
                v.scales = __ldg(reinterpret_cast<const uint32_t *>(vs));
            }
        };
        // The largest scale byte but 255, plus one.
        auto most_of = [](const Piece &x, bool in) -> uint32_t {
            uint32_t m = ((x.scales & 0x00ff00ffu) + 0x00010001u) & 0x00ff00ffu;
            if (C::kPieces > 1)
                m = max_u16x2(m, ((x.scales >> 8 & 0x00ff00ffu) + 0x00010001u) & 0x00ff00ffu);
            return !in ? 0u : C::kPieces > 2 ? max(m & 0xffffu, m >> 16) : m & 0xffffu;
        };
        // Pieces -> the tile at `tile`: 16-byte chunk c of a token's slice at c ^ (token & 7).
        const uint32_t at = (C::kPieces * half >> 1) * C::kKVSlice + token * 128 + ((token & 7) << 4);
        auto put = [&](const Piece &x, bool in, int ref, uint32_t tile) {
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                const int se = (int)(x.scales >> 8 * i & 255u);
                // 2^(13 + se - ref): exponent field 28 + se - ref.
                const int up = max(15 + kQ4TcKv + se - ref, 0);
                const uint32_t f = !in ? 0u : se == 255 ? 0x7fff7fffu : (uint32_t)up * 0x4000400u;
                const uint32_t w[4] = {x.codes[i].x, x.codes[i].y, x.codes[i].z, x.codes[i].w};
                const int first = C::kPieces == 1 ? half * 4 : (i & 1) * 4; // its first chunk of a slice
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t h[4];
                    e2m1x8(w[j], h);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[k]) : "r"(f));
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     ((tile + at) ^ ((first + j) << 4)) + (i >> 1) * C::kKVSlice),
                                 "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                                 : "memory");
                }
            }
        };
        // Tiles further ahead are brought into L2: one on its way to registers is too few to
        // hide DRAM's latency (16 new tokens 124 us, 110 with it).
        auto prefetch = [&](int32_t id, int ahead) {
            if (id < 0 || id >= p.num_blocks)
                return;
            const uint32_t row = (uint32_t)(((id * p.num_kv_heads + kv) << sh) + ((tok + ahead) & in_block));
            // (a row's codes take 32 to 128 bytes, its scales share a line with its neighbours')
            const uint8_t *const line = half ? row_at<C::kRB>(p.value_cache, row) : row_at<C::kRB>(p.key_cache, row);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
            if ((lane & 7) == 0)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(half ? row_at<C::kSB>(p.v_scales, row) : row_at<C::kSB>(p.k_scales, row)));
        };
        Piece k, v, k_next, v_next;
        load(fetch_id(0), k, v);
        int32_t id_next = fetch_id(kTcTok);
#pragma unroll 1
        for (int i = 2; i < kQ4TcAhead; ++i)
            prefetch(fetch_id(i * kTcTok), i * kTcTok);
        int32_t id_ahead = fetch_id(kQ4TcAhead * kTcTok);
        int ref = 0;            // V's reference
        int ks = 0, vs = 0;     // ring stages of tile t
        uint32_t kph = 1u, vph = 1u;
        bool alive = true;      // (a warp that gave up still meets the others)
        auto step = [&](int t, const Piece &k, const Piece &v, Piece &k_next, Piece &v_next) {
            prefetch(id_ahead, kQ4TcAhead * kTcTok);
            tok += kTcTok;
            load(id_next, k_next, v_next);
            id_next = fetch_id(kTcTok);
            id_ahead = fetch_id(kQ4TcAhead * kTcTok);
            const uint32_t mk = __reduce_max_sync(0xffffffffu, most_of(k, k.in));
            const uint32_t mv = __reduce_max_sync(0xffffffffu, most_of(v, k.in));
            if (lane == 0)
                s_most[t & 1][cw] = mk | mv << 16;
            asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
            const uint4 of = *reinterpret_cast<const uint4 *>(s_most[t & 1]);
            const uint32_t tops = max_u16x2(max_u16x2(of.x, of.y), max_u16x2(of.z, of.w));
            const int k_top = max((int)(tops & 0xffffu) - 1, 0), v_top = max((int)(tops >> 16) - 1, 0);
            if (v_top > ref)
                ref = min(v_top + 1, 254);
            if (cw == 0 && lane == 0)
                s_e[t % (2 * kMaxStages)] = make_int2(k_top, ref);
            if (alive && t >= kst)
                alive = __all_sync(0xffffffffu, mbar_wait_abortable(b_k_empty + 8 * ks, kph, abort_flag));
            if (alive) {
                put(k, k.in, k_top, k_sm + ks * C::kKVBytes);
                fence_proxy_async();
                mbar_arrive(b_k_full + 8 * ks);
            }
            if (alive && t >= vst)
                alive = __all_sync(0xffffffffu, mbar_wait_abortable(b_v_empty + 8 * vs, vph, abort_flag));
            if (alive) {
                put(v, k.in, ref, v_sm + vs * C::kKVBytes);
                fence_proxy_async();
                mbar_arrive(b_v_full + 8 * vs);
            } else {
                status_bits |= PA_STATUS_TIMEOUT;
                *abort_flag = 1;
            }
            if (++ks == kst) {
                ks = 0;
                kph ^= 1u;
            }
            if (++vs == vst) {
                vs = 0;
                vph ^= 1u;
            }
        };
        for (int t = 0; t < ntiles; t += 2) { // (two sets of registers take turns)
            step(t, k, v, k_next, v_next);
            if (t + 1 < ntiles)
                step(t + 1, k_next, v_next, k, v);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        // Order: S(0), S(1), then per tile P.V(t) followed by S(t + 2) into the buffer P(t)
        // occupied; MMAs of one thread run in issue order.
        if (lane == 0) {
            constexpr uint32_t idesc_s = idesc_f16<false>(kTcRows, kTcTok, false);
            constexpr uint32_t idesc_o = idesc_f16<false>(kTcRows, D, true);
            const uint64_t qd = smem_desc_sw128(q_half ? q_sm - C::kQSlice / 2 : q_sm, 16, 1024);
            const uint64_t kd = smem_desc_sw128(k_sm, 16, 1024);
            const uint64_t vd = smem_desc_sw128(v_sm, C::kKVSlice, 1024);
            int ks_next = 0;
            uint32_t kph = 0u;
            auto issue_s = [&](int t) -> bool {
                if (!mbar_wait_abortable(b_k_full + 8 * ks_next, kph, abort_flag))
                    return false;
                tc_fence_after();
                const uint32_t sc = tmem + C::kSCol + (uint32_t)(t & 1) * kTcTok;
                const uint64_t kb = kd + (((uint32_t)ks_next * C::kKVBytes) >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off_q = (ks >> 2) * q_slice + (ks & 3) * 32;
                    const uint32_t off_k = (ks >> 2) * C::kKVSlice + (ks & 3) * 32;
                    tc_mma_ss(sc, qd + (off_q >> 4), kb + (off_k >> 4), idesc_s, ks > 0);
                }
                tc_commit(b_s_full + 8 * (t & 1));
                tc_commit(b_k_empty + 8 * ks_next);
                if (++ks_next == kst) {
                    ks_next = 0;
                    kph ^= 1u;
                }
                return true;
            };
            bool ok = mbar_wait_abortable(b_q_full, 0, abort_flag) && issue_s(0) && (ntiles == 1 || issue_s(1));
            int vs = 0;
            uint32_t vph = 0u;
            for (int t = 0; ok && t < ntiles; ++t) {
                const uint32_t pc = tmem + C::kSCol + (uint32_t)(t & 1) * kTcTok;
                ok = mbar_wait_abortable(b_p_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1u, abort_flag) &&
                     mbar_wait_abortable(b_v_full + 8 * vs, vph, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t vb = vd + (((uint32_t)vs * C::kKVBytes) >> 4);
#pragma unroll
                for (int kt = 0; kt < kTcTok / 16; ++kt)
                    tc_mma_ts(tmem, pc + kt * 8, vb + ((kt * 2048) >> 4), idesc_o, (t > 0 || kt > 0) ? 1u : 0u);
                tc_commit(b_o_done + 8 * (t & 1));
                tc_commit(b_v_empty + 8 * vs);
                if (++vs == vst) {
                    vs = 0;
                    vph ^= 1u;
                }
                if (t + 2 < ntiles)
                    ok = issue_s(t + 2);
            }
            if (!ok) {
                status_bits |= PA_STATUS_TIMEOUT;
                *abort_flag = 1;
            }
            // Every MMA issued has completed once this commit arrives.
            tc_commit(b_drained);
            mbar_wait_bounded(b_drained, 0, kWaitLimitNs);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- rows
        // Q rows -> shared memory; tile row `first` + i is row i there, zero for padding.
        const int first = q_half ? kTcRows / 2 : 0;
        auto q_row = [&](int i) -> const uint8_t * {
            const int x = first + i - roff;
            if (x < 0 || x >= nrows)
                return nullptr;
            const int t = new_token(c0 + x);
            return static_cast<const uint8_t *>(p.query) +
                   ((size_t)(b * p.q_len + t) * p.num_heads + (kv * p.group + c0 + x - t * p.group)) * (D * 2);
        };
        const bool aligned = (reinterpret_cast<uintptr_t>(p.query) & 15) == 0; // (4 bytes are asked for)
        q4_put_rows<D>(warp, lane, kTcRows - first, p.dtype == PA_BF16, aligned, q_sm, q_slice, q_row,
                       [&](int i, float inv) { s_cf[first + i] = inv; });
        asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
        const float cf_row = row_ok ? p.scale * kLog2e * (1.f / (1 << kQ4TcKv)) * s_cf[r] : 0.f;
        fence_proxy_async();
        mbar_arrive(b_q_full);
        if (warp * 32 + 32 > roff) {
            // Visible tokens of this row: tokA <= t < hi (unsigned span from tokA).
            const int hi = row_ok ? min(tokE, L - p.q_len + qi + 1) : tokA;
            const unsigned span = (unsigned)max(hi - tokA, 0);
            const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
            float m_run = -3.4028234663852886e38f, l_run = 0.f;
            int ref = 0;
            bool ok = true;
            for (int t = 0; t < ntiles; ++t) {
                const uint32_t sc = lane_base + C::kSCol + (uint32_t)(t & 1) * kTcTok;
                if (!__all_sync(0xffffffffu, mbar_wait_abortable(b_s_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1u, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int2 es = s_e[t % (2 * kMaxStages)];
                // A score in log2 units is S * cf.
                const float cf = cf_row * __uint_as_float(es.x ? (uint32_t)es.x << 23 : 1u << 22);
                const int off = tok0 + t * kTcTok - tokA; // token (t's first) - tokA
                // Tiles that every row of the warp sees whole skip the masks.
                const bool full = __all_sync(0xffffffffu, !row_ok || (off >= 0 && off + kTcTok <= (int)span));
                // Weights under the present M, and the largest exponent among them.
                uint32_t ph[2][16];
                uint64_t ls, ls2;
                float top;
                auto weigh_as = [&](auto whole_tile) {
                    const uint64_t cf2 = f2_pack(cf, cf), nm2 = f2_pack(kQ4TcUnit - m_run, kQ4TcUnit - m_run);
                    ls = ls2 = 0;
                    top = -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t sr[32];
                        tmem_ld32_async(sc + 32 * h, sr);
                        tmem_ld_wait(sr);
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const uint64_t x = f2_fma(f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), cf2, nm2);
                            float x0, x1;
                            f2_unpack(x, x0, x1);
                            if constexpr (!decltype(whole_tile)::value) {
                                x0 = (unsigned)(off + 32 * h + c) < span ? x0 : -INFINITY;
                                x1 = (unsigned)(off + 32 * h + c + 1) < span ? x1 : -INFINITY;
                            }
                            top = fmax3(top, x0, x1);
                            const float w0 = fast_exp2(x0), w1 = fast_exp2(x1);
                            if (c & 2)
                                ls2 = f2_add(ls2, f2_pack(w0, w1));
                            else
                                ls = f2_add(ls, f2_pack(w0, w1));
                            ph[h][c / 2] = H::pack(w0, w1);
                        }
                    }
                };
                auto weigh = [&]() {
                    if (full)
                        weigh_as(std::true_type());
                    else
                        weigh_as(std::false_type());
                };
                weigh();
                const bool moved = es.y != ref;
                if (__any_sync(0xffffffffu, row_ok && top > kQ4TcUnit + kQ4TcGrow) || moved) {
                    // M moves to the row's maximum, V's reference to the tile's; the row's
                    // scores are still there.
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t sr[32];
                        tmem_ld32_async(sc + 32 * h, sr);
                        tmem_ld_wait(sr);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            mx = fmaxf(mx, (unsigned)(off + 32 * h + c) < span ? __uint_as_float(sr[c]) * cf : -INFINITY);
                    }
                    const float mn = fmaxf(m_run, mx);
                    const float a = fast_exp2(m_run - mn);
                    m_run = mn;
                    l_run *= a;
                    // O is rescaled once the last P.V has landed (tile 0 has no O yet).
                    const float o_by = moved ? a * fast_exp2((float)(ref - es.y)) : a;
                    ref = es.y;
                    if (t > 0 && __any_sync(0xffffffffu, row_ok && o_by != 1.f)) {
                        if (!__all_sync(0xffffffffu, mbar_wait_abortable(b_o_done + 8 * ((t - 1) & 1),
                                                                         (uint32_t)((t - 1) >> 1) & 1u, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < D; cc += 32) {
                            uint32_t o[32];
                            tmem_ld32(lane_base + cc, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * o_by);
                            tmem_st32(lane_base + cc, o);
                        }
                    }
                    weigh();
                }
                // P over S in the same buffer.
                tmem_st16_async(sc, ph[0]);
                tmem_st16_async(sc + 16, ph[1]);
                float l0, l1;
                f2_unpack(f2_add(ls, ls2), l0, l1);
                l_run += l0 + l1;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(b_p_full + 8 * (t & 1));
            }
            // P.V(ntiles - 1), the last MMA.
            if (ok && !__all_sync(0xffffffffu, mbar_wait_abortable(b_o_done + 8 * ((ntiles - 1) & 1),
                                                                  (uint32_t)((ntiles - 1) >> 1) & 1u, abort_flag)))
                ok = false;
            if (!ok) {
                status_bits |= PA_STATUS_TIMEOUT;
                *abort_flag = 1;
            } else {
                tc_fence_after();
                // ---- epilogue: O / l for the row, V's largest scale put back
                const bool seen = !(l_run == 0.f);
                const float inv = 1.f / ((float)(1 << kQ4TcKv) * l_run);
                const float vf = __uint_as_float(ref ? (uint32_t)ref << 23 : 1u << 22);
                const size_t slot = qrow * p.max_num_partitions + part;
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + cc, o);
                    if (!row_ok)
                        continue;
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) // (a row that sees nothing: 0, whatever its O holds)
                        x[k] = seen ? __uint_as_float(o[k]) * inv * vf : 0.f;
                    if (whole) {
                        uint32_t *const out = static_cast<uint32_t *>(p.out) + (qrow * D + cc) / 2;
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            put_pair(out + k / 2, x[k], x[k + 1]);
                    } else {
                        float4 *const tmp = reinterpret_cast<float4 *>(p.tmp_output + slot * D + cc);
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            tmp[k / 4] = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                    }
                }
                if (row_ok && !whole) {
                    p.exp_sums[slot] = l_run * 0.0078125f; // 2^-7
                    p.max_logits[slot] = seen ? m_run * 0.69314718055994531f : -INFINITY;
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
}

template <int D>
static Q4Kernel q4_tc_pick(int mode)
{
    const void *fn = mode == kQ8V1   ? reinterpret_cast<const void *>(&q4_tc_kernel<D, true>)
                     : mode == kQ8V2 ? reinterpret_cast<const void *>(&q4_tc_kernel<D, false>)
                                     : nullptr;
    return {fn, kQ4TcThreads, Q4TcCfg<D>::kCtas, 0};
}

} // namespace pa
