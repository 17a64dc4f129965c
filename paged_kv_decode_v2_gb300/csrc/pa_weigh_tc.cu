// pa_weigh_tc.cu -- accumulated attention weights of many query rows (a window of new
// tokens), on the tcgen05 tensor cores.  The scores would outgrow the keys, so both passes
// compute them:
//
//   totals    S = Q K_t^T, 128 query rows by 128 tokens: a thread per row keeps its
//             running maximum and sum;
//   weights   S = K_t Q^T, 128 tokens by 128 rows: a thread per token adds up its rows'
//             e^(s - M) / total, so that neither pass sums across threads.
//
// The products are one MMA tile for either; only operands change places.  Warp roles: 0-3
// read scores from tensor memory, 4 issues the MMAs and owns that memory, 5-8 bring keys:
// 16-bit ones by cp.async into the 128-byte swizzled rows that the MMA reads; codes through
// registers, as binary16 at the largest scale of the tile's 128 tokens times 2^13 (see
// pa_q4_tc.cuh: 0 below 2^-27 of that scale).  Keys are read twice, from L2 where they fit.
//
// Measured (32 new tokens, 32 heads on 8 of 128, 16-bit keys): 4 sequences of 4096 to 9216
// tokens 34 to 39 us a call (scores kept or computed again by mma.sync: 100 and 87), of 16,384
// 66 us (4.1 TB/s over both passes), of 128 tokens 12: long calls are bound by reading the
// keys, short ones by two launches whose CTAs fetch Q, then keys, then totals.  One wave of
// CTAs: 10 parts for 9.5 per sequence made 320 of them on 304 places, 82 us instead of 66.
// Cutting sequences on the device by their lengths, so that CTAs come out even, cost more
// (9 us) than it gained.
#include <atomic>
#include <type_traits>

#include "pa_weigh.cuh"

namespace pa {

namespace {

constexpr int kThreads = 288;
constexpr int kTok = 128;       // tokens of a tile
constexpr int kMmaWarp = 4, kLoadWarp = 5;
constexpr uint32_t kSlice = kTok * 128; // bytes of 64 dims of a tile, of Q too
constexpr int kKeysUp = 13;     // codes: K times 2^13 at its largest scale
constexpr int kTops = 8;

__host__ __device__ constexpr int stages_of(int D) { return D == 64 ? 4 : 2; }
constexpr size_t smem_of(int D) { return 1024 + (size_t)(1 + stages_of(D)) * (D / 64) * kSlice; }

template <int D, typename T, bool TOTALS>
__global__ void __launch_bounds__((kThreads + 127) / 128 * 128, D <= 128 ? 2 : 1) weigh_tc_kernel(const WeighParams p)
{
    constexpr bool kCodes = sizeof(T) == 1;
    using M = typename std::conditional<kCodes, __half, T>::type; // of the products
    constexpr bool kBf16 = std::is_same<M, __nv_bfloat16>::value;
    constexpr int kStages = stages_of(D);
    constexpr uint32_t kTile = D / 64 * kSlice;
    __shared__ uint64_t k_full[kStages], k_empty[kStages], q_full, s_full[2], s_empty[2], drained;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ int s_top[kTops];      // codes: the largest scale byte of tile t
    __shared__ uint32_t s_most[2][4]; // of each loading warp
    __shared__ __align__(16) float s_cf[kTcRows], s_nm[kTcRows];
    __shared__ float s_sum[TOTALS ? 1 : kWeighTile];
    extern __shared__ uint8_t dyn_smem[];

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // blockIdx.x = (unit * KV + KV head) * row tiles + row tile; units are partitions of
    // sequences, by size where CTAs wait for their turn.  In the second pass a CTA goes
    // through all row tiles of its tokens.
    int unit = blockIdx.x;
    const int rt0 = TOTALS ? unit % p.col_groups : 0;
    unit /= TOTALS ? p.col_groups : 1;
    const int kv = unit % p.num_kv_heads;
    unit /= p.num_kv_heads;
    const bool reporter = TOTALS && kv == 0 && rt0 == 0;
    auto length = [&](int at, bool report) -> int {
        const int len = __ldg(p.seq_lens + at);
        if (len >= 0 && len <= p.seq_len_cap)
            return len;
        if (report)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        return len < 0 ? 0 : p.seq_len_cap;
    };
    int b, part, L;
    const int tok_part = TOTALS ? p.part : p.tile; // a multiple of 128
    if (TOTALS ? p.sorted : p.tiles_sorted) {
        if (!pick_by_size<false, kThreads>(p.num_seqs, tok_part, 32.f / (float)tok_part, unit,
                                           [&](int at) { return length(at, reporter && unit == 0); }, b, part, L))
            return;
    } else {
        const int parts = TOTALS ? p.num_parts : p.num_tiles;
        b = unit / parts;
        part = unit - b * parts;
        L = length(b, reporter && part == 0 && threadIdx.x == 0);
    }
    const int tokA = part * tok_part;
    if (tokA >= L)
        return;
    const int tokE = tokA + min(L - tokA, tok_part);
    const int ntiles = (tokE - tokA + kTok - 1) / kTok;
    const int rt1 = TOTALS ? rt0 + 1 : (p.cols + kTcRows - 1) / kTcRows;
    const int total = (rt1 - rt0) * ntiles;
    auto new_token = [&](int r) -> int { return p.group == 1 ? r : (int)__umulhi((uint32_t)r, p.group_inv); };
    const int rel = L - p.q_len; // new token i sees positions <= rel + i
    // Warps of padding rows only have no scores to read.
    const int nrows0 = min(kTcRows, p.cols - rt0 * kTcRows);
    const int readers = TOTALS ? (nrows0 + 31) / 32 * 32 : kTcRows;

    const uint32_t q_sm = (smem_addr(dyn_smem) + 1023u) & ~1023u, k_sm = q_sm + kTile;
    const uint32_t b_k_full = smem_addr(k_full), b_k_empty = smem_addr(k_empty), b_q_full = smem_addr(&q_full);
    const uint32_t b_s_full = smem_addr(s_full), b_s_empty = smem_addr(s_empty), b_drained = smem_addr(&drained);
    volatile int *const abort_flag = &abort_sh;
    const bool aligned = (reinterpret_cast<uintptr_t>(p.query) & 15) == 0; // (4 bytes are asked for)
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&tmem_base_sh), 2 * kTok);
        tmem_relinquish();
    }
    if (threadIdx.x == kLoadWarp * 32) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(b_k_full + 8 * s, 128);
            mbar_init(b_k_empty + 8 * s, 1);
        }
        mbar_init(b_q_full, 128);
        for (int j = 0; j < 2; ++j) {
            mbar_init(b_s_full + 8 * j, 1);
            mbar_init(b_s_empty + 8 * j, readers);
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

    if (warp >= kLoadWarp) {
        // ---------------------------------------------------------- keys
        // Iteration i: tile i % ntiles.  A warp brings 32 tokens, whose rows its lanes know.
        const int lw = warp - kLoadWarp;
        const int sh = p.block_shift, in_block = (1 << sh) - 1;
        const int32_t *const bt = p.block_tables + (size_t)b * p.max_blocks;
        const uint8_t *const keys = static_cast<const uint8_t *>(p.key_cache);
        const int first = tokA + lw * 32 + lane; // this lane's token of tile 0
        // The block of this lane's token of tile t, or -1 behind the range.
        auto fetch_id = [&](int t) -> int32_t { return first + t * kTok < tokE ? __ldg(bt + ((first + t * kTok) >> sh)) : -1; };
        auto row_of = [&](int32_t id, int t) -> uint32_t {
            if (first + t * kTok >= tokE)
                return 0u;
            if (id < 0 || id >= p.num_blocks) {
                status_bits |= TOTALS ? PA_STATUS_BAD_BLOCK_ID : 0;
                id = 0; // read a valid block instead of memory outside the cache
            }
            return (uint32_t)(((id * p.num_kv_heads + kv) << sh) + ((first + t * kTok) & in_block));
        };
        auto next = [&](int t) -> int { return t + 1 == ntiles ? 0 : t + 1; };
        int ks = 0; // stage of iteration i
        uint32_t kph = 1u;
        bool alive = true;
        auto wait_empty = [&](int i) {
            if (alive && i >= kStages)
                alive = __all_sync(0xffffffffu, mbar_wait_abortable(b_k_empty + 8 * ks, kph, abort_flag));
        };
        auto step_stage = [&]() {
            if (++ks == kStages) {
                ks = 0;
                kph ^= 1u;
            }
        };
        if constexpr (!kCodes) {
            // Four lanes a row, 64 bytes of eight rows a copy: 16-byte chunk c of a row's
            // slice lies at c ^ (row & 7).
            const uint32_t at = lw * 32 * 128 + (lane >> 2) * 128 + (((lane & 3) ^ (lane >> 2)) << 4);
            const uint8_t *const from0 = keys + (lane & 3) * 16;
            auto hand_over = [&](int stage) {
                fence_proxy_async();
                mbar_arrive(b_k_full + 8 * stage);
            };
            int32_t id = fetch_id(0);
            int t = 0, done = 0; // (done: the stage handed over next)
            for (int i = 0; i < total && alive; ++i) {
                const uint32_t row = row_of(id, t);
                const int left = tokE - (tokA + t * kTok + lw * 32); // rows of this warp's 32 in the range
                t = next(t);
                id = fetch_id(t);
                wait_empty(i);
                if (alive) {
                    const uint32_t st = k_sm + ks * kTile + at;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint8_t *const from = row_at<D * 2>(from0, __shfl_sync(0xffffffffu, row, j * 8 + (lane >> 2)));
                        const uint32_t bytes = j * 8 + (lane >> 2) < left ? 16u : 0u;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
                            q4_copy16((st ^ ((c & 1) << 6)) + (c >> 1) * kSlice + j * 1024, from + c * 64, bytes);
                    }
                }
                q4_commit();
                step_stage();
                if (alive && i >= kStages - 1) {
                    q4_wait<kStages - 1>();
                    hand_over(done);
                    done = done + 1 == kStages ? 0 : done + 1;
                }
            }
            q4_wait<0>();
            if (alive)
                for (int i = max(total - (kStages - 1), 0); i < total; ++i) {
                    hand_over(done);
                    done = done + 1 == kStages ? 0 : done + 1;
                }
        } else {
            constexpr int kPieces = D / 32; // of 16 bytes of codes and one scale
            const int token = lw * 32 + lane;
            struct Keys {
                uint4 codes[kPieces];
                uint32_t scales[(kPieces + 3) / 4];
                bool in;
            };
            auto load = [&](int32_t id, int t, Keys &x) {
                x.in = first + t * kTok < tokE;
                const uint32_t row = row_of(id, t);
                const uint4 *const from = reinterpret_cast<const uint4 *>(row_at<D / 2>(keys, row));
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    x.codes[i] = __ldg(from + i);
                const uint8_t *const s = row_at<kPieces>(p.k_scales, row);
                if constexpr (kPieces == 2) {
                    x.scales[0] = __ldg(reinterpret_cast<const uint16_t *>(s));
                } else {
#pragma unroll
                    for (int i = 0; i < kPieces / 4; ++i)
                        x.scales[i] = __ldg(reinterpret_cast<const uint32_t *>(s) + i);
                }
            };
            auto prefetch = [&](int32_t id, int t) {
                if (id < 0 || id >= p.num_blocks)
                    return;
                const uint32_t row = (uint32_t)(((id * p.num_kv_heads + kv) << sh) + ((first + t * kTok) & in_block));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(row_at<D / 2>(keys, row)));
                if ((lane & 7) == 0)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(row_at<kPieces>(p.k_scales, row)));
            };
            // The largest scale byte but 255, plus one.
            auto most_of = [](const Keys &x) -> uint32_t {
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < (kPieces + 3) / 4; ++i) {
                    m = max_u16x2(m, ((x.scales[i] & 0x00ff00ffu) + 0x00010001u) & 0x00ff00ffu);
                    m = max_u16x2(m, ((x.scales[i] >> 8 & 0x00ff00ffu) + 0x00010001u) & 0x00ff00ffu);
                }
                // (the 16-bit load's upper half is no scale)
                if (kPieces == 2)
                    m = max(((x.scales[0] & 255u) + 1u) & 255u, ((x.scales[0] >> 8 & 255u) + 1u) & 255u);
                return !x.in ? 0u : kPieces == 2 ? m : max(m & 0xffffu, m >> 16);
            };
            const uint32_t at = token * 128 + ((token & 7) << 4);
            Keys x, y;
            load(fetch_id(0), 0, x);
            int t = 0;
            int32_t id_next = fetch_id(next(0));
            int t_ahead = next(next(0)); // brought into L2 (the first row tile only)
            int32_t id_ahead = fetch_id(t_ahead);
            auto step = [&](int i, const Keys &x, Keys &y) {
                if (i + 2 < ntiles)
                    prefetch(id_ahead, t_ahead);
                t = next(t);
                load(id_next, t, y);
                id_next = fetch_id(next(t));
                t_ahead = next(t_ahead);
                id_ahead = fetch_id(t_ahead);
                const uint32_t m = __reduce_max_sync(0xffffffffu, most_of(x));
                if (lane == 0)
                    s_most[i & 1][lw] = m;
                asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
                const uint32_t *const of = s_most[i & 1];
                const int top = max((int)max(max(of[0], of[1]), max(of[2], of[3])) - 1, 0);
                wait_empty(i);
                if (alive) {
                    if (token == 0)
                        s_top[i % kTops] = top;
                    const uint32_t tile = k_sm + ks * kTile + at;
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) {
                        const int se = (int)(x.scales[k / 4] >> 8 * (k & 3) & 255u);
                        // 2^(13 + se - top): exponent field 28 + se - top.
                        const int up = max(15 + kKeysUp + se - top, 0);
                        const uint32_t f = !x.in ? 0u : se == 255 ? 0x7fff7fffu : (uint32_t)up * 0x4000400u;
                        const uint32_t w[4] = {x.codes[k].x, x.codes[k].y, x.codes[k].z, x.codes[k].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t h[4];
                            e2m1x8(w[j], h);
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[n]) : "r"(f));
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             (tile ^ (((k & 1) * 4 + j) << 4)) + (k >> 1) * kSlice),
                                         "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                                         : "memory");
                        }
                    }
                    fence_proxy_async();
                    mbar_arrive(b_k_full + 8 * ks);
                }
                step_stage();
            };
            for (int i = 0; i < total; i += 2) { // (two sets of registers take turns)
                step(i, x, y);
                if (i + 1 < total)
                    step(i + 1, y, x);
            }
        }
        if (!alive) {
            status_bits |= PA_STATUS_TIMEOUT;
            *abort_flag = 1;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16<kBf16>(kTcRows, kTok, false);
            const uint64_t qd = smem_desc_sw128(q_sm, 16, 1024), kd = smem_desc_sw128(k_sm, 16, 1024);
            int ks = 0, t = 0;
            uint32_t kph = 0u, qph = 0u;
            bool ok = true;
            for (int i = 0; ok && i < total; ++i) {
                const int j = i & 1;
                if (t == 0) {
                    ok = mbar_wait_abortable(b_q_full, qph, abort_flag);
                    qph ^= 1u;
                }
                ok = ok && mbar_wait_abortable(b_k_full + 8 * ks, kph, abort_flag) &&
                     (i < 2 || mbar_wait_abortable(b_s_empty + 8 * j, (uint32_t)((i >> 1) - 1) & 1u, abort_flag));
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t kb = kd + (((uint32_t)ks * kTile) >> 4);
                const uint64_t a = TOTALS ? qd : kb, c = TOTALS ? kb : qd;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * kSlice + (k & 3) * 32) >> 4;
                    tc_mma_ss(tmem + j * kTok, a + off, c + off, idesc, k > 0);
                }
                tc_commit(b_s_full + 8 * j);
                tc_commit(b_k_empty + 8 * ks);
                if (++ks == kStages) {
                    ks = 0;
                    kph ^= 1u;
                }
                t = t + 1 == ntiles ? 0 : t + 1;
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
        // ---------------------------------------------------------- scores
        const int r = threadIdx.x; // a row of the tile (totals), or a token
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        int i = 0;
        for (int rt = rt0; rt < rt1; ++rt) { // (a warp that gave up still meets the others)
            const int c0 = rt * kTcRows, nrows = min(kTcRows, p.cols - c0), nrows32 = (nrows + 31) / 32 * 32;
            const size_t row0 = ((size_t)b * p.num_kv_heads + kv) * p.cols + c0;
            if (rt > rt0) // the rows before this one's have been used
                asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
            // Q rows into shared memory: as they are beside 16-bit keys; beside codes in
            // binary16 scaled to [2^14, 2^15).  Padding rows are the last row again: weight 0,
            // as their M is infinite, while zeros would make NaN of an infinite key.  (Padding
            // follows the last new token alone, which sees every key.)
            auto row_of = [&](int at) -> const uint8_t * {
                const int x = c0 + min(at, nrows - 1), t = new_token(x);
                return static_cast<const uint8_t *>(p.query) +
                       ((size_t)(b * p.q_len + t) * p.num_heads + (kv * p.group + x - t * p.group)) * (D * 2);
            };
            if constexpr (!kCodes) {
                constexpr int kPieces = D / 8; // 16 bytes each, of a row
                const int piece = lane % kPieces;
#pragma unroll 4
                for (int q = warp; q < nrows32 * kPieces / 32; q += 4) {
                    const int at = (q * 32 + lane) / kPieces;
                    const uint8_t *const from = row_of(at) + piece * 16;
                    const uint32_t to = q_sm + (piece >> 3) * kSlice + at * 128 + (((piece & 7) ^ (at & 7)) << 4);
                    if (aligned) {
                        q4_copy16(to, from, 16u);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * k), "l"(from + 4 * k)
                                         : "memory");
                    }
                }
                q4_commit();
                if (r < nrows32)
                    s_cf[r] = p.scale * kLog2e;
            } else {
                q4_put_rows<D>(warp, lane, nrows32, p.dtype == PA_BF16, aligned, q_sm, kSlice,
                               [&](int at) -> const uint8_t * { return at < nrows ? row_of(at) : nullptr; },
                               [&](int at, float inv) { s_cf[at] = p.scale * kLog2e * inv * (1.f / (1 << kKeysUp)); });
            }
            if constexpr (!TOTALS) {
                // A row's -(M + log2 of its total); a row that sees nothing, or is none: -inf.
                const int parts = (int)(((unsigned)L + p.part - 1) / p.part);
                float m = kWeighNoMax, sum = 0.f;
                if (r < nrows) {
                    constexpr int kMany = 8; // under way at a time (their slots number kWeighParts)
                    const float4 *const mm = reinterpret_cast<const float4 *>(p.maxima + (row0 + r) * kWeighParts);
                    const float4 *const ll = reinterpret_cast<const float4 *>(p.sums + (row0 + r) * kWeighParts);
                    for (int i = 0; i < parts; i += kMany) {
                        float x[kMany], y[kMany];
#pragma unroll
                        for (int k = 0; k < kMany / 4; ++k) {
                            reinterpret_cast<float4 *>(x)[k] = __ldcg(mm + i / 4 + k);
                            reinterpret_cast<float4 *>(y)[k] = __ldcg(ll + i / 4 + k);
                        }
                        float now = m;
#pragma unroll
                        for (int k = 0; k < kMany; ++k)
                            now = fmaxf(now, i + k < parts ? x[k] : kWeighNoMax);
                        sum *= fast_exp2(m - now);
                        m = now;
#pragma unroll
                        for (int k = 0; k < kMany; ++k)
                            sum += i + k < parts ? y[k] * fast_exp2(x[k] - m) : 0.f;
                    }
                }
                if (r < nrows32)
                    s_nm[r] = sum == 0.f ? -INFINITY : -(m + log2f(sum));
            }
            if constexpr (!kCodes)
                q4_wait<0>();
            fence_proxy_async();
            mbar_arrive(b_q_full);
            asm volatile("barrier.cta.sync 2, 128;" ::: "memory");

            if constexpr (TOTALS) {
                if (warp * 32 >= readers)
                    break;
                const bool row_ok = r < nrows;
                const float cf_row = s_cf[r];
                // Visible tokens of this row: tokA <= t < hi (unsigned span from tokA).
                const int hi = row_ok ? min(tokE, rel + new_token(c0 + r) + 1) : tokA;
                const unsigned span = (unsigned)max(hi - tokA, 0);
                float m_run = kWeighNoMax, l_run = 0.f;
                for (; ok && i < total; ++i) {
                    const uint32_t sc = lane_base + (i & 1) * kTok;
                    if (!__all_sync(0xffffffffu, mbar_wait_abortable(b_s_full + 8 * (i & 1), (uint32_t)(i >> 1) & 1u, abort_flag))) {
                        ok = false;
                        *abort_flag = 1;
                        break;
                    }
                    tc_fence_after();
                    float cf = cf_row;
                    if constexpr (kCodes) {
                        const int e = s_top[i % kTops];
                        cf *= __uint_as_float(e ? (uint32_t)e << 23 : 1u << 22);
                    }
                    const int off = i * kTok; // token (tile's first) - tokA
                    const bool full = __all_sync(0xffffffffu, !row_ok || off + kTok <= (int)span);
                    // Sum of weights under the present M, and the largest exponent.
                    float top, l;
                    auto weigh_as = [&](auto whole) {
                        const uint64_t cf2 = f2_pack(cf, cf), nm2 = f2_pack(-m_run, -m_run);
                        uint64_t ls[2] = {0, 0};
                        top = -INFINITY;
                        uint32_t sr[2][32];
                        tmem_ld32_async(sc, sr[0]);
#pragma unroll
                        for (int h = 0; h < kTok / 32; ++h) {
                            tmem_ld_wait(sr[h & 1]);
                            if (h + 1 < kTok / 32)
                                tmem_ld32_async(sc + 32 * (h + 1), sr[(h + 1) & 1]);
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[h & 1][c]), __uint_as_float(sr[h & 1][c + 1])), cf2, nm2), x0, x1);
                                if constexpr (!decltype(whole)::value) {
                                    x0 = (unsigned)(off + 32 * h + c) < span ? x0 : -INFINITY;
                                    x1 = (unsigned)(off + 32 * h + c + 1) < span ? x1 : -INFINITY;
                                }
                                top = fmax3(top, x0, x1);
                                ls[c >> 1 & 1] = f2_add(ls[c >> 1 & 1], f2_pack(fast_exp2(x0), fast_exp2(x1)));
                            }
                        }
                        float l0, l1;
                        f2_unpack(f2_add(ls[0], ls[1]), l0, l1);
                        l = l0 + l1;
                    };
                    auto weigh = [&]() {
                        if (full)
                            weigh_as(std::true_type());
                        else
                            weigh_as(std::false_type());
                    };
                    if (i > 0)
                        weigh();
                    if (i == 0 || __any_sync(0xffffffffu, row_ok && top > kWeighGrow)) {
                        // M moves to the row's maximum; the row's scores are still there.
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int h = 0; h < kTok / 32; ++h) {
                            uint32_t sr[32];
                            tmem_ld32_async(sc + 32 * h, sr);
                            tmem_ld_wait(sr);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                mx = fmaxf(mx, (unsigned)(off + 32 * h + c) < span ? __uint_as_float(sr[c]) * cf : -INFINITY);
                        }
                        const float mn = fmaxf(m_run, mx);
                        l_run *= fast_exp2(m_run - mn);
                        m_run = mn;
                        weigh();
                    }
                    l_run += l;
                    tc_fence_before();
                    mbar_arrive(b_s_empty + 8 * (i & 1));
                }
                if (ok && row_ok) {
                    p.maxima[(row0 + r) * kWeighParts + part] = m_run;
                    p.sums[(row0 + r) * kWeighParts + part] = l_run;
                }
            } else {
                const uint32_t cf_at = smem_addr(s_cf), nm_at = smem_addr(s_nm);
                for (int t = 0; ok && t < ntiles; ++t, ++i) {
                    const uint32_t sc = lane_base + (i & 1) * kTok;
                    const int pos = tokA + t * kTok + r;
                    // The weight of earlier calls, asked for early.
                    float *slot = nullptr;
                    float old = 0.f;
                    if (rt + 1 == rt1 && pos < tokE) {
                        slot = weight_at(p, b, kv, pos);
                        // (The newest tokens have none, whatever their slots hold; 0 times what is not
                        // finite would be NaN.)
                        if (slot && pos < rel && p.decay != 0.f)
                            old = *slot;
                    }
                    if (!__all_sync(0xffffffffu, mbar_wait_abortable(b_s_full + 8 * (i & 1), (uint32_t)(i >> 1) & 1u, abort_flag))) {
                        ok = false;
                        *abort_flag = 1;
                        break;
                    }
                    tc_fence_after();
                    uint64_t up = f2_pack(1.f, 1.f);
                    if constexpr (kCodes) {
                        const int e = s_top[i % kTops];
                        const float x = __uint_as_float(e ? (uint32_t)e << 23 : 1u << 22);
                        up = f2_pack(x, x);
                    }
                    // First row that sees this token: new token i = (c0 + r) / group sees it
                    // when i >= pos - rel.
                    const long long i0 = (long long)pos - rel;
                    const long long first = i0 > 0 ? i0 * p.group - c0 : 0;
                    const int r_min = first > kTcRows ? kTcRows : (int)max(first, 0ll);
                    uint64_t ws[2] = {0, 0};
                    auto weigh_as = [&](auto whole) {
#pragma unroll 1
                        for (int c0 = 0; c0 < nrows32; c0 += 32) {
                            uint32_t sr[32];
                            tmem_ld32_async(sc + c0, sr);
                            tmem_ld_wait(sr);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                uint32_t cf[4], nm[4];
                                lds_words(cf_at + (c0 + c) * 4, cf);
                                lds_words(nm_at + (c0 + c) * 4, nm);
#pragma unroll
                                for (int k = 0; k < 4; k += 2) {
                                    uint64_t cf2 = f2_pack(__uint_as_float(cf[k]), __uint_as_float(cf[k + 1]));
                                    if constexpr (kCodes)
                                        cf2 = f2_fma(cf2, up, 0);
                                    float x0, x1;
                                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c + k]), __uint_as_float(sr[c + k + 1])), cf2,
                                                     f2_pack(__uint_as_float(nm[k]), __uint_as_float(nm[k + 1]))), x0, x1);
                                    if constexpr (!decltype(whole)::value) {
                                        x0 = c0 + c + k >= r_min ? x0 : -INFINITY;
                                        x1 = c0 + c + k + 1 >= r_min ? x1 : -INFINITY;
                                    }
                                    ws[k >> 1] = f2_add(ws[k >> 1], f2_pack(fast_exp2(x0), fast_exp2(x1)));
                                }
                            }
                        }
                    };
                    if (__all_sync(0xffffffffu, r_min == 0))
                        weigh_as(std::true_type());
                    else
                        weigh_as(std::false_type());
                    tc_fence_before();
                    mbar_arrive(b_s_empty + 8 * (i & 1));
                    float w0, w1;
                    f2_unpack(f2_add(ws[0], ws[1]), w0, w1);
                    float w = w0 + w1;
                    if (rt > rt0)
                        w += s_sum[t * kTok + r];
                    if (rt + 1 < rt1)
                        s_sum[t * kTok + r] = w;
                    else if (slot)
                        *slot = fmaf(old, p.decay, w);
                }
            }
        }
        if (!ok)
            status_bits |= PA_STATUS_TIMEOUT;
    }

    if (status_bits)
        set_status(p.status, status_bits);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kTok);
    }
}

std::atomic<int> g_prepared[64][2][9]; // [pass][type, head_dim]

template <int D, typename T, bool TOTALS>
cudaError_t launch(const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    const auto fn = &weigh_tc_kernel<D, T, TOTALS>;
    if (g_prepared[dev][TOTALS][cell].load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(D));
        if (e != cudaSuccess)
            return e;
        g_prepared[dev][TOTALS][cell].store(1, std::memory_order_release);
    }
    void *args[] = {const_cast<WeighParams *>(&p)};
    const long long units = TOTALS ? (long long)p.col_groups * p.num_parts : p.num_tiles;
    return launch_pdl(fn, (unsigned)(p.num_seqs * (long long)p.num_kv_heads * units), kThreads, stream, args, smem_of(D));
}

template <int D, typename T>
cudaError_t both(const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    const cudaError_t e = launch<D, T, true>(p, dev, cell, stream);
    return e != cudaSuccess ? e : launch<D, T, false>(p, dev, cell, stream);
}

template <typename T>
cudaError_t pick_dim(int head_dim, const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    return head_dim == 64    ? both<64, T>(p, dev, cell, stream)
           : head_dim == 128 ? both<128, T>(p, dev, cell + 1, stream)
                             : both<256, T>(p, dev, cell + 2, stream);
}

} // namespace

int weigh_tc_ctas(int head_dim) { return head_dim <= 128 ? 2 : 1; }
int weigh_tc_threads() { return kThreads; }

cudaError_t launch_weigh_tc(int head_dim, const WeighParams &p, int dev, cudaStream_t stream)
{
    return p.k_scales           ? pick_dim<uint8_t>(head_dim, p, dev, 6, stream)
           : p.dtype == PA_BF16 ? pick_dim<__nv_bfloat16>(head_dim, p, dev, 3, stream)
                                : pick_dim<__half>(head_dim, p, dev, 0, stream);
}

} // namespace pa
