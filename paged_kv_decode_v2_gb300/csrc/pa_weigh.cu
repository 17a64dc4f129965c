// pa_weigh.cu -- the attention weight that each cached token receives, added up over
// calls:
//     a_t = decay * a_t (0 for the q_len newest tokens) + sum over the KV head's rows r
//           of softmax_r(scale <q_r, K_.>)_t.
//
// A row's total is known only behind its last token, so there are two passes.  Few new
// tokens (this file): the first writes the scores (fp32, in log2 units) beside each
// partition's maximum and sum, and the second turns them into weights and sums them over
// the rows; the keys are read once, and scores of a decode step, rows * 4 bytes a token
// and head beside 34 (4-bit, 64 dims) to 512 bytes of keys, mostly stay in L2.  From
// kWeighAgain new tokens on they are computed twice instead (pa_weigh_tc.cu): kept, those of
// 16 new tokens of one head take 128 bytes a token, written and read, beside a 4-bit key's 68.
// Both forms, us (kept, twice; head_dim 128, 16 sequences of up to 8192 tokens unless it says
// otherwise): 2 new tokens of 4 heads per KV head 24 and 93; 8 of 4, 4 bits 57 and 94, 16 bits
// 65 and 95; 15 of 4, 117 and 109, 121 and 98, of 256 dims (8 sequences) 73 and 96; a window of
// 32 of 4 (4 sequences, 16 bits) 100 and 36.  The rule does not ask for heads: with many of them
// twice comes out ahead earlier (4 new tokens of 16 heads 52 and 38, 16 bits 52 and 31; 8 of 8
// 67 and 61, 69 and 54; 8 sequences, 8 of 16, 59 and 34, 59 and 24).
//
// Tokens are the M side of mma.sync, 8 query rows an N tile; a lane's 16 bytes of 8
// consecutive dims of a row (or the 8 codes of a word, see pa_q4_attn.cuh) take the places
// of two K-steps' fragments.  Warps walk their own tiles through their own rings, filled
// by cp.async; a lane keeps its own maximum and sum, and lanes and warps meet at the end.
// Sums are fp32 in a fixed order: results do not depend on timing (but in the slot of a token
// that several sequences of a call hold).
//
// Measured: the newest tokens of 32 sequences of up to 8192 tokens, 32 heads on 8 of 128,
// 4 bits, 34 to 38 us a call (by lengths): scores 29 (73 MB of keys; 58% of the issue slots),
// weights 14 alone, the launches partly behind one another.  Cut for two waves of CTAs, five
// partitions of up to 1664 tokens, 36.2 us; for one (2816) 40.9, for three (1152) 35.7, but 27.1
// for 24.4 (2 new tokens of 16 sequences) and 69 for 64 (16-bit keys of 256 dims).
#include <atomic>
#include <type_traits>

#include "pa_weigh.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

// What a K row is: 16-bit values of T, or (T = uint8_t) codes.
template <int D, typename T>
struct KeyTile {
    static constexpr bool kCodes = sizeof(T) == 1;
    using M = typename std::conditional<kCodes, __half, T>::type; // of the products
    static constexpr int kTok = kCodes ? 4096 / D : D == 64 ? 32 : 16;
    static constexpr int kRB = kCodes ? D / 2 : D * 2;
    static constexpr int kSB = kCodes ? D / kQ4Group : 0;
    static constexpr uint32_t kStage = kTok * (kRB + kSB);
    // Row r's 16-byte piece i lies at i ^ swizzle(r), so that the fragments' loads of 8
    // rows (codes: a word each; 16 bits: 16 bytes, two rows at a time) meet no conflict.
    static __device__ __forceinline__ int swizzle(int r)
    {
        return !kCodes ? (r & 1) << 2 : D == 64 ? (r >> 2) & 1 : D == 128 ? (r >> 1) & 3 : r & 7;
    }
};

// CTAs that registers let share an SM, and ring stages: many rows compute longer on a tile.
// (Shared memory holds as many over codes; over 16-bit keys three, and of head_dim 256 one up to
// 16 rows, two above.)
__host__ __device__ constexpr int ctas_of(int nt) { return nt <= 2 ? 4 : 3; }
__host__ __device__ constexpr int stages_of(int nt) { return nt <= 2 ? 4 : 2; }

constexpr int kSumRows = 64;

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, ctas_of(NT)) scores_kernel(const WeighParams p)
{
    using K = KeyTile<D, T>;
    constexpr int kStages = stages_of(NT);
    using M = Elem<typename K::M>;
    constexpr int kR = 8 * NT, kG = D / 32, kQRow = D * 2 + 64;
    __shared__ float s_cf[kR];
    __shared__ float s_m[kWarps][kR], s_l[kWarps][kR];
    __shared__ __align__(16) uint8_t s_q[kR * kQRow];
    extern __shared__ __align__(16) uint8_t dyn_smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, g8 = lane >> 2;

    // blockIdx.x = (unit * KV + KV head) * row tiles + row tile; units are partitions of
    // sequences, by size where CTAs wait for their turn.
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
    int b, part, L;
    if (p.sorted) {
        if (!pick_by_size<false, kThreads>(p.num_seqs, p.part, 32.f / (float)p.part, unit,
                                           [&](int at) { return length(at, reporter && unit == 0); }, b, part, L))
            return;
    } else {
        b = unit / p.num_parts;
        part = unit - b * p.num_parts;
        L = length(b, reporter && part == 0 && threadIdx.x == 0);
    }
    const int tokA = part * p.part;
    if (tokA >= L)
        return;
    const int tokE = tokA + min(L - tokA, p.part);
    auto new_token = [&](int r) -> int { return p.group == 1 ? r : (int)__umulhi((uint32_t)r, p.group_inv); };
    const int rel = L - p.q_len; // new token i sees positions <= rel + i

    const int ntiles = (tokE - tokA + K::kTok - 1) / K::kTok;
    const int mine = warp < ntiles ? (ntiles - warp + kWarps - 1) / kWarps : 0;
    const int sh = p.block_shift, in_block = (1 << sh) - 1;
    const int32_t *bt = p.block_tables + (size_t)b * p.max_blocks;
    const uint32_t ring = smem_addr(dyn_smem) + warp * kStages * K::kStage;
    // Lane l holds where 8 tokens l % kOct of tile base + l / kOct begin, kPer tiles at a time.
    constexpr int kOct = K::kTok / 8, kPer = 32 / kOct;
    auto fetch_rows = [&](int base) -> int {
        const int i = base + lane / kOct;
        const int tok = tokA + (warp + i * kWarps) * K::kTok + lane % kOct * 8;
        if (i >= mine || tok >= tokE)
            return 0;
        int id = __ldg(bt + (tok >> sh));
        if (id < 0 || id >= p.num_blocks) {
            set_status(p.status, PA_STATUS_BAD_BLOCK_ID);
            id = 0; // read a valid block instead of memory outside the cache
        }
        return (id * p.num_kv_heads + kv) << sh; // (all rows number less than 2^31)
    };
    int rows_now = 0, rows_next = fetch_rows(0);
    const uint8_t *const keys = static_cast<const uint8_t *>(p.key_cache);
    auto issue = [&](int i) {
        if (i < mine) {
            const int at = i % kPer;
            if (at == 0) { // (the first rows were asked for ahead)
                rows_now = rows_next;
                rows_next = fetch_rows(i + kPer < mine ? i + kPer : 0);
            }
            const int t0 = tokA + (warp + i * kWarps) * K::kTok;
            const uint32_t st = ring + (uint32_t)(i % kStages) * K::kStage;
            constexpr int kPieces = K::kRB / 16;
#pragma unroll
            for (int q = 0; q < K::kTok * kPieces / 32; ++q) {
                const int row = (q * 32 + lane) / kPieces, piece = lane % kPieces;
                const int r0 = __shfl_sync(0xffffffffu, rows_now, at * kOct + row / 8);
                const size_t src = (size_t)(r0 + ((t0 + row) & in_block)) * K::kRB + piece * 16;
                q4_copy16(st + row * K::kRB + ((piece ^ K::swizzle(row)) << 4), keys + src, t0 + row < tokE ? 16u : 0u);
            }
            if constexpr (K::kCodes) {
                const int row = (lane & 7) * (16 / K::kSB);
                const int r0 = __shfl_sync(0xffffffffu, rows_now, at * kOct + row / 8);
                if (lane < 8) {
                    const size_t src = (size_t)(r0 + ((t0 + row) & in_block)) * K::kSB;
                    q4_copy16(st + K::kTok * K::kRB + lane * 16, p.k_scales + src,
                           (uint32_t)min(max((tokE - t0 - row) * K::kSB, 0), 16));
                }
            }
        }
        q4_commit();
    };
    const uint32_t q_sm = smem_addr(s_q);
    const int c0 = rt * kR, nrows = min(kR, p.cols - c0);
    const size_t row0 = ((size_t)b * p.num_kv_heads + kv) * p.cols + c0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        issue(i);

    // ---- Q rows into shared memory, a warp per row: as they are beside 16-bit keys;
    // beside codes in binary16 scaled to [2^14, 2^15).
    for (int r = warp; r < kR; r += kWarps) {
        constexpr int kDW = D / 64; // words of a lane
        const int x = c0 + (r < nrows ? r : 0), i = new_token(x);
        const uint32_t *q32 = static_cast<const uint32_t *>(p.query) +
                              ((size_t)(b * p.q_len + i) * p.num_heads + (kv * p.group + x - i * p.group)) * (D / 2) +
                              lane * kDW;
        uint32_t w[kDW];
#pragma unroll
        for (int k = 0; k < kDW; ++k)
            w[k] = r < nrows ? __ldg(q32 + k) : 0u;
        float cf = p.scale * kLog2e;
        if constexpr (K::kCodes) {
            float v[2 * kDW], m = 0.f;
#pragma unroll
            for (int k = 0; k < kDW; ++k) {
                v[2 * k] = p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::lo(w[k]) : Elem<__half>::lo(w[k]);
                v[2 * k + 1] = p.dtype == PA_BF16 ? Elem<__nv_bfloat16>::hi(w[k]) : Elem<__half>::hi(w[k]);
                m = fmaxf(m, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            float f, inv;
            q4_row_scale(m, f, inv);
            cf *= inv;
#pragma unroll
            for (int k = 0; k < kDW; ++k)
                w[k] = Elem<__half>::pack(q4_scaled(v[2 * k], f), q4_scaled(v[2 * k + 1], f));
        }
        if (lane == 0)
            s_cf[r] = cf;
#pragma unroll
        for (int k = 0; k < kDW; ++k)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(q_sm + r * kQRow + (lane * kDW + k) * 4), "r"(w[k]) : "memory");
    }
    __syncthreads();

    const uint32_t q_at = q_sm + g8 * kQRow + c * 16;
    float nm[NT][2], l[NT][2], cf[NT][2]; // rows nt * 8 + 2 c + j: -M, of this lane's tokens
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            cf[n][j] = s_cf[n * 8 + 2 * c + j];
            nm[n][j] = -kWeighNoMax;
            l[n][j] = 0.f;
        }
    // Scores of row 2 c, the lane's first token; rows n * 8 + j from there.
    float *const out = p.scores + (row0 + 2 * c) * p.row_stride + g8, *const out1 = out + p.row_stride;
    const long long n_step = 8 * p.row_stride;
    const int tok_all = min(tokE, rel + (p.q_len == 1 ? 0 : new_token(c0)) + 1);
    for (int i = 0; i < mine; ++i) {
        q4_wait<kStages - 2>();
        __syncwarp();
        issue(i + kStages - 1); // into the stage that tile i - 1 has left
        const int t0 = tokA + (warp + i * kWarps) * K::kTok;
        const uint32_t st = ring + (uint32_t)(i % kStages) * K::kStage;
        const bool full = t0 + K::kTok <= tok_all;
#pragma unroll 1
        for (int u = 0; u < K::kTok; u += 16) {
            const int r0 = u + g8, r1 = r0 + 8;
            float s[NT][4];
            float sc0[kG], sc1[kG];
            if constexpr (K::kCodes) {
                const uint32_t at = st + K::kTok * K::kRB;
                q4_scales<kG>(at + r0 * K::kSB, sc0);
                q4_scales<kG>(at + r1 * K::kSB, sc1);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[n][k] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                uint32_t x0[4], x1[4];
                if constexpr (K::kCodes) {
                    e2m1x8(lds32(st + r0 * K::kRB + ((g ^ K::swizzle(r0)) << 4) + c * 4), x0);
                    e2m1x8(lds32(st + r1 * K::kRB + ((g ^ K::swizzle(r1)) << 4) + c * 4), x1);
                } else {
                    lds_words(st + r0 * K::kRB + (((g * 4 + c) ^ K::swizzle(r0)) << 4), x0);
                    lds_words(st + r1 * K::kRB + (((g * 4 + c) ^ K::swizzle(r1)) << 4), x1);
                }
                const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t q[4];
                    lds_words(q_at + n * 8 * kQRow + g * 64, q);
                    if constexpr (K::kCodes) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        M::mma(acc, a0, q[0], q[1]);
                        M::mma(acc, a1, q[2], q[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float f = k < 2 ? sc0[g] : sc1[g];
                            s[n][k] = g == 0 ? acc[k] * f : fmaf(acc[k], f, s[n][k]);
                        }
                    } else {
                        M::mma(s[n], a0, q[0], q[1]);
                        M::mma(s[n], a1, q[2], q[3]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[n][k] *= cf[n][k & 1];
            if (!full) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // First visible row of a token: new token i = (c0 + r) / group sees it
                    // when i >= pos - rel.
                    const int pos = t0 + (h ? r1 : r0);
                    const long long i0 = (long long)pos - rel;
                    const long long first = i0 > 0 ? i0 * p.group - c0 : 0;
                    const int r_min = pos >= tokE || first > kR ? kR : (int)max(first, 0ll);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (n * 8 + 2 * c + j < r_min)
                                s[n][2 * h + j] = -INFINITY;
                }
            }
            float *to = out + t0 + u, *to1 = out1 + t0 + u; // rows n * 8 + 2 c, and the next
            const bool in0 = t0 + r0 < tokE, in1 = t0 + r1 < tokE;
#pragma unroll
            for (int n = 0; n < NT; ++n, to += n_step, to1 += n_step) {
                const bool a = n * 8 + 2 * c < nrows, d = n * 8 + 2 * c + 1 < nrows;
                if (a && in0)
                    to[0] = s[n][0];
                if (d && in0)
                    to1[0] = s[n][1];
                if (a && in1)
                    to[8] = s[n][2];
                if (d && in1)
                    to1[8] = s[n][3];
            }
            // (-inf for the hidden: their weights are 0)
            float x[NT][4], top = -INFINITY;
            auto exponents = [&]() {
                top = -INFINITY;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[n][k] = s[n][k] + nm[n][k & 1];
                    top = fmax3(top, x[n][0], x[n][1]);
                    top = fmax3(top, x[n][2], x[n][3]);
                }
            };
            exponents();
            if (__any_sync(0xffffffffu, top > kWeighGrow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float now = fminf(nm[n][j], -fmaxf(s[n][j], s[n][2 + j]));
                        l[n][j] *= fast_exp2(now - nm[n][j]);
                        nm[n][j] = now;
                    }
                exponents();
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    l[n][k & 1] += fast_exp2(x[n][k]);
        }
    }
    q4_wait<0>();
    // ---- lanes, then warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, nm[n][j], off);
                const float ol = __shfl_xor_sync(0xffffffffu, l[n][j], off);
                const float least = fminf(nm[n][j], om);
                l[n][j] = l[n][j] * fast_exp2(least - nm[n][j]) + ol * fast_exp2(least - om);
                nm[n][j] = least;
            }
            if (g8 == 0) {
                s_m[warp][n * 8 + 2 * c + j] = -nm[n][j];
                s_l[warp][n * 8 + 2 * c + j] = l[n][j];
            }
        }
    __syncthreads();
    if (threadIdx.x < nrows) {
        const int r = threadIdx.x;
        float top = s_m[0][r], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            top = fmaxf(top, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            sum += s_l[w][r] * fast_exp2(s_m[w][r] - top);
        p.maxima[(row0 + r) * kWeighParts + part] = top;
        p.sums[(row0 + r) * kWeighParts + part] = sum;
    }
}

constexpr int kSumThreads = 256;

template <int V>
__device__ __forceinline__ void load_v(const float *from, float (&x)[V])
{
    if constexpr (V == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(from));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(from));
        x[0] = v.x, x[1] = v.y;
    }
}

// A thread per V tokens, of one block: their weights of all rows, kAhead of which are on
// their way at a time.  HIDES: several new tokens, the last of which the first do not see.
template <int V, int kAhead, bool HIDES>
__global__ void __launch_bounds__(kSumThreads, V * kAhead <= 16 ? 6 : 4) weights_kernel(const WeighParams p, int tiles)
{
    constexpr int kSumTokens = V * kSumThreads;
    __shared__ float s_m[kSumRows], s_inv[kSumRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    int unit = blockIdx.x;
    const int tile = unit % tiles;
    unit /= tiles;
    const int kv = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
    const int t = tile * kSumTokens + V * (int)threadIdx.x;
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.seq_len_cap);
    if (tile * kSumTokens >= L)
        return;
    const size_t row0 = ((size_t)b * p.num_kv_heads + kv) * p.cols;
    const float *const scores = p.scores + row0 * p.row_stride + t;
    float sc[kAhead][V];
    auto fetch = [&](int base) { // (a row's scores end on a multiple of 32)
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t < L && base + i < p.cols)
                load_v(scores + (base + i) * p.row_stride, sc[i]);
    };
    fetch(0);
    float *at = nullptr;
    float now[V] = {};
    if (t < L) {
        at = weight_at(p, b, kv, t);
        if (at && p.decay != 0.f) // (0 times what is not finite would be NaN)
            load_v(at, now);
    }
    const int parts = (int)(((unsigned)L + p.part - 1) / p.part);
    float sum[V] = {};
    auto add_rows = [&](auto masked) {
        // First row that sees a token: new token i = row / group sees it when i >= t - (L - q_len).
        int first[V];
#pragma unroll
        for (int k = 0; k < V; ++k)
            first[k] = t + k < L ? max(t + k - (L - p.q_len), 0) * p.group : 0;
        for (int base = 0; base < p.cols; base += kSumRows) {
            const int n = min(kSumRows, p.cols - base);
            __syncthreads();
            // A row's maximum and total: four threads a row.
            const int r = threadIdx.x >> 2, q = threadIdx.x & 3;
            if (r < n) {
                float top, total;
                row_total(p, row0 + base + r, parts, q, top, total);
                if (q == 0) {
                    s_m[r] = top;
                    s_inv[r] = total == 0.f ? 0.f : 1.f / total; // (a row that sees nothing)
                }
            }
            __syncthreads();
            for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (t < L && i0 + i < n) {
                        const float m = s_m[i0 + i], inv = s_inv[i0 + i];
#pragma unroll
                        for (int k = 0; k < V; ++k) {
                            const float more = fmaf(fast_exp2(sc[i][k] - m), inv, sum[k]);
                            if constexpr (decltype(masked)::value)
                                sum[k] = base + i0 + i >= first[k] ? more : sum[k];
                            else
                                sum[k] = more;
                        }
                    }
                }
                fetch(base + i0 + kAhead);
            }
        }
    };
    // Scores of hidden tokens are -inf, but 0 times the share of a row that is not finite is
    // NaN: where a tile holds some, they are passed over.  (A kernel of its own for one new
    // token: 36.2 us for 32 sequences, 37.1 with this branch.)
    if (HIDES && tile * kSumTokens + kSumTokens - 1 > L - p.q_len)
        add_rows(std::bool_constant<HIDES>());
    else
        add_rows(std::false_type());
    if (!at)
        return;
    // The newest tokens have no weight of earlier calls, whatever their slots hold.
#pragma unroll
    for (int k = 0; k < V; ++k)
        now[k] = t + k < L - p.q_len ? fmaf(now[k], p.decay, sum[k]) : sum[k];
    // Slots behind the last token may be another sequence's, whose update would be lost under
    // one of this thread's: they are not written.
    if (t + V <= L) {
        if constexpr (V == 4)
            *reinterpret_cast<float4 *>(at) = make_float4(now[0], now[1], now[2], now[3]);
        else
            *reinterpret_cast<float2 *>(at) = make_float2(now[0], now[1]);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (t + k < L)
                at[k] = now[k];
    }
}

std::atomic<int> g_prepared[64][3 * 3 * 4]; // [type, head_dim, rows]

template <int D, int NT, typename T>
cudaError_t launch_scores(const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    const auto fn = &scores_kernel<D, NT, T>;
    const size_t smem = kWarps * stages_of(NT) * KeyTile<D, T>::kStage;
    if (g_prepared[dev][cell].load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
        g_prepared[dev][cell].store(1, std::memory_order_release);
    }
    void *args[] = {const_cast<WeighParams *>(&p)};
    return launch_pdl(fn, (unsigned)(p.num_seqs * (long long)p.num_kv_heads * p.col_groups * p.num_parts), kThreads, stream, args, smem);
}

template <int D, typename T>
cudaError_t pick_rows(int rows, const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    switch (rows) {
    case 8: return launch_scores<D, 1, T>(p, dev, cell, stream);
    case 16: return launch_scores<D, 2, T>(p, dev, cell + 1, stream);
    case 32: return launch_scores<D, 4, T>(p, dev, cell + 2, stream);
    default: return launch_scores<D, 8, T>(p, dev, cell + 3, stream);
    }
}

template <typename T>
cudaError_t pick_dim(int head_dim, int rows, const WeighParams &p, int dev, int cell, cudaStream_t stream)
{
    return head_dim == 64    ? pick_rows<64, T>(rows, p, dev, cell, stream)
           : head_dim == 128 ? pick_rows<128, T>(rows, p, dev, cell + 4, stream)
                             : pick_rows<256, T>(rows, p, dev, cell + 8, stream);
}

template <bool HIDES>
auto weights_fn(int cols)
{
    return cols > 32  ? &weights_kernel<2, 16, HIDES>
           : cols > 4 ? &weights_kernel<4, 8, HIDES>
                      : &weights_kernel<4, 4, HIDES>;
}

} // namespace

int weigh_ctas(int rows) { return ctas_of(rows / 8); }
int weigh_threads() { return kThreads; }

cudaError_t launch_weigh(int head_dim, int rows, const WeighParams &p, int dev, cudaStream_t stream)
{
    const cudaError_t e = p.k_scales           ? pick_dim<uint8_t>(head_dim, rows, p, dev, 24, stream)
                          : p.dtype == PA_BF16 ? pick_dim<__nv_bfloat16>(head_dim, rows, p, dev, 12, stream)
                                               : pick_dim<__half>(head_dim, rows, p, dev, 0, stream);
    if (e != cudaSuccess)
        return e;
    // Many rows: fewer tokens per thread, more rows ahead.  Few: only they ahead, and more
    // CTAs (32 sequences of up to 8192 tokens, 4 rows, 37.5 us with 4 ahead and 6 CTAs an SM,
    // 38.5 with 8 and 4; one of 100,000, 8 rows, 24.1 and 22.6).
    const int per = (p.cols > 32 ? 2 : 4) * kSumThreads;
    int tiles = (p.seq_len_cap + per - 1) / per;
    void *args[] = {const_cast<WeighParams *>(&p), &tiles};
    const unsigned grid = (unsigned)((long long)p.num_seqs * p.num_kv_heads * tiles);
    return p.q_len > 1 ? launch_pdl(weights_fn<true>(p.cols), grid, kSumThreads, stream, args)
                       : launch_pdl(weights_fn<false>(p.cols), grid, kSumThreads, stream, args);
}

} // namespace pa
