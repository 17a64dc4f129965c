// pa_q8.cuh -- attention over a paged cache held in 8 bits (e4m3) with one
// fp32 scale per (block, KV head) for K and for V: phase 1 of split-K decode
// ("V2") and the single-pass form ("V1").
//
//     s_t = scale * ks[blk(t)] * <q, kq_t>,    out = sum_t softmax(s)_t vs[blk(t)] vq_t
//
// Bound by reading the cache, at half the bytes of a 16-bit one; what has to
// fit under that read is twice the arithmetic per byte plus the conversion.
// One CTA owns one (partition, KV head, sequence) and serves up to 16 query
// rows of the GQA group, as the 16-bit kernel does; each warp owns a ring of
// TMA stages and walks every W-th unit (a block, or two 8-token blocks).
//
// Math on mma.sync, fp32 accumulation.  The codes go into the tensor cores as
// they are; the scales stay outside the products.  Tokens (S^T = K Q^T) or dims
// (O^T = V^T P^T) are the M side, query rows the N side, 32 tokens a step.
//   Q.K runs on e4m3 operands (m16n8k32; measured four times the rate of
//   binary16 products per dim).  A query row is scaled by a power of two that
//   brings its largest value to [2^7, 2^8), then split into e4m3 parts, each
//   the rounding of what the parts before it leave: two parts hold bf16's 8
//   significant bits, three hold binary16's 11, exactly down to 2^-10 of the
//   row's largest value and within 2^-17 of it below.  ldmatrix of the 16-byte
//   chunks of the tile is the A fragment as it stands.
//   P.V runs on binary16 operands (m16n8k16): every e4m3 value is a binary16
//   value, two codes are converted by one instruction.  The transposing
//   ldmatrix moves pairs of dims as its 16-bit elements: a lane gets dims (2 g4, 2 g4 + 1) of tokens 2 t4 and
//   2 t4 + 1; one byte permutation gives the two tokens of dim 2 g4 (row g4 of
//   the fragment) and of dim 2 g4 + 1 (row g4 + 8).  O's rows are permuted
//   dims, put right when they are stored.
//
// V's scales go into the softmax's exponent.  With r the largest scale that
// the warp has met and lv_t = log2(vs_t / r), floored at -60,
//     w_t = 2^(s_t + lv_t - M),   O = sum w_t vq_t,   l = sum w_t 2^(-lv_t),
// s in log2 units: O / l * r is the output, and O accumulates in the MMAs'
// registers with no multiplication.  M bounds the weighted exponents, so P's
// rounding (binary16: 2^-12 of each term, below 2^-14 at most 2^-25) is
// relative to the largest contribution, whatever the blocks' scales.  M moves
// only when a weight would pass 2^8 (the first step always), so most steps
// reduce nothing across lanes.  l and M stay a valid pair for the merge:
// l = sum 2^(s_t - M).
//
// Measured on GB300 (batch of 32, up to 8192 tokens, 284 MB of cache; the
// stress shape, 2.1 GB): binary16 products for both with O scaled every 16
// tokens 53.2 and 341 us; this form FIGURES.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_q8.h"

namespace pa {

#ifndef Q8_MB
#define Q8_MB 4
#endif
#ifndef Q8_MB2
#define Q8_MB2 3
#endif
#ifndef Q8_CH
#define Q8_CH 1
#endif
constexpr float kQ8Ln2 = 0.69314718055994531f;

// Two e4m3 codes (the low or high half of x) -> two binary16 values.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x)
{
    uint32_t y;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x)
{
    uint32_t y;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(y) : "r"(x));
    return y;
}

// d (+)= a * b, m16n8k32, e4m3 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^k and 2^-k for the power of two that brings a row whose largest magnitude
// is amax to [2^7, 2^8) (k limited to keep both finite).
__device__ __forceinline__ void q_row_scale_mma(float amax, float &f, float &inv)
{
    const int e = (int)(__float_as_uint(amax) >> 23); // biased exponent
    const int fe = amax > 0.f ? min(127 + 7 - (e - 127), 253) : 127;
    f = __uint_as_float((uint32_t)fe << 23);
    inv = __uint_as_float((uint32_t)(254 - fe) << 23);
}

// Four values -> PL words of four e4m3 codes, word k holding the rounding of
// what the words before it leave.  A value that is not finite gives NaN.
template <int PL>
__device__ __forceinline__ void split_e4m3(float (&x)[4], uint32_t (&w)[PL])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = fabsf(x[i]) <= 3.4028234663852886e38f ? x[i] : NAN;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
        w[k] = lo | (hi << 16);
        const uint32_t a = e4m3_lo(w[k]), b = e4m3_hi(w[k]);
        x[0] -= Elem<__half>::lo(a);
        x[1] -= Elem<__half>::hi(a);
        x[2] -= Elem<__half>::lo(b);
        x[3] -= Elem<__half>::hi(b);
    }
}

__device__ __forceinline__ float fast_lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D, int NT, bool V1>
struct Q8Bounds {
    static constexpr bool kNarrow = !V1 && D <= 128;
    static constexpr int kThreads = kNarrow ? 128 : kMaxWarps * 32;
    static constexpr int kMinBlocks = kNarrow ? (NT == 1 ? Q8_MB : Q8_MB2) : 1;
};

constexpr float kQ8NoMax = -1e30f;  // M before a row has seen a token
constexpr float kQ8Grow = 8.f;      // M moves when a weight would pass 2^8
constexpr float kQ8Floor = -60.f;   // of log2(vs / r)

// PL: e4m3 parts of a query row (2 for bf16, 3 for binary16).
template <int D, int BS, int NT, int PL, bool V1>
__global__ void __launch_bounds__(Q8Bounds<D, NT, V1>::kThreads, Q8Bounds<D, NT, V1>::kMinBlocks)
    q8_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const Q8Params p)
{
    constexpr int kKS = D / 16;                       // 16-dim steps: chunks of a row
    constexpr int kRB = D < 128 ? D : 128;            // bytes of a row in one slice
    constexpr int kSlices = D / kRB;
    constexpr int kUB = BS < 32 ? 32 / BS : 1;        // blocks per unit
    constexpr int kUT = BS * kUB;                     // tokens per unit
    constexpr bool kBf16 = PL == 2;
    using T = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
    constexpr uint32_t kSliceBytes = kUT * kRB;
    constexpr uint32_t kStageBytes = 2 * kSlices * kSliceBytes; // K slices, then V slices
    constexpr int kSteps = kUT / 32;
    constexpr int kHeads = NT * 8;
    constexpr int kScr = D + 4;

    __shared__ uint64_t bars[kMaxWarps * kMaxStages];
    __shared__ float s_factor[kMaxWarps][kMaxGroup];
    __shared__ float s_stat[3][kMaxGroup];
    __shared__ float s_vref[kMaxWarps];
    extern __shared__ uint8_t dyn_smem[];

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5;
    const int g4 = lane >> 2;
    const int t4 = lane & 3;
    const int cgi = V1 ? (int)blockIdx.x : (int)blockIdx.x % p.col_groups;
    const int part = V1 ? 0 : (int)blockIdx.x / p.col_groups;
    const int kv = blockIdx.y;
    const int b = blockIdx.z;

    // Programmatic stream serialisation: nothing global is touched before the
    // previous grid in the stream has completed.
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int head0 = kv * p.group;
    const int col0 = cgi * kHeads;
    const int ncols = min(kHeads, p.cols - col0);
    auto col_row = [&](int n) -> size_t { // row of [S * q_len * H] of local column n
        const int c = col0 + n;
        return ((size_t)b * p.q_len + c / p.group) * p.num_heads + head0 + c % p.group;
    };
    const int tokA = V1 ? 0 : part * p.partition_size;
    const int blk0 = tokA / BS;
    const int range_max =
        V1 ? p.max_blocks
           : (int)min(((long long)tokA + p.partition_size + BS - 1) / BS, (long long)p.max_blocks) -
                 blk0;
    const int32_t *bt_row = p.block_tables + (size_t)b * p.max_blocks + blk0;
    const int Lraw = __ldg(&p.seq_lens[b]);
    // Block ids of the warp's units u = warp + nwarps * i, one unit per lane of a 32-unit chunk.
    auto load_ids = [&](int chunk, int bound, int32_t(&dst)[kUB]) {
        const int u = warp + nwarps * (chunk * 32 + lane);
#pragma unroll
        for (int k = 0; k < kUB; ++k) {
            const int bi = u * kUB + k;
            dst[k] = bi < bound ? __ldg(bt_row + bi) : 0;
        }
    };
    int32_t ids_cur[kUB], ids_next[kUB];
    load_ids(0, range_max, ids_cur);
    load_ids(1, range_max, ids_next);

    // Q^T fragments: row 8 j + g4, dims 32 cp + 4 t4 .. + 3 and 16 up.
    uint32_t qf[NT][kKS / 2][PL][2];
    float q_inv[NT]; // of row 8 j + g4
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = j * 8 + g4;
        const bool has = n < ncols;
        const uint32_t *q32 = static_cast<const uint32_t *>(p.query) + col_row(has ? n : 0) * (D / 2);
        uint32_t raw[kKS][2];
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            raw[ks][0] = has ? __ldg(q32 + ks * 8 + 2 * t4) : 0u;
            raw[ks][1] = has ? __ldg(q32 + ks * 8 + 2 * t4 + 1) : 0u;
        }
        float m = 0.f;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int w = 0; w < 2; ++w)
                m = fmaxf(m, fmaxf(fabsf(Elem<T>::lo(raw[ks][w])), fabsf(Elem<T>::hi(raw[ks][w]))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float f;
        q_row_scale_mma(m, f, q_inv[j]);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            float x[4] = {Elem<T>::lo(raw[ks][0]) * f, Elem<T>::hi(raw[ks][0]) * f,
                          Elem<T>::lo(raw[ks][1]) * f, Elem<T>::hi(raw[ks][1]) * f};
            uint32_t w[PL];
            split_e4m3<PL>(x, w);
#pragma unroll
            for (int k = 0; k < PL; ++k)
                qf[j][ks >> 1][k][ks & 1] = w[k];
        }
    }

    int L = Lraw;
    if (L < 0 || L > p.seq_len_cap) {
        if (threadIdx.x == 0 && part == 0 && kv == 0)
            set_status(p.status, PA_STATUS_BAD_SEQ_LEN);
        L = L < 0 ? 0 : p.seq_len_cap;
    }
    if (!V1 && tokA >= L)
        return; // partition past the end of the sequence
    const int tok0 = blk0 * BS;
    const int lo = tokA - tok0;
    const int ntok = V1 ? L : (int)(min((long long)tokA + p.partition_size, (long long)L) - tok0);
    const int nblk = (ntok + BS - 1) / BS;
    const int nunit = (ntok + kUT - 1) / kUT;
    auto store_out = [&](size_t row, int d, const float4 &v) {
        uint32_t *o = static_cast<uint32_t *>(p.out) + (row * D + d) / 2;
        o[0] = Elem<T>::pack(v.x, v.y);
        o[1] = Elem<T>::pack(v.z, v.w);
    };
    if (V1 && nblk == 0) { // empty sequence: zero output
        for (int idx = threadIdx.x; idx < ncols * (D / 4); idx += blockDim.x)
            store_out(col_row(idx / (D / 4)), (idx % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }

    // Visible tokens of this lane's columns 8 j + 2 t4 (+1), and the factor
    // that turns a raw product into log2 units (but for the block's K scale).
    unsigned vis[NT][2], vis_min = 0xffffffffu;
    float cf[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = j * 8 + 2 * t4 + k;
            const int last = (n < ncols ? L - p.q_len + (col0 + n) / p.group : L - 1) - tok0;
            vis[j][k] = (unsigned)max(min(last + 1, ntok) - lo, 0);
            vis_min = min(vis_min, vis[j][k]);
            // Lane 4 r holds row 8 j + r's factor.
            cf[j][k] = p.scale * __shfl_sync(0xffffffffu, q_inv[j], (2 * t4 + k) * 4) * kLog2e;
        }

    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    const uint32_t smem0 = (smem_addr(dyn_smem) + 1023u) & ~1023u;
    const uint32_t ring = smem0 + (uint32_t)warp * (uint32_t)p.stages * kStageBytes;
    const uint32_t bar0 = smem_addr(&bars[warp * kMaxStages]);
    const int stages = p.stages;
    const int cnt = warp < nunit ? (nunit - warp + nwarps - 1) / nwarps : 0;
    if (lane == 0) {
        for (int s = 0; s < stages; ++s)
            mbar_init(bar0 + 8 * s, 1);
        mbar_init_fence();
    }
    __syncwarp();

    const uint64_t policy = l2_evict_first_policy();
    int32_t status_bits = 0;
    int chunk_cur = 0;
    // Scales of a chunk's blocks, one unit per lane: as loaded for the chunk
    // being issued (sc_new; at most one chunk ahead of the one being computed,
    // the ring being shorter than a chunk), and for the chunk being computed
    // ks, lv and 2^-lv.  Unloaded blocks get 0.
    float sc_new[kUB][2], sc_ks[kUB], sc_lv[kUB], sc_rl[kUB];
    auto load_scales = [&](int chunk) {
        const int u = warp + nwarps * (chunk * 32 + lane);
#pragma unroll
        for (int k = 0; k < kUB; ++k) {
            const bool in = u * kUB + k < nblk;
            int32_t id = ids_cur[k];
            id = id < 0 || id >= p.num_blocks ? 0 : id;
            const size_t at = (size_t)id * p.num_kv_heads + kv;
            sc_new[k][0] = in ? __ldg(p.k_scales + at) : 0.f;
            sc_new[k][1] = in ? __ldg(p.v_scales + at) : 0.f;
        }
    };
    load_scales(0);

    // Issue the TMA loads of the warp's i-th unit into stage s (warp-uniform call).
    auto issue = [&](int i, int s) {
        const int c = i >> 5;
        if (c != chunk_cur) {
#pragma unroll
            for (int k = 0; k < kUB; ++k)
                ids_cur[k] = ids_next[k];
            load_ids(c + 1, nblk, ids_next);
            load_scales(c);
            chunk_cur = c;
        }
        const int u = warp + nwarps * i;
        const int nb = kUB == 1 ? 1 : min(kUB, nblk - u * kUB);
        const uint32_t bar = bar0 + 8 * s;
        const uint32_t dst = ring + (uint32_t)s * kStageBytes;
        if (lane == 0)
            mbar_arrive_expect_tx(bar, kUB == 1 ? kStageBytes : (uint32_t)nb * BS * D * 2u);
#pragma unroll
        for (int k = 0; k < kUB; ++k) {
            int32_t phys = __shfl_sync(0xffffffffu, ids_cur[k], i & 31);
            if (k < nb) {
                if (phys < 0 || phys >= p.num_blocks) {
                    status_bits |= PA_STATUS_BAD_BLOCK_ID;
                    phys = 0; // read a valid block instead of memory outside the cache
                }
                if (lane == 0) {
                    const int row = (int)(((long long)phys * p.num_kv_heads + kv) * BS);
#pragma unroll
                    for (int sl = 0; sl < kSlices; ++sl)
                        tma_load_3d(dst + sl * kSliceBytes + k * BS * kRB, &tmap_k, 0, sl, row, bar,
                                    policy);
#pragma unroll
                    for (int sl = 0; sl < kSlices; ++sl)
                        tma_load_3d(dst + (kSlices + sl) * kSliceBytes + k * BS * kRB, &tmap_v, 0,
                                    sl, row, bar, policy);
                }
            }
        }
    };

    int issued = 0;
    for (; issued < cnt && issued < stages; ++issued)
        issue(issued, issued);

    // Running softmax state (log2 units) of this lane's columns, and the
    // warp's largest V scale.
    float m_run[NT][2], l_run[NT][2], vref = 0.f, vref_lg = 0.f;
    float o[NT][kKS][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        m_run[j][0] = m_run[j][1] = kQ8NoMax;
        l_run[j][0] = l_run[j][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kKS; ++mt)
            o[j][mt][0] = o[j][mt][1] = o[j][mt][2] = o[j][mt][3] = 0.f;
    }
    // Takes the loaded scales into use.  A larger r than before rescales the
    // state so that O stays: M falls and l rises by log2 of its growth, up to
    // 60; growth beyond that scales O down instead.
    auto take_scales = [&]() {
        float v = 1.1754943508222875e-38f; // 2^-126
#pragma unroll
        for (int k = 0; k < kUB; ++k)
            v = fmaxf(v, sc_new[k][1]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        if (v > vref) {
            const float lg = fast_lg2(v);
            if (vref > 0.f) {
                const float up = lg - vref_lg;
                const float d = fminf(up, -kQ8Floor);
                const float f = fast_exp2(d), g = fast_exp2(d - up);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        m_run[j][c] -= d;
                        l_run[j][c] *= f;
                    }
                    if (up > d) {
#pragma unroll
                        for (int mt = 0; mt < kKS; ++mt)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                o[j][mt][c] *= g;
                    }
                }
            }
            vref = v;
            vref_lg = lg;
        }
#pragma unroll
        for (int k = 0; k < kUB; ++k) {
            sc_ks[k] = sc_new[k][0];
            sc_lv[k] = fmaxf(fast_lg2(sc_new[k][1]) - vref_lg, kQ8Floor);
            sc_rl[k] = fast_exp2(-sc_lv[k]);
        }
    };

    // Shared-memory address of 16-byte chunk c of row r in a tile of slices,
    // as TMA swizzles it: 128-byte rows c ^ (r & 7), 64-byte rows c ^ (r >> 1 & 3).
    auto at = [&](uint32_t base, int r, int c) -> uint32_t {
        if (kRB == 128)
            return base + (c >> 3) * kSliceBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        return base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    };
    // ldmatrix lane address: matrix lane >> 3 = (rows 0-7 or 8-15, chunk even or odd).
    const int ld_row = ((lane >> 3) & 1) * 8 + (lane & 7);
    const int ld_chunk = lane >> 4;

    int s = 0;
    uint32_t parity = 0u;
    int i = 0;
    for (; i < cnt; ++i) {
        if (!mbar_wait_bounded(bar0 + 8 * s, parity, kWaitLimitNs)) {
            status_bits |= PA_STATUS_TIMEOUT;
            break;
        }
        if ((i & 31) == 0)
            take_scales();
        const int unit = warp + nwarps * i;
        const int valid = min(kUT, ntok - unit * kUT);
        const uint32_t kbase = ring + (uint32_t)s * kStageBytes;
        const uint32_t vbase = kbase + kSlices * kSliceBytes;
        float ks[kUB], lv[kUB], rl[kUB];
#pragma unroll
        for (int k = 0; k < kUB; ++k) {
            ks[k] = __shfl_sync(0xffffffffu, sc_ks[k], i & 31);
            lv[k] = __shfl_sync(0xffffffffu, sc_lv[k], i & 31);
            rl[k] = __shfl_sync(0xffffffffu, sc_rl[k], i & 31);
        }

        if (valid < kUT) {
            // Rows past the range: zero V so that no stale value reaches P.V.
            const int nchunks = (kUT - valid) * kKS;
            for (int c = lane; c < nchunks; c += 32)
                st_shared_zero16(at(vbase, valid + c / kKS, c % kKS));
            __syncwarp();
        }

#pragma unroll 1
        for (int step = 0; step < kSteps; ++step) {
            if (step * 32 >= valid)
                break;
            const int t0 = step * 32; // first row of the step in the unit
            // Block of the unit that rows 16 tile + 8 half .. + 7 belong to.
            auto blk = [](int tile, int half) { return (tile * 16 + half * 8) / BS; };
            // ---- S^T = K_step Q^T: two 16-token tiles
            constexpr int kChains = Q8_CH; // accumulators per tile and n-tile
            float sacc[2][NT][kChains][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int k = 0; k < kChains; ++k)
                        sacc[t][j][k][0] = sacc[t][j][k][1] = sacc[t][j][k][2] = sacc[t][j][k][3] = 0.f;
#pragma unroll
            for (int cp = 0; cp < kKS / 2; ++cp) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t a[4];
                    ldsm_x4(at(kbase, t0 + t * 16 + ld_row, 2 * cp + ld_chunk), a);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < PL; ++k)
                            mma_e4m3(sacc[t][j][k % kChains], a, qf[j][cp][k][0], qf[j][cp][k][1]);
                }
            }
            float sv[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float x = sacc[t][j][0][c];
#pragma unroll
                        for (int k = 1; k < kChains; ++k)
                            x += sacc[t][j][k][c];
                        sv[t][j][c] = x;
                    }

            // ---- weights: exponents s + lv - M, M moved if one passes 8
            const unsigned r0 = (unsigned)(unit * kUT + t0 + g4 - lo);
            // Every row of the step inside the range and seen by every column.
            const unsigned first = (unsigned)(unit * kUT + t0 - lo);
            const bool full = first < 0x80000000u && first + 32u <= vis_min;
            auto hide = [&](float(&x)[2][NT][4]) {
                if (!full) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                x[t][j][c] = r0 + t * 16u + (c >> 1) * 8u < vis[j][c & 1] ? x[t][j][c]
                                                                                        : -INFINITY;
                }
            };
            float x[2][NT][4], top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        x[t][j][c] = fmaf(sv[t][j][c], cf[j][c & 1] * ks[blk(t, c >> 1)],
                                          lv[blk(t, c >> 1)] - m_run[j][c & 1]);
            hide(x);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        top = fmaxf(top, x[t][j][c]);
            if (__any_sync(0xffffffffu, top > kQ8Grow)) {
                // The exponents without M (M may be -1e30 so far), their
                // maximum over the step's tokens, and the state moved to it.
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            x[t][j][c] = fmaf(sv[t][j][c], cf[j][c & 1] * ks[blk(t, c >> 1)],
                                              lv[blk(t, c >> 1)]);
                hide(x);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(fmaxf(x[0][j][c], x[0][j][c + 2]),
                                         fmaxf(x[1][j][c], x[1][j][c + 2]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float mn = fmaxf(m_run[j][c], mx);
                        const float al = fast_exp2(m_run[j][c] - mn);
                        m_run[j][c] = mn;
                        l_run[j][c] *= al;
#pragma unroll
                        for (int mt = 0; mt < kKS; ++mt) {
                            o[j][mt][c] *= al;
                            o[j][mt][c + 2] *= al;
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            x[t][j][c] -= mn;
                            x[t][j][c + 2] -= mn;
                        }
                    }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w[c] = fast_exp2(x[t][j][c]);
                        l_run[j][c & 1] = fmaf(w[c], rl[blk(t, c >> 1)], l_run[j][c & 1]);
                    }
                    pb[t][j][0] = movmatrix_trans(Elem<__half>::pack(w[0], w[1]));
                    pb[t][j][1] = movmatrix_trans(Elem<__half>::pack(w[2], w[3]));
                }

            // ---- O^T += V_step^T P^T
#pragma unroll
            for (int cp = 0; cp < kKS / 2; ++cp) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t r[4];
                    ldsm_x4_trans(at(vbase, t0 + t * 16 + ld_row, 2 * cp + ld_chunk), r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t y0 = __byte_perm(r[2 * h], 0u, 0x3120);
                        const uint32_t y1 = __byte_perm(r[2 * h + 1], 0u, 0x3120);
                        const uint32_t a[4] = {e4m3_lo(y0), e4m3_hi(y0), e4m3_lo(y1), e4m3_hi(y1)};
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            Elem<__half>::mma(o[j][2 * cp + h], a, pb[t][j][0], pb[t][j][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (issued < cnt) {
            if (valid < kUT)
                fence_proxy_async();
            issue(issued, s);
            ++issued;
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }
    }

    if (status_bits & PA_STATUS_TIMEOUT) {
        // Let copies still in flight into this warp's ring land (bounded again).
        for (int k = i; k < issued; ++k)
            mbar_wait_bounded(bar0 + 8 * (k % stages), (uint32_t)(k / stages) & 1u, kWaitLimitNs);
    }
    if (status_bits && lane == 0)
        set_status(p.status, status_bits);

    // ---- hand the warp's {m, l, o} to the CTA merge (scratch = this warp's own ring)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l_run[j][0] += __shfl_xor_sync(0xffffffffu, l_run[j][0], off);
            l_run[j][1] += __shfl_xor_sync(0xffffffffu, l_run[j][1], off);
        }
    }
    __syncwarp();
    float *scr = reinterpret_cast<float *>(dyn_smem + (ring - smem_addr(dyn_smem)));
    float *scr_m = scr;
    float *scr_l = scr + kHeads;
    float *scr_o = scr + 2 * kHeads; // [kHeads][kScr]
    if (lane == 0)
        s_vref[warp] = vref;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int hA = j * 8 + 2 * t4;
        if (g4 == 0) {
            scr_m[hA] = m_run[j][0];
            scr_m[hA + 1] = m_run[j][1];
            scr_l[hA] = l_run[j][0];
            scr_l[hA + 1] = l_run[j][1];
        }
#pragma unroll
        for (int mt = 0; mt < kKS; ++mt) {
            // Fragment rows g4 and g4 + 8 are dims 2 g4 and 2 g4 + 1.
            const int d = mt * 16 + 2 * g4;
            *reinterpret_cast<float2 *>(scr_o + hA * kScr + d) = make_float2(o[j][mt][0], o[j][mt][2]);
            *reinterpret_cast<float2 *>(scr_o + (hA + 1) * kScr + d) =
                make_float2(o[j][mt][1], o[j][mt][3]);
        }
    }
    __syncthreads();

    // ---- merge the warps: M = max m_w, f_w = 2^(m_w - M), l = sum f_w l_w,
    // o = sum f_w r_w o_w / l
    const uint32_t warp_stride = (uint32_t)stages * kStageBytes / 4;
    const float *scr0 = reinterpret_cast<const float *>(dyn_smem + (smem0 - smem_addr(dyn_smem)));
    if (threadIdx.x < ncols) {
        const int h = threadIdx.x;
        // Warps that saw no token have l = 0 (their M is about -1e30).
        float M = -INFINITY;
        for (int w = 0; w < nwarps; ++w)
            if (scr0[w * warp_stride + kHeads + h] != 0.f)
                M = fmaxf(M, scr0[w * warp_stride + h]);
        float lsum = 0.f;
        for (int w = 0; w < nwarps; ++w) {
            const float lw = scr0[w * warp_stride + kHeads + h];
            const float f = lw != 0.f ? fast_exp2(scr0[w * warp_stride + h] - M) : 0.f;
            s_factor[w][h] = f * s_vref[w];
            lsum = fmaf(f, lw, lsum);
        }
        s_stat[0][h] = M * kQ8Ln2; // natural-log units, as the merge expects
        s_stat[1][h] = lsum;
        s_stat[2][h] = lsum > 0.f ? 1.f / lsum : 0.f;
    }
    __syncthreads();
    constexpr int kQuads = D / 4;
    for (int idx = threadIdx.x; idx < ncols * kQuads; idx += blockDim.x) {
        const int h = idx / kQuads;
        const int d = (idx % kQuads) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < nwarps; ++w) {
            const float f = s_factor[w][h];
            const float4 v =
                *reinterpret_cast<const float4 *>(scr0 + w * warp_stride + 2 * kHeads + h * kScr + d);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        const float inv = s_stat[2][h];
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const size_t bh = col_row(h);
        if (V1) {
            store_out(bh, d, acc);
        } else {
            const size_t slot = bh * p.max_num_partitions + part;
            *reinterpret_cast<float4 *>(p.tmp_output + slot * D + d) = acc;
            if (d == 0) {
                p.exp_sums[slot] = s_stat[1][h];
                p.max_logits[slot] = s_stat[0][h];
            }
        }
    }
}

template <int D>
static const void *q8_kernel_ptr(int block_size, int cols, int dtype, bool v1)
{
#define PA_PICK_V(BS, NT, PL)                                                                     \
    return v1 ? reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, NT, PL, true>)              \
              : reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, NT, PL, false>);
#define PA_PICK(BS)                                                                               \
    if (block_size == BS) {                                                                       \
        if (cols > 8) {                                                                           \
            if (dtype == PA_BF16) {                                                               \
                PA_PICK_V(BS, 2, 2)                                                               \
            }                                                                                     \
            PA_PICK_V(BS, 2, 3)                                                                   \
        }                                                                                         \
        if (dtype == PA_BF16) {                                                                   \
            PA_PICK_V(BS, 1, 2)                                                                   \
        }                                                                                         \
        PA_PICK_V(BS, 1, 3)                                                                       \
    }
    PA_PICK(8)
    PA_PICK(16)
    PA_PICK(32)
    PA_PICK(64)
#undef PA_PICK
#undef PA_PICK_V
    return nullptr;
}

#define PA_DEFINE_Q8_OPS(NAME, D)                                                                 \
    const Q8Ops *NAME()                                                                           \
    {                                                                                             \
        static const Q8Ops ops = {&q8_kernel_ptr<D>};                                             \
        return &ops;                                                                              \
    }

} // namespace pa
