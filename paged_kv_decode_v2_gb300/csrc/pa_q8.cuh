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
// Math on mma.sync m16n8k16 with binary16 operands and fp32 accumulation.
// Every e4m3 value is a binary16 value, so the codes are converted two at a
// time (one instruction) and never rounded; the scales stay outside the
// products.  Tokens (S^T = K Q^T) or dims (O^T = V^T P^T) are the M side, query rows the
// N side.  The 8-bit tiles need no other layout than the one TMA writes:
//   K: ldmatrix moves 16-byte rows, so a lane holds four consecutive dims
//      4 t4 .. 4 t4 + 3 of token g4.  The contraction runs over dims in any
//      order as long as Q uses the same: k-index pair (2 t4, 2 t4 + 1) is
//      dims (4 t4, 4 t4 + 1), pair (2 t4 + 8, + 9) dims (4 t4 + 2, + 3), and
//      Q's fragment loads those four dims as one 8-byte word.
//   V: the transposing ldmatrix moves pairs of dims as its 16-bit elements: a
//      lane gets dims (2 g4, 2 g4 + 1) of tokens 2 t4 and 2 t4 + 1.  One byte
//      permutation gives the two tokens of dim 2 g4 (row g4 of the fragment)
//      and of dim 2 g4 + 1 (row g4 + 8): O's rows are permuted dims, put
//      right when they are stored.
// Q is binary16 too.  bf16 queries are scaled by a power of two per row that
// brings the row's largest value to [2^14, 2^15): their 8 bits then fit
// exactly down to 2^-28 of that value, and smaller ones are off by at most
// 2^-39 of it.
// P (<= 1) is rounded to binary16's 11 bits: each term moves by at most 2^-12
// of itself, and P below 2^-14 by at most 2^-25.
// V's scale multiplies the block's fp32 product, O = O a + vs (V^T P^T), so
// no block's scale ever limits another block's precision (with two 8-token
// blocks in one product, the smaller scale's ratio to the larger goes into P).
#pragma once

#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_q8.h"

namespace pa {

constexpr float kLn2 = 0.69314718055994531f;

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

// mma with a zero accumulator on input.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 1 / 2^k and 2^k for the power of two that brings a row whose largest
// magnitude is amax to [2^14, 2^15) (k limited to keep both finite).
__device__ __forceinline__ void q_row_scale(float amax, float &f, float &inv)
{
    const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent
    const int fe = amax > 0.f ? min(127 + 14 - (e - 127), 253) : 127;
    f = __uint_as_float((uint32_t)fe << 23);
    inv = __uint_as_float((uint32_t)(254 - fe) << 23);
}

template <int D, int NT, bool V1>
struct Q8Bounds {
    static constexpr bool kNarrow = !V1 && D <= 128;
    static constexpr int kThreads = kNarrow ? 128 : kMaxWarps * 32;
    static constexpr int kMinBlocks = kNarrow ? (NT == 1 ? 4 : 3) : 1;
};

template <int D, int BS, int NT, bool V1>
__global__ void __launch_bounds__(Q8Bounds<D, NT, V1>::kThreads, Q8Bounds<D, NT, V1>::kMinBlocks)
    q8_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const Q8Params p)
{
    constexpr int kKS = D / 16;                       // 16-dim steps: chunks of a row
    constexpr int kRB = D < 128 ? D : 128;            // bytes of a row in one slice
    constexpr int kSlices = D / kRB;
    constexpr int kUB = BS < 16 ? 16 / BS : 1;        // blocks per unit
    constexpr int kUT = BS * kUB;                     // tokens per unit
    constexpr uint32_t kSliceBytes = kUT * kRB;
    constexpr uint32_t kStageBytes = 2 * kSlices * kSliceBytes; // K slices, then V slices
    constexpr int kTiles = kUT / 16;
    constexpr int kHeads = NT * 8;
    constexpr int kScr = D + 4;

    __shared__ uint64_t bars[kMaxWarps * kMaxStages];
    __shared__ float s_factor[kMaxWarps][kMaxGroup];
    __shared__ float s_stat[3][kMaxGroup];
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

    // Q^T fragments (see above): row 8 j + g4, dims 16 ks + 4 t4 .. + 3.
    uint32_t qf[NT][kKS][2];
    float q_inv[NT]; // of row 8 j + g4
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = j * 8 + g4;
        const bool has = n < ncols;
        const uint32_t *q32 = static_cast<const uint32_t *>(p.query) + col_row(has ? n : 0) * (D / 2);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            qf[j][ks][0] = has ? __ldg(q32 + ks * 8 + 2 * t4) : 0u;
            qf[j][ks][1] = has ? __ldg(q32 + ks * 8 + 2 * t4 + 1) : 0u;
        }
        q_inv[j] = 1.f;
        if (p.dtype == PA_BF16) {
            using B = Elem<__nv_bfloat16>;
            float m = 0.f;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    m = fmaxf(m, fmaxf(fabsf(B::lo(qf[j][ks][w])), fabsf(B::hi(qf[j][ks][w]))));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            float f;
            q_row_scale(m, f, q_inv[j]);
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    qf[j][ks][w] = Elem<__half>::pack(B::lo(qf[j][ks][w]) * f, B::hi(qf[j][ks][w]) * f);
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
        if (p.dtype == PA_BF16) {
            o[0] = Elem<__nv_bfloat16>::pack(v.x, v.y);
            o[1] = Elem<__nv_bfloat16>::pack(v.z, v.w);
        } else {
            o[0] = Elem<__half>::pack(v.x, v.y);
            o[1] = Elem<__half>::pack(v.z, v.w);
        }
    };
    if (V1 && nblk == 0) { // empty sequence: zero output
        for (int idx = threadIdx.x; idx < ncols * (D / 4); idx += blockDim.x)
            store_out(col_row(idx / (D / 4)), (idx % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }

    // Visible tokens of this lane's columns 8 j + 2 t4 (+1), and the factor
    // that turns a raw product into log2 units (but for the block's K scale).
    unsigned vis[NT][2];
    float cf[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = j * 8 + 2 * t4 + k;
            const int last = (n < ncols ? L - p.q_len + (col0 + n) / p.group : L - 1) - tok0;
            vis[j][k] = (unsigned)max(min(last + 1, ntok) - lo, 0);
            // Lane 4 r holds row 8 j + r's factor.
            cf[j][k] = p.scale * __shfl_sync(0xffffffffu, q_inv[j], (2 * t4 + k) * 4) * kLog2e;
        }

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
    // Scales of a chunk's blocks, one unit per lane: sc_use for the chunk being
    // computed, sc_new for the one being issued (at most one chunk ahead, the
    // ring being shorter than a chunk).  Unloaded blocks get 0.
    float sc_use[kUB][2], sc_new[kUB][2];
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
#pragma unroll
    for (int k = 0; k < kUB; ++k) {
        sc_use[k][0] = sc_new[k][0];
        sc_use[k][1] = sc_new[k][1];
    }

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

    // Running softmax state (log2 units) of this lane's columns.
    float m_run[NT][2], l_run[NT][2];
    float o[NT][kKS][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        m_run[j][0] = m_run[j][1] = -INFINITY;
        l_run[j][0] = l_run[j][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kKS; ++mt)
            o[j][mt][0] = o[j][mt][1] = o[j][mt][2] = o[j][mt][3] = 0.f;
    }

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
        if (i > 0 && (i & 31) == 0) {
#pragma unroll
            for (int k = 0; k < kUB; ++k) {
                sc_use[k][0] = sc_new[k][0];
                sc_use[k][1] = sc_new[k][1];
            }
        }
        const int unit = warp + nwarps * i;
        const int valid = min(kUT, ntok - unit * kUT);
        const uint32_t kbase = ring + (uint32_t)s * kStageBytes;
        const uint32_t vbase = kbase + kSlices * kSliceBytes;
        // The unit's scales: rows r and r + 8 of a tile (one block unless two
        // 8-token blocks share the unit).
        float ks[2], vr[2], vs;
        ks[0] = __shfl_sync(0xffffffffu, sc_use[0][0], i & 31);
        vs = __shfl_sync(0xffffffffu, sc_use[0][1], i & 31);
        ks[1] = ks[0];
        vr[0] = vr[1] = 1.f;
        if constexpr (kUB == 2) {
            ks[1] = __shfl_sync(0xffffffffu, sc_use[1][0], i & 31);
            const float v0 = vs, v1 = __shfl_sync(0xffffffffu, sc_use[1][1], i & 31);
            vs = fmaxf(v0, v1);
            vr[0] = vs > 0.f ? v0 / vs : 0.f;
            vr[1] = vs > 0.f ? v1 / vs : 0.f;
        }

        if (valid < kUT) {
            // Rows past the range: zero V so that no stale value reaches P.V.
            const int nchunks = (kUT - valid) * kKS;
            for (int c = lane; c < nchunks; c += 32)
                st_shared_zero16(at(vbase, valid + c / kKS, c % kKS));
            __syncwarp();
        }

#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile) {
            if (tile * 16 >= valid)
                break;
            // ---- S^T = K_tile Q^T
            float sacc[NT][2][4]; // two chains per n-tile
#pragma unroll
            for (int cp = 0; cp < kKS / 2; ++cp) {
                uint32_t r[4];
                ldsm_x4(at(kbase, tile * 16 + ld_row, 2 * cp + ld_chunk), r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {e4m3_lo(r[2 * h]), e4m3_lo(r[2 * h + 1]),
                                           e4m3_hi(r[2 * h]), e4m3_hi(r[2 * h + 1])};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (cp == 0)
                            mma_f16_zero(sacc[j][h], a, qf[j][2 * cp + h][0], qf[j][2 * cp + h][1]);
                        else
                            Elem<__half>::mma(sacc[j][h], a, qf[j][2 * cp + h][0],
                                              qf[j][2 * cp + h][1]);
                    }
                }
            }

            // ---- mask and streaming softmax, in log2 units
            const unsigned r0 = (unsigned)(unit * kUT + tile * 16 + g4 - lo);
            uint32_t pb[NT][2];
            float al[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float sv[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sv[c] = r0 + (c >> 1) * 8u < vis[j][c & 1]
                                ? (sacc[j][0][c] + sacc[j][1][c]) * (cf[j][c & 1] * ks[c >> 1])
                                : -INFINITY;
                float mx0 = fmaxf(sv[0], sv[2]);
                float mx1 = fmaxf(sv[1], sv[3]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
                }
                const float mn0 = fmaxf(m_run[j][0], mx0);
                const float mn1 = fmaxf(m_run[j][1], mx1);
                // A column with no visible token yet (max still -inf) keeps l = o = 0.
                al[j][0] = mn0 != -INFINITY ? fast_exp2(m_run[j][0] - mn0) : 1.f;
                al[j][1] = mn1 != -INFINITY ? fast_exp2(m_run[j][1] - mn1) : 1.f;
                m_run[j][0] = mn0;
                m_run[j][1] = mn1;
                const float mb0 = mn0 != -INFINITY ? mn0 : 0.f, mb1 = mn1 != -INFINITY ? mn1 : 0.f;
                float pv[4];
                pv[0] = fast_exp2(sv[0] - mb0);
                pv[1] = fast_exp2(sv[1] - mb1);
                pv[2] = fast_exp2(sv[2] - mb0);
                pv[3] = fast_exp2(sv[3] - mb1);
                l_run[j][0] = fmaf(l_run[j][0], al[j][0], pv[0] + pv[2]);
                l_run[j][1] = fmaf(l_run[j][1], al[j][1], pv[1] + pv[3]);
                if constexpr (kUB == 2) {
                    pv[0] *= vr[0];
                    pv[1] *= vr[0];
                    pv[2] *= vr[1];
                    pv[3] *= vr[1];
                }
                pb[j][0] = movmatrix_trans(Elem<__half>::pack(pv[0], pv[1]));
                pb[j][1] = movmatrix_trans(Elem<__half>::pack(pv[2], pv[3]));
            }

            // ---- O^T = O^T a + vs (V_tile^T P^T)
#pragma unroll
            for (int cp = 0; cp < kKS / 2; ++cp) {
                uint32_t r[4];
                ldsm_x4_trans(at(vbase, tile * 16 + ld_row, 2 * cp + ld_chunk), r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = __byte_perm(r[2 * h], 0u, 0x3120);
                    const uint32_t y = __byte_perm(r[2 * h + 1], 0u, 0x3120);
                    const uint32_t a[4] = {e4m3_lo(x), e4m3_hi(x), e4m3_lo(y), e4m3_hi(y)};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float acc[4];
                        mma_f16_zero(acc, a, pb[j][0], pb[j][1]);
                        float(&oo)[4] = o[j][2 * cp + h];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            oo[c] = fmaf(acc[c], vs, oo[c] * al[j][c & 1]);
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

    // ---- merge the warps: M = max m_w, f_w = 2^(m_w - M), l = sum f_w l_w, o = sum f_w o_w / l
    const uint32_t warp_stride = (uint32_t)stages * kStageBytes / 4;
    const float *scr0 = reinterpret_cast<const float *>(dyn_smem + (smem0 - smem_addr(dyn_smem)));
    if (threadIdx.x < ncols) {
        const int h = threadIdx.x;
        float M = -INFINITY;
        for (int w = 0; w < nwarps; ++w)
            M = fmaxf(M, scr0[w * warp_stride + h]);
        float lsum = 0.f;
        for (int w = 0; w < nwarps; ++w) {
            const float mw = scr0[w * warp_stride + h];
            const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
            s_factor[w][h] = f;
            lsum = fmaf(f, scr0[w * warp_stride + kHeads + h], lsum);
        }
        s_stat[0][h] = M * kLn2; // natural-log units, as the merge expects
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
static const void *q8_kernel_ptr(int block_size, int cols, bool v1)
{
#define PA_PICK(BS)                                                                               \
    if (block_size == BS) {                                                                       \
        if (cols > 8)                                                                             \
            return v1 ? reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, 2, true>)           \
                      : reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, 2, false>);         \
        return v1 ? reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, 1, true>)               \
                  : reinterpret_cast<const void *>(&q8_attn_kernel<D, BS, 1, false>);             \
    }
    PA_PICK(8)
    PA_PICK(16)
    PA_PICK(32)
    PA_PICK(64)
#undef PA_PICK
    return nullptr;
}

#define PA_DEFINE_Q8_OPS(NAME, D)                                                                 \
    const Q8Ops *NAME()                                                                           \
    {                                                                                             \
        static const Q8Ops ops = {&q8_kernel_ptr<D>};                                             \
        return &ops;                                                                              \
    }

} // namespace pa
