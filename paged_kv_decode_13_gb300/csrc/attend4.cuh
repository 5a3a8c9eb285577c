// Split-K attention over a 4-bit paged cache (sm_103a).
//
// The segment-table attention of the bf16 kernels (same segments, windows,
// rings, left padding, errors) over PKV_FP4 pages.  Grid (C, kv_heads x row
// tiles, segments), the C CTAs along x one thread-block cluster that shares a
// key range.  A CTA holds 8 * NT query rows of one kv head's group; its KW warps
// take every KW-th page of the CTA's range, each with its own ring of NST
// stages: a page block of one kv head is contiguous, so a stage is two bulk
// copies (9 D bytes of K, 9 D of V) on one mbarrier.
//
//   S^T (16 tokens x 8 rows) = K (16 x D) . Q^T
//   O^T (D x 8 rows)        += V^T (D x 16 tokens) . P^T
//
// with fp16 mma.sync and fp32 accumulation.  K and V values are exact in fp16
// (fp4.cuh), and a bf16 query row, scaled by the power of two that brings its
// largest value to [2^14, 2^15), is exact in fp16 down to 2^-31 of that value, so the
// scores are those of the stored values to fp32.  P is rounded to fp16 (2^-11
// relative at most, an eighth of the rounding of a bf16 output).
//
// The lanes read codes in fragment order (fp4.cuh), so a page costs four 16-byte
// and a few narrow shared loads a lane, a conversion (two values) and one fp16
// multiply by the scale for each fragment register, and no shuffles.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include "attend4_launch.h"
#include "fp4.cuh"

namespace pkv {

constexpr int kWaitProbes4 = 1 << 20;  // probes of one barrier phase before PKV_ERR_TIMEOUT
constexpr float kLazy4 = 8.f;          // a row's reference maximum moves when a score passes it by 2^8

template <int D_, int NT_, int KW_, int NST_, int CTAS_>
struct Cfg4 {
    static constexpr int D = D_, NT = NT_, KW = KW_, NST = NST_, kCtas = CTAS_;
    static constexpr int kThreads = KW * 32;
    static constexpr int R = 8 * NT;                 // query rows of a CTA
    static constexpr int kBlock = block4_bytes(D);   // K or V bytes of a page
    static constexpr int kStage = 2 * kBlock;
    static constexpr int KS = D / 16;                // 16-wide steps of S, 16-row tiles of O
    static constexpr bool kQShared = NT > 1;         // Q fragments in shared memory (else in registers)
    static constexpr int LD = D + 4;                 // padded row of a warp's partial
    static constexpr size_t kPartFloats = (size_t)R * LD + 2 * R;
    static constexpr size_t kPipe = (size_t)KW * NST * kStage;
    static constexpr size_t kParts = (size_t)KW * kPartFloats * 4;
    static constexpr size_t kBody = ((kPipe > kParts ? kPipe : kParts) + 127) & ~size_t(127);
    static constexpr size_t kQBytes = kQShared ? (size_t)NT * KS * 32 * 8 : 0;
    static constexpr size_t kRecv = (size_t)R * D * 4 + 16 * 16;
    static constexpr size_t kStat = (size_t)16 * R * 8;
    static constexpr size_t kWeight = (size_t)R * 16 * 4;
    static constexpr size_t kRow = (size_t)R * 3 * 4;
    static constexpr size_t kBars = (size_t)KW * NST * 8;
    static constexpr size_t kSmem = 128 + kBody + kQBytes + kRecv + kStat + kWeight + kRow + kBars + 128;
    static_assert(kSmem <= 232448, "exceeds the per-CTA shared memory limit");
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                              unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned transpose8x8(unsigned x) {
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ unsigned pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&v);
}
// N words from shared memory, 8- or 16-byte aligned.
template <int N>
__device__ __forceinline__ void lds_words(unsigned (&w)[N], const unsigned char *s) {
    if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(s);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(s + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
}

// Four output columns from `at` on.
__device__ __forceinline__ void store_out4(const Attend4Params &p, long long at, float4 v) {
    if (p.out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + at) = v;
}
__device__ __forceinline__ void zero_row4(const Attend4Params &p, long long row, int h0, int heads, int D, int lane, int lanes) {
    for (int e = lane; e < heads * D / 4; e += lanes) store_out4(p, (row * p.Hq + h0) * D + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse)
        for (int e = lane; e < heads; e += lanes) p.lse[row * p.Hq + h0 + e] = -CUDART_INF_F;
}
// Rows of no segment read zero, rows of two set PKV_ERR_OVERLAP: the grid's
// CTAs share the rows, a warp a row at a time, lanes over the segments.
template <int D>
__device__ __noinline__ void coverage4(const Attend4Params &p) {
    const int lane = threadIdx.x & 31;
    const long long cta = blockIdx.x + (long long)gridDim.x * (blockIdx.y + (long long)gridDim.y * blockIdx.z);
    const long long warps = (long long)gridDim.x * gridDim.y * gridDim.z * (blockDim.x >> 5);
    for (long long row = cta * (blockDim.x >> 5) + (threadIdx.x >> 5); row < p.total_rows; row += warps) {
        int n = 0;
        for (int s = lane; s < p.S; s += 32) {
            const int4 v = p.seq_info[s];
            n += v.x >= 0 && v.x <= row && row < (long long)v.x + v.y;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (n == 0) zero_row4(p, row, 0, p.Hq, D, lane, 32);
        if (n > 1 && lane == 0) atomicOr(p.err, PKV_ERR_OVERLAP);
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) attend4_kernel(const __grid_constant__ Attend4Params p) {
    namespace cg = cooperative_groups;
    constexpr int D = C::D, NT = C::NT, KW = C::KW, NST = C::NST, KS = C::KS, R = C::R, LD = C::LD, NTHR = C::kThreads;
    constexpr float kLn2 = 0.6931471805599453f;

    extern __shared__ unsigned char smem_raw[];
    unsigned char *pipe = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint2 *sQ = reinterpret_cast<uint2 *>(pipe + C::kBody);                         // [NT][KS][32]
    float *sRecv = reinterpret_cast<float *>(pipe + C::kBody + C::kQBytes);         // [ncl][per4] float4
    float2 *sStat = reinterpret_cast<float2 *>(reinterpret_cast<unsigned char *>(sRecv) + C::kRecv);  // [16][R]
    float *sW = reinterpret_cast<float *>(sStat + 16 * R);                          // [R][16]
    float *sScale = sW + R * 16;                                                    // [R]
    int *sLo = reinterpret_cast<int *>(sScale + R), *sHi = sLo + R;                 // [R]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sHi + R);                         // [KW][NST]
    int *sFlag = reinterpret_cast<int *>(bars + KW * NST);                          // own flags: 1 bad page, 2 timeout
    int *sAllF = sFlag + 1;                                                         // [16] flags of the cluster

    const int tid = threadIdx.x, kw = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const int rank = blockIdx.x, ncta = gridDim.x;
    const int tile = blockIdx.y % p.row_tiles, h = blockIdx.y / p.row_tiles, s = blockIdx.z;

    if (p.S == 0) {
        pdl_wait();
        pdl_trigger();
        coverage4<D>(p);
        return;
    }
    // ---- the segment and this tile's key range (read before the dependency wait)
    const Segment sg = load_segment(p.seq_info, s);
    unsigned fault = segment_fault(sg, p.total_rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
    if (!fault && sg.ql > p.max_q_len) fault = PKV_ERR_QLEN;
    const int row0 = tile * R;
    const int rows_here = fault ? 0 : min(R, sg.ql * p.G - row0);
    if (rows_here <= 0) {  // uniform across the cluster
        pdl_wait();
        pdl_trigger();
        if (fault && rank == 0) {
            if (tid == 0) atomicOr(p.err, fault);
            if (tile == 0 && sg.q0 >= 0)  // a negative q_start covers nothing
                for (long long r = sg.q0; r < min((long long)sg.q0 + sg.ql, (long long)p.total_rows); ++r)
                    zero_row4(p, r, h * p.G, p.G, D, tid, NTHR);
        }
        coverage4<D>(p);
        return;
    }
    const int kend = sg.kend, new_start = kend - sg.ql;
    const int first = first_valid_of(p.first_valid, sg.col);
    // Bounds grow with the row: the tile's keys are [lo of its first row, hi of
    // its last), and every row sees all of [lo of the last, hi of the first).
    int lo_u, hi_u, lo_in, hi_in;
    row_key_bounds(new_start + row0 / p.G, kend, p.causal, p.window, first, lo_u, hi_in);
    row_key_bounds(new_start + (row0 + rows_here - 1) / p.G, kend, p.causal, p.window, first, lo_in, hi_u);
    const int pb_begin = lo_u / kPage, pb_end = (hi_u + kPage - 1) / kPage, nblk = pb_end - pb_begin;
    // A range of a few pages a warp runs on one CTA, without the cluster's merge.
    const bool solo = nblk <= kSolo4 * KW;
    const int ncl = solo ? 1 : ncta;
    if (rank >= ncl) {
        pdl_wait();
        pdl_trigger();
        coverage4<D>(p);
        return;
    }
    const int bps = (nblk + ncl - 1) / ncl;
    const int cb0 = pb_begin + rank * bps;
    const int nb = max(0, min(bps, pb_end - cb0));
    const int n_mine = nb > kw ? (nb - kw + KW - 1) / KW : 0;
    if (ncl > 1)  // announce this CTA to the cluster; waited on before any remote store
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");

    const int *bt_row = p.block_table + (long long)sg.col * p.mbps;
    uint64_t *wbars = bars + kw * NST;
    unsigned char *wstage = pipe + (size_t)kw * NST * C::kStage;
    if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < NST; ++i) mbar_init(wbars + i, 1);
        fence_barrier_init();
    }
    if (tid == 0) sFlag[0] = 0;
    if (tid < R) {
        int lo = 0, hi = 0;  // padding rows see no key
        if (tid < rows_here) row_key_bounds(new_start + (row0 + tid) / p.G, kend, p.causal, p.window, first, lo, hi);
        sLo[tid] = lo;
        sHi[tid] = hi;
    }
    __syncthreads();

    // ---- page ids and copies (lane l holds the id of the warp's page window + l)
    int id_reg = -1, id_window = -1;
    bool bad = false, timed_out = false;
    auto issue = [&](int j) {
        if ((j & ~31) != id_window) {
            id_window = j & ~31;
            const int li = kw + (id_window + lane) * KW;
            id_reg = li < nb ? bt_row[table_page(cb0 + li, p.ring_rows)] : -1;
        }
        const int bid = __shfl_sync(0xffffffffu, id_reg, j & 31);
        const bool ok = bid >= 0 && (long long)bid < p.num_blocks;
        bad |= !ok;
        if (lane == 0) {
            uint64_t *bar = wbars + j % NST;
            unsigned char *st = wstage + (size_t)(j % NST) * C::kStage;
            if (ok) {
                const size_t at = ((size_t)bid * p.Hkv + h) * C::kBlock;
                fence_proxy_async();  // the stage was read through the generic proxy
                mbar_expect_tx(bar, C::kStage);
                bulk_load(st, p.k + at, C::kBlock, bar);
                bulk_load(st + C::kBlock, p.v + at, C::kBlock, bar);
            } else {
                mbar_arrive(bar);  // nothing to fetch: the result is discarded
            }
        }
    };
    auto wait_page = [&](int j) {
        if (timed_out) return;
        bool done = false;
#pragma unroll 1
        for (int it = 0; it < kWaitProbes4 && !done; ++it) done = mbar_try_wait(wbars + j % NST, (j / NST) & 1);
        if (!__all_sync(0xffffffffu, done)) timed_out = true;
    };
    // Pages wholly below this step's rows are in the cache already, whatever
    // the kernel before this one still writes.
    int issued = 0;
#pragma unroll 1
    for (; issued < NST && issued < n_mine && (cb0 + kw + issued * KW + 1) * kPage <= new_start; ++issued) issue(issued);

    pdl_wait();
    pdl_trigger();

#pragma unroll 1
    for (; issued < NST && issued < n_mine; ++issued) issue(issued);

    // ---- Q^T fragments of one 8-row tile: lane (g, t) holds row g, columns t D/4 ..
    auto load_q = [&](int nt, unsigned (&f)[KS][2]) {
        const int r = nt * 8 + gq;
        const bool real = r < rows_here;
        const int i = (row0 + (real ? r : 0)) / p.G, jh = (row0 + (real ? r : 0)) % p.G;
        const unsigned char *src = reinterpret_cast<const unsigned char *>(
            p.q + (((long long)sg.q0 + i) * p.Hq + (long long)h * p.G + jh) * D + tq * (D / 4));
        unsigned w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 v = real ? *reinterpret_cast<const uint4 *>(src + 16 * c) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
        unsigned mx = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) mx = max(mx, max((w[c] << 16) & 0x7fffffffu, w[c] & 0x7fff0000u));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int k = mx ? min(141 - (int)(mx >> 23), 100) : 0;
        const float up = __uint_as_float((unsigned)(127 + k) << 23);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
            f[c >> 1][c & 1] = pack_f16x2(__uint_as_float(w[c] << 16) * up, __uint_as_float(w[c] & 0xffff0000u) * up);
        return p.scale_log2 * __uint_as_float((unsigned)(127 - k) << 23);
    };
    unsigned qf[C::kQShared ? 1 : KS][2];
    float sc[NT][2];
    if constexpr (!C::kQShared) {
        const float own = load_q(0, qf);
        sc[0][0] = __shfl_sync(0xffffffffu, own, 8 * tq);
        sc[0][1] = __shfl_sync(0xffffffffu, own, 8 * tq + 4);
    } else {
#pragma unroll 1
        for (int nt = kw; nt < NT; nt += KW) {
            unsigned f[KS][2];
            const float own = load_q(nt, f);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) sQ[(nt * KS + kk) * 32 + lane] = make_uint2(f[kk][0], f[kk][1]);
            if (tq == 0) sScale[nt * 8 + gq] = own;
        }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            sc[nt][0] = sScale[nt * 8 + 2 * tq];
            sc[nt][1] = sScale[nt * 8 + 2 * tq + 1];
        }
    }

    // ---- the warp's pages
    float acc[NT][KS][4];
    float m_r[NT][2], l_r[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m_r[nt][0] = m_r[nt][1] = -CUDART_INF_F;
        l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < n_mine; ++j) {
        const unsigned char *st = wstage + (size_t)(j % NST) * C::kStage;
        const int pos0 = (cb0 + kw + j * KW) * kPage;
        wait_page(j);
        // S^T: lane (g, t) holds tokens g and g + 8, columns t D/4 ..
        float sa[NT][4], sb[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sa[nt][e] = sb[nt][e] = 0.f;
        {
            constexpr int W = D / 32;  // code words of a token and lane
            unsigned ka[W], kb[W];
            lds_words<W>(ka, st + gq * (D / 2) + tq * (D / 8));
            lds_words<W>(kb, st + (gq + 8) * (D / 2) + tq * (D / 8));
            unsigned wa, wb;  // scale bytes of the two tokens
            const unsigned char *ss = st + 8 * D + gq * (D / 16) + tq * (D / 64);
            if constexpr (D == 64) {
                wa = ss[0];
                wb = ss[8 * (D / 16)];
            } else if constexpr (D == 128) {
                wa = *reinterpret_cast<const unsigned short *>(ss);
                wb = *reinterpret_cast<const unsigned short *>(ss + 8 * (D / 16));
            } else {
                wa = *reinterpret_cast<const unsigned *>(ss);
                wb = *reinterpret_cast<const unsigned *>(ss + 8 * (D / 16));
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const unsigned fa = scale4_both(wa, w / 2), fb = scale4_both(wb, w / 2);
                unsigned a[4], b[4];
                unpack_e2m1x8(a, ka[w]);
                unpack_e2m1x8(b, kb[w]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = hmul2(a[e], fa);
                    b[e] = hmul2(b[e], fb);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint2 q0, q1;
                    if constexpr (C::kQShared) {
                        q0 = sQ[(nt * KS + 2 * w) * 32 + lane];
                        q1 = sQ[(nt * KS + 2 * w + 1) * 32 + lane];
                    } else {
                        q0 = make_uint2(qf[2 * w][0], qf[2 * w][1]);
                        q1 = make_uint2(qf[2 * w + 1][0], qf[2 * w + 1][1]);
                    }
                    mma_f16_16816(sa[nt], a[0], b[0], a[1], b[1], q0.x, q0.y);
                    mma_f16_16816(sb[nt], a[2], b[2], a[3], b[3], q1.x, q1.y);
                }
            }
        }
        // Online softmax (base 2) with a lazy maximum: this lane has tokens g,
        // g + 8 of rows 2t, 2t + 1.
        const bool inside = pos0 >= lo_in && pos0 + kPage <= hi_in;
        unsigned pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (sa[nt][e] + sb[nt][e]) * sc[nt][e & 1];
            if (!inside) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = pos0 + gq + (e >> 1) * 8, r = nt * 8 + 2 * tq + (e & 1);
                    if (key < sLo[r] || key >= sHi[r]) v[e] = -CUDART_INF_F;
                }
            }
            float mx0 = fmaxf(v[0], v[2]), mx1 = fmaxf(v[1], v[3]);
            if (__any_sync(0xffffffffu, mx0 > m_r[nt][0] + kLazy4 || mx1 > m_r[nt][1] + kLazy4)) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
                }
                const float mn0 = fmaxf(m_r[nt][0], mx0), mn1 = fmaxf(m_r[nt][1], mx1);
                const float al0 = mn0 == -CUDART_INF_F ? 1.f : exp2f(m_r[nt][0] - mn0);
                const float al1 = mn1 == -CUDART_INF_F ? 1.f : exp2f(m_r[nt][1] - mn1);
                m_r[nt][0] = mn0;
                m_r[nt][1] = mn1;
                l_r[nt][0] *= al0;
                l_r[nt][1] *= al1;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    acc[nt][i][0] *= al0; acc[nt][i][1] *= al1;
                    acc[nt][i][2] *= al0; acc[nt][i][3] *= al1;
                }
            }
            const float mu0 = m_r[nt][0] == -CUDART_INF_F ? 0.f : m_r[nt][0], mu1 = m_r[nt][1] == -CUDART_INF_F ? 0.f : m_r[nt][1];
            const float p00 = exp2f(v[0] - mu0), p01 = exp2f(v[1] - mu1), p10 = exp2f(v[2] - mu0), p11 = exp2f(v[3] - mu1);
            l_r[nt][0] += p00 + p10;
            l_r[nt][1] += p01 + p11;
            pb[nt][0] = transpose8x8(pack_f16x2(p00, p01));
            pb[nt][1] = transpose8x8(pack_f16x2(p10, p11));
        }
        // O^T += V^T P^T: lane (g, t) holds columns g D/8 .., tokens 2t, 2t + 1, 2t + 8, 2t + 9
        {
            const unsigned char *sv = st + C::kBlock;
            unsigned fa = 0, fb = 0;
#pragma unroll
            for (int pl = 0; pl < D / 64; ++pl) {
                if (pl % 2 == 0) {
                    unsigned w = *reinterpret_cast<const unsigned *>(sv + 8 * D + (((gq * (D / 8) + pl * 8) / 16) * 4 + tq) * 4);
                    if (!inside) {
                        // Keys that no row sees may hold anything: their scales read zero.  A key
                        // that some rows see may hold a NaN, which must not reach the others
                        // through a zero weight: its scale reads zero too, and the rows that
                        // see it are set to NaN in the columns it scales.
                        unsigned keep = 0, nan = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = pos0 + 2 * tq + (e >> 1) * 8 + (e & 1);
                            const unsigned m = 0xffu << (8 * e);
                            if (key >= lo_u && key < hi_u) {
                                if ((w & m) >= (0xf8u << (8 * e))) nan |= m;
                                else keep |= m;
                            }
                        }
                        w &= keep;
                        if (__any_sync(0xffffffffu, nan != 0)) {
#pragma unroll 1
                            for (int o = 0; o < 16; ++o) {  // tokens of the page; their bytes sit with lane (g, o % 8 / 2)
                                const unsigned b = __shfl_sync(0xffffffffu, nan, (lane & 28) | ((o & 7) >> 1));
                                if (!(b >> (8 * ((o >> 3) * 2 + (o & 1))) & 1u)) continue;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int r = nt * 8 + 2 * tq + e;
                                        if (pos0 + o >= sLo[r] && pos0 + o < sHi[r])
#pragma unroll
                                            for (int k = pl * 4; k < (pl + 2 < D / 64 ? pl + 2 : D / 64) * 4; ++k)
                                                acc[nt][k][e] = acc[nt][k][e + 2] = CUDART_NAN_F;
                                    }
                            }
                        }
                    }
                    fa = scale4_pair(w, 0);
                    fb = scale4_pair(w, 2);
                }
                unsigned vw[4];
                lds_words<4>(vw, sv + pl * 512 + lane * 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    unsigned x[4];
                    unpack_e2m1x8(x, vw[k]);  // (column 0: tokens 2t.., 2t+8..), (column 1: ..)
                    const unsigned a0 = hmul2(x[0], fa), a2 = hmul2(x[1], fb), a1 = hmul2(x[2], fa), a3 = hmul2(x[3], fb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt][pl * 4 + k], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                }
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (j + NST < n_mine) issue(j + NST);
    }
    if (timed_out && lane == 0) {
        // copies still in flight get a bounded chance to land before the stages are reused
#pragma unroll 1
        for (int j = max(0, n_mine - NST); j < n_mine; ++j)
#pragma unroll 1
            for (int it = 0; it < kWaitProbes4 && !mbar_try_wait(wbars + j % NST, (j / NST) & 1); ++it) {
            }
    }
    if ((bad || timed_out) && lane == 0) atomicOr(sFlag, (bad ? 1 : 0) | (timed_out ? 2 : 0));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l_r[nt][0] += __shfl_xor_sync(0xffffffffu, l_r[nt][0], o);
            l_r[nt][1] += __shfl_xor_sync(0xffffffffu, l_r[nt][1], o);
        }
    // A row whose scores are all NaN has no maximum: give it one, so that its
    // NaN sum and columns reach the output.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (m_r[nt][e] == -CUDART_INF_F && l_r[nt][e] != l_r[nt][e]) m_r[nt][e] = 0.f;
    // ---- the warps' partials, over the idle stages of all of them
    __syncthreads();
    {
        float *part = reinterpret_cast<float *>(pipe) + (size_t)kw * C::kPartFloats;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float *r0 = part + (nt * 8 + 2 * tq) * LD + gq * (D / 8), *r1 = r0 + LD;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                *reinterpret_cast<float2 *>(r0 + 2 * i) = make_float2(acc[nt][i][0], acc[nt][i][2]);
                *reinterpret_cast<float2 *>(r1 + 2 * i) = make_float2(acc[nt][i][1], acc[nt][i][3]);
            }
            if (gq == 0) {
                float *st = part + R * LD + nt * 8 + 2 * tq;
                st[0] = m_r[nt][0];
                st[1] = m_r[nt][1];
                st[R] = l_r[nt][0];
                st[R + 1] = l_r[nt][1];
            }
        }
    }
    __syncthreads();
    const int flags = sFlag[0];
    if (tid == 0 && flags) atomicOr(p.err, ((flags & 1) ? PKV_ERR_BLOCK : 0u) | ((flags & 2) ? PKV_ERR_TIMEOUT : 0u));
    auto out_row = [&](int r) {
        const int i = (row0 + r) / p.G, jh = (row0 + r) % p.G;
        return ((long long)sg.q0 + i) * p.Hq + (long long)h * p.G + jh;
    };
    cg::cluster_group cluster = cg::this_cluster();
    const int items = rows_here * (D / 4), per4 = (items + ncl - 1) / ncl;
    if (ncl > 1) {
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");  // every CTA of the cluster runs
        if (tid < ncl) *cluster.map_shared_rank(sAllF + rank, tid) = flags;
    }
#pragma unroll 1
    for (int e = tid; e < items; e += NTHR) {
        const int r = e / (D / 4), c4 = e % (D / 4);
        const float *base = reinterpret_cast<const float *>(pipe);
        float mk[KW], M = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            mk[k] = base[k * C::kPartFloats + R * LD + r];
            M = fmaxf(M, mk[k]);
        }
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            // a warp that saw no key of the row has weight 0 and a zero accumulator
            const float w = mk[k] == -CUDART_INF_F ? 0.f : exp2f(mk[k] - M);
            const float4 v = *reinterpret_cast<const float4 *>(base + k * C::kPartFloats + r * LD + 4 * c4);
            L = fmaf(w, base[k * C::kPartFloats + R * LD + R + r], L);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
        if (ncl == 1) {
            const bool zero = flags || L == 0.f;  // a NaN sum stays: the row holds a NaN
            const float inv = 1.f / L;
            const long long row = out_row(r);
            store_out4(p, row * D + 4 * c4, zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
            if (c4 == 0 && p.lse) p.lse[row] = zero ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
        } else {
            const int owner = e / per4;
            *cluster.map_shared_rank(reinterpret_cast<float4 *>(sRecv) + rank * per4 + (e - owner * per4), owner) = o;
            if (c4 < ncl) *cluster.map_shared_rank(sStat + rank * R + r, c4) = make_float2(M, L);
        }
    }
    if (ncl > 1) {
        cluster.sync();  // publishes every CTA's partials
        int poison = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) poison |= c < ncl ? sAllF[c] : 0;
#pragma unroll 1
        for (int b = 0; b < R * 16; b += NTHR) {  // row, source CTA: normalised weights by 16-lane shuffles
            const int r = (b + tid) >> 4, c = tid & 15;
            const float2 stt = c < ncl && r < rows_here ? sStat[c * R + r] : make_float2(-CUDART_INF_F, 0.f);
            float M = stt.x;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float w = stt.x == -CUDART_INF_F ? 0.f : exp2f(stt.x - M);
            float W = w * stt.y;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
            const bool zero = poison || W == 0.f;
            if (b + tid < R * 16) sW[r * 16 + c] = zero ? 0.f : w / W;
            if (c == 0 && r < rows_here && rank == 0 && p.lse) p.lse[out_row(r)] = zero ? -CUDART_INF_F : (M + log2f(W)) * kLn2;
        }
        __syncthreads();
#pragma unroll 1
        for (int e = tid; e < per4 && rank * per4 + e < items; e += NTHR) {
            const int r = (rank * per4 + e) / (D / 4), c4 = (rank * per4 + e) % (D / 4);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < ncl; ++c) {
                const float w = sW[r * 16 + c];
                const float4 v = reinterpret_cast<const float4 *>(sRecv)[c * per4 + e];
                if (w != 0.f) {  // a zero weight must not touch its partial: a poisoned one may hold NaN
                    o.x = fmaf(w, v.x, o.x);
                    o.y = fmaf(w, v.y, o.y);
                    o.z = fmaf(w, v.z, o.z);
                    o.w = fmaf(w, v.w, o.w);
                }
            }
            store_out4(p, out_row(r) * D + 4 * c4, o);
        }
    }
    coverage4<D>(p);
}

}  // namespace pkv
