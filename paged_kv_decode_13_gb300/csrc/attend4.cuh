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
// scores are those of the stored values to fp32.  P is rounded to fp16: by
// at most 2^-11 of itself (an eighth of the rounding of a bf16 output), or, where it is
// below 2^-21 of its row's largest weight, by at most 2^-32 of that.
//
// The lanes read codes in fragment order (fp4.cuh), so a page costs four 16-byte
// and a few narrow shared loads a lane, a conversion (two values) and one fp16
// multiply by the scale for each fragment register, and no shuffles.
//
// A page of one kv head (2,304 bytes at D = 128) costs a warp about 300 issue slots, a
// quarter of them conversions (two a value pair at half rate), so four
// or five warps an SM sub-partition are needed to keep up with HBM: CTAs of four
// warps, four an SM for 8 rows.  Sequences of equal length stream at 0.8 to
// 0.9 of the rate of a copy once a CTA has some 100 pages; short calls are a chain of
// launch (2.5 us), tables and first pages (2 us), and the merge (1 to 2 us).
// Eight warps a CTA double the pages in flight for few ranges.  At most 8 rows,
// head_dim 128: 300 keys 6.4 us, 8192 keys 9.1 us (the launch, the
// merge), 32 sequences of up to 16384 keys 58 us (37 at the rate of a copy; HBM 57 %
// busy: starts and ends of 1,000 pieces); head_dim 256, 4 x 131072 keys 107
// us (89; HBM 73 %).  More splits, one large CTA an SM, sixteen warps and
// integer unpacking (2.2 times the conversion's time) were slower.
//
// Two ways to cut the work.  attend4_kernel: a cluster a range, its size by the
// cost of clusters, partials merged through distributed shared memory.
// balance4_kernel: one wave of CTAs, equal shares of all ranges end to
// end, partials of shared ranges merged by a second launch; it evens out lengths that differ.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include "attend4_launch.h"
#include "fp4.cuh"

namespace pkv {

constexpr int kWaitProbes4 = 1 << 20;  // probes of one barrier phase before PKV_ERR_TIMEOUT
constexpr float kNoMax = -1e30f;       // reference maximum of a row that has seen no key
// Weights are 2^(score - reference).  A row's reference is set 7 below the score
// that moves it, and moves again when a score passes it by 15: the largest weight
// is then between 2^7 and 2^15, within fp16, and weights down to 2^-21 of 2^7 are normal
// numbers of it (set at the score itself, those below 2^-25 of the largest would vanish from
// the product with V while the sum still counts them).
constexpr float kLift4 = 7.f, kLazy4 = 15.f;

template <int D_, int NT_, int KW_, int NST_, int PP_, int CTAS_, bool QSH_>
struct Cfg4 {
    static constexpr int D = D_, NT = NT_, KW = KW_, NST = NST_, kCtas = CTAS_;
    static constexpr int PP = PP_;                   // pages of a stage
    static constexpr int kThreads = KW * 32;
    static constexpr int R = 8 * NT;                 // query rows of a CTA
    static constexpr int kBlock = block4_bytes(D);   // K or V bytes of a page
    static constexpr int kPageBytes = 2 * kBlock;    // a page's K block, then its V block
    static constexpr int kStage = PP * kPageBytes;
    static constexpr int KS = D / 16;                // 16-wide steps of S, 16-row tiles of O
    static constexpr bool kQShared = QSH_;           // Q fragments in shared memory (else in registers)
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
    static_assert(NT == 1 || kQShared, "wider tiles keep Q in shared memory");
    static_assert(kSmem <= 232448, "exceeds the per-CTA shared memory limit");
};

// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                              unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^x for x <= about 15; results below fp32's normal range are zero.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
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
__device__ __noinline__ void cover_rows4(const Attend4Params &p, long long row) {
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * gridDim.y * gridDim.z * (blockDim.x >> 5);
    for (; row < p.total_rows; row += warps) {
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
template <int D>
__device__ __forceinline__ void coverage4(const Attend4Params &p) {
    const long long cta = blockIdx.x + (long long)gridDim.x * (blockIdx.y + (long long)gridDim.y * blockIdx.z);
    const long long row = cta * (blockDim.x >> 5) + (threadIdx.x >> 5);  // the warp's first
    if (row < p.total_rows) cover_rows4<D>(p, row);
}

// The dependency wait.  Every launch is a programmatic dependent one, so that
// its start overlaps the kernel before it; with PKV_FLAG_PDL (p.early) the
// segment table, the block table and old pages are read before the wait
// (second call), otherwise nothing is (first call).
__device__ __forceinline__ void depend4(const Attend4Params &p, bool second) {
    if ((p.early != 0) == second) {
        pdl_wait();
        pdl_trigger();
    }
}

// A piece of work: 8 NT rows of one (segment, kv head) against pages of its range.
struct Piece4 {
    Segment sg;
    int h, row0, rows;           // kv head, first row of the tile, rows of it
    int lo_u, hi_u;              // keys some row sees
    int lo_in, hi_in;            // keys every row sees
    int page0, pages;            // the piece's pages
};

// Shared memory of a CTA.
template <class C>
struct Smem4 {
    unsigned char *pipe;         // the warps' stages; then their partials, [KW][R][LD] and (max, sum)
    uint2 *q;                    // [NT][KS][32] Q fragments
    float *recv;                 // partials pushed by the cluster
    float2 *stat;                // [16][R]
    float *w;                    // [R][16]
    float *scale;                // [R]
    int *lo, *hi;                // [R] key bounds of the rows
    uint64_t *bars;              // [KW][NST]
    int *flag, *all_flags;       // own flags (1 bad page, 2 timeout), the cluster's [16]
    __device__ explicit Smem4(unsigned char *raw) {
        pipe = raw + (-smem_u32(raw) & 127u);  // pointer arithmetic keeps the shared address space (a cast would lose it)
        q = reinterpret_cast<uint2 *>(pipe + C::kBody);
        recv = reinterpret_cast<float *>(pipe + C::kBody + C::kQBytes);
        stat = reinterpret_cast<float2 *>(reinterpret_cast<unsigned char *>(recv) + C::kRecv);
        w = reinterpret_cast<float *>(stat + 16 * C::R);
        scale = w + C::R * 16;
        lo = reinterpret_cast<int *>(scale + C::R);
        hi = lo + C::R;
        bars = reinterpret_cast<uint64_t *>(hi + C::R);
        flag = reinterpret_cast<int *>(bars + C::KW * C::NST);
        all_flags = flag + 1;
    }
};

// The tile's key range: bounds grow with the row, so it is [lo of the first
// row, hi of the last), and every row sees all of [lo of the last, hi of the first).
__device__ __forceinline__ void piece_bounds(const Attend4Params &p, Piece4 &w) {
    const int start = w.sg.kend - w.sg.ql, first = first_valid_of(p.first_valid, w.sg.col);
    row_key_bounds(start + w.row0 / p.G, w.sg.kend, p.causal, p.window, first, w.lo_u, w.hi_in);
    row_key_bounds(start + (w.row0 + w.rows - 1) / p.G, w.sg.kend, p.causal, p.window, first, w.lo_in, w.hi_u);
    w.page0 = w.lo_u / kPage;
    w.pages = (w.hi_u + kPage - 1) / kPage - w.page0;
}
__device__ __forceinline__ unsigned fault4(const Attend4Params &p, const Segment &sg) {
    const unsigned f = segment_fault(sg, p.total_rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
    return f ? f : sg.ql > p.max_q_len ? PKV_ERR_QLEN : 0u;
}
// A refused segment: its error, and zero rows of kv heads [h0, h1).
template <int D>
__device__ __forceinline__ void refuse4(const Attend4Params &p, const Segment &sg, unsigned fault, int h0, int h1) {
    if (threadIdx.x == 0) atomicOr(p.err, fault);
    if (sg.q0 >= 0)  // a negative q_start covers nothing
        for (long long r = sg.q0; r < min((long long)sg.q0 + sg.ql, (long long)p.total_rows); ++r)
            zero_row4(p, r, h0 * p.G, (h1 - h0) * p.G, D, threadIdx.x, blockDim.x);
}

// Attend one piece: every warp takes every KW-th of its pages and leaves its
// partial rows and (max, sum) in shared memory.  ring: stages this warp has
// used so far.  dep: the dependency wait happens in here, after the first
// copies, and with it the rows no segment covers.  Returns the CTA's flags.
template <class C>
__device__ __forceinline__ int attend_piece(const Attend4Params &p, const Smem4<C> &sm, const Piece4 &w, int &ring, bool dep) {
    constexpr int D = C::D, NT = C::NT, KW = C::KW, NST = C::NST, KS = C::KS, R = C::R, LD = C::LD, PP = C::PP;
    const int tid = threadIdx.x, kw = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const Segment &sg = w.sg;
    const int h = w.h, row0 = w.row0, rows_here = w.rows, kend = sg.kend, new_start = kend - sg.ql;
    const int lo_u = w.lo_u, hi_u = w.hi_u, lo_in = w.lo_in, hi_in = w.hi_in, cb0 = w.page0, nb = w.pages;
    const int n_mine = nb > kw ? (nb - kw + KW - 1) / KW : 0;
    uint2 *sQ = sm.q;
    float *sScale = sm.scale;
    int *sLo = sm.lo, *sHi = sm.hi, *sFlag = sm.flag;
    unsigned char *pipe = sm.pipe;
    uint64_t *wbars = sm.bars + kw * NST;
    unsigned char *wstage = pipe + (size_t)kw * NST * C::kStage;
    const int *bt_row = p.block_table + (long long)sg.col * p.mbps;
    // ids of the warp's first 32 pages (lane l: page l), on their way while the bounds are formed
    const int id_first = kw + lane * KW < nb ? bt_row[table_page(cb0 + kw + lane * KW, p.ring_rows)] : -1;
    if (tid == 0) sFlag[0] = 0;
    if (tid < R) {
        int lo = 0, hi = 0;  // padding rows see no key
        if (tid < rows_here)
            row_key_bounds(new_start + (row0 + tid) / p.G, kend, p.causal, p.window, first_valid_of(p.first_valid, sg.col), lo, hi);
        sLo[tid] = lo;
        sHi[tid] = hi;
    }
    __syncthreads();

    // ---- page ids and copies.  The warp's j-th stage is its pages j PP .. (j + 1) PP - 1;
    // lane l holds the id of its page window + l.
    const int stages = (n_mine + PP - 1) / PP, base = ring;
    int id_reg = id_first, id_window = 0;
    bool bad = false, timed_out = false;
    const unsigned char *copy_base = ((lane & 1) ? p.v : p.k) + (size_t)h * C::kBlock;
    const size_t block_stride = (size_t)p.Hkv * C::kBlock;
    auto slot = [&](int j) { return (base + j) % NST; };
    auto issue = [&](int j) {
        const int j0 = j * PP;
        if ((j0 & ~31) != id_window) {
            id_window = j0 & ~31;
            const int li = kw + (id_window + lane) * KW;
            id_reg = li < nb ? bt_row[table_page(cb0 + li, p.ring_rows)] : -1;
        }
        // lane 2 e copies the stage's e-th K block, lane 2 e + 1 its V block
        const int bid = __shfl_sync(0xffffffffu, id_reg, (j0 + (lane >> 1)) & 31);
        if (lane < 2 * PP) {
            const bool some = j0 + (lane >> 1) < n_mine, ok = (unsigned)bid < (unsigned)p.num_blocks;
            bad |= some && !ok;
            uint64_t *bar = wbars + slot(j);
            if (some && ok) {
                mbar_expect_tx(bar, C::kBlock);
                bulk_load(wstage + (size_t)slot(j) * C::kStage + lane * C::kBlock, copy_base + (unsigned)bid * block_stride, C::kBlock, bar);
            } else {
                mbar_arrive(bar);  // nothing to fetch; after a bad page the result is discarded
            }
        }
    };
    auto wait_stage = [&](int j) {
        const unsigned parity = ((base + j) / NST) & 1;
        if (mbar_try_wait(wbars + slot(j), parity)) return;
        bool done = timed_out;
#pragma unroll 1
        for (int it = 0; it < kWaitProbes4 && !done; ++it) done = mbar_try_wait(wbars + slot(j), parity);
        timed_out |= !done;
    };
    int issued = 0;
    if (dep) {
        // Pages wholly below this step's rows are in the cache already, whatever
        // the kernel before this one still writes.
#pragma unroll 1
        for (; issued < NST && issued < stages && cb0 + kw + (issued * PP + PP - 1) * KW < new_start / kPage; ++issued) issue(issued);
        depend4(p, true);
    }
#pragma unroll 1
    for (; issued < NST && issued < stages; ++issued) issue(issued);
    if (dep) coverage4<D>(p);  // while the copies are on their way

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
        m_r[nt][0] = m_r[nt][1] = kNoMax;
        l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < stages; ++j) {
        const unsigned char *stage = wstage + (size_t)slot(j) * C::kStage;
        const int pos_first = (cb0 + kw + j * PP * KW) * kPage;  // position of the stage's first page; the next ones follow KW pages on
        const int pages = min(PP, n_mine - j * PP);
        wait_stage(j);
        // S^T: lane (g, t) holds tokens g and g + 8, columns t D/4 ..  (A stage's
        // missing last page holds whatever was there: its scores and scales are masked.)
        float sa[PP][NT][4];
#pragma unroll
        for (int e = 0; e < PP; ++e) {
            const unsigned char *st = stage + e * C::kPageBytes;
            // One accumulation chain a page and tile; a lone one is split in two.
            constexpr bool kTwo = PP * NT == 1;
            float sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sa[e][nt][i] = 0.f;
            constexpr int W = D / 32;  // code words of a token and lane
            unsigned ka[W], kb[W];
            lds_words<W>(ka, st + gq * (D / 2) + tq * (D / 8));
            lds_words<W>(kb, st + (gq + 8) * (D / 2) + tq * (D / 8));
            const unsigned char *ss = st + 8 * D + gq * (D / 16) + tq * (D / 64);  // scale bytes of the two tokens
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const unsigned fa = scale4_both(ss[w / 2]), fb = scale4_both(ss[w / 2 + D / 2]);
                unsigned a[4], b[4];
                unpack_e2m1x8(a, ka[w]);
                unpack_e2m1x8(b, kb[w]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = hmul2(a[i], fa);
                    b[i] = hmul2(b[i], fb);
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
                    mma_f16_16816(sa[e][nt], a[0], b[0], a[1], b[1], q0.x, q0.y);
                    if constexpr (kTwo) mma_f16_16816(sb, a[2], b[2], a[3], b[3], q1.x, q1.y);
                    else mma_f16_16816(sa[e][nt], a[2], b[2], a[3], b[3], q1.x, q1.y);
                }
            }
            if constexpr (kTwo)
#pragma unroll
                for (int i = 0; i < 4; ++i) sa[e][0][i] += sb[i];
        }
        // Online softmax (base 2) with a lazy maximum: this lane has tokens g,
        // g + 8 of rows 2t, 2t + 1.  x = score - reference; the reference moves
        // only when some x passes kLazy4.
        const bool inside = pages == PP && pos_first >= lo_in && pos_first + (PP - 1) * KW * kPage + kPage <= hi_in;
        unsigned pb[PP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[PP][4], top = -CUDART_INF_F;
#pragma unroll
            for (int e = 0; e < PP; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[e][i] = fmaf(sa[e][nt][i], sc[nt][i & 1], -m_r[nt][i & 1]);
            if (!inside) {
#pragma unroll
                for (int e = 0; e < PP; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = pos_first + e * KW * kPage + gq + (i >> 1) * 8, r = nt * 8 + 2 * tq + (i & 1);
                        if (e >= pages || key < sLo[r] || key >= sHi[r]) x[e][i] = -CUDART_INF_F;
                    }
            }
#pragma unroll
            for (int e = 0; e < PP; ++e) top = fmaxf(top, fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3])));
            if (__any_sync(0xffffffffu, top > kLazy4)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = m_r[nt][i];
#pragma unroll
                    for (int e = 0; e < PP; ++e)
#pragma unroll
                        for (int o = 0; o < 4; o += 2)
                            if (x[e][i + o] != -CUDART_INF_F) mx = fmaxf(mx, fmaf(sa[e][nt][i + o], sc[nt][i], -kLift4));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float al = ex2(m_r[nt][i] - mx);
                    m_r[nt][i] = mx;
                    l_r[nt][i] *= al;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        acc[nt][k][i] *= al;
                        acc[nt][k][i + 2] *= al;
                    }
#pragma unroll
                    for (int e = 0; e < PP; ++e)
#pragma unroll
                        for (int o = 0; o < 4; o += 2)
                            if (x[e][i + o] != -CUDART_INF_F) x[e][i + o] = fmaf(sa[e][nt][i + o], sc[nt][i], -mx);
                }
            }
#pragma unroll
            for (int e = 0; e < PP; ++e) {
                const float p00 = ex2(x[e][0]), p01 = ex2(x[e][1]), p10 = ex2(x[e][2]), p11 = ex2(x[e][3]);
                l_r[nt][0] += p00 + p10;
                l_r[nt][1] += p01 + p11;
                pb[e][nt][0] = transpose8x8(pack_f16x2(p00, p01));
                pb[e][nt][1] = transpose8x8(pack_f16x2(p10, p11));
            }
        }
        // O^T += V^T P^T: lane (g, t) holds columns g D/8 .., tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int e = 0; e < PP; ++e) {
            const int pos0 = pos_first + e * KW * kPage;
            const unsigned char *sv = stage + e * C::kPageBytes + C::kBlock;
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
                        for (int i = 0; i < 4; ++i) {
                            const int key = pos0 + 2 * tq + (i >> 1) * 8 + (i & 1);
                            const unsigned m = 0xffu << (8 * i);
                            if (e < pages && key >= lo_u && key < hi_u) {
                                if ((w & m) >= (0xf8u << (8 * i))) nan |= m;
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
                                    for (int i = 0; i < 2; ++i) {
                                        const int r = nt * 8 + 2 * tq + i;
                                        if (pos0 + o >= sLo[r] && pos0 + o < sHi[r])
#pragma unroll
                                            for (int k = pl * 4; k < (pl + 2 < D / 64 ? pl + 2 : D / 64) * 4; ++k)
                                                acc[nt][k][i] = acc[nt][k][i + 2] = CUDART_NAN_F;
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
                    for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt][pl * 4 + k], a0, a1, a2, a3, pb[e][nt][0], pb[e][nt][1]);
                }
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (j + NST < stages) issue(j + NST);
    }
    timed_out = __any_sync(0xffffffffu, timed_out);
    bad = __any_sync(0xffffffffu, bad);
    if (timed_out && lane == 0) {
        // copies still in flight get a bounded chance to land before the stages are reused
#pragma unroll 1
        for (int j = max(0, stages - NST); j < stages; ++j)
#pragma unroll 1
            for (int it = 0; it < kWaitProbes4 && !mbar_try_wait(wbars + slot(j), ((base + j) / NST) & 1); ++it) {
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
            if (m_r[nt][e] == kNoMax) m_r[nt][e] = l_r[nt][e] != l_r[nt][e] ? 0.f : -CUDART_INF_F;
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
    ring = base + stages;
    __syncthreads();
    return sFlag[0];
}

// The warps' partials of row r, columns 4 c4 .. + 3, merged: unnormalised sum, max and sum of weights.
template <class C>
__device__ __forceinline__ float4 merge_warps(const Smem4<C> &sm, int r, int c4, float &M, float &L) {
    constexpr int KW = C::KW, R = C::R, LD = C::LD;
    const float *base = reinterpret_cast<const float *>(sm.pipe);
    float mk[KW];
    M = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
        mk[k] = base[k * C::kPartFloats + R * LD + r];
        M = fmaxf(M, mk[k]);
    }
    L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KW; ++k) {
        // a warp that saw no key of the row has weight 0 and a zero accumulator
        const float w = mk[k] == -CUDART_INF_F ? 0.f : ex2(mk[k] - M);
        const float4 v = *reinterpret_cast<const float4 *>(base + k * C::kPartFloats + r * LD + 4 * c4);
        L = fmaf(w, base[k * C::kPartFloats + R * LD + R + r], L);
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    return o;
}
__device__ __forceinline__ long long out_row4(const Attend4Params &p, const Piece4 &w, int r) {
    const int i = (w.row0 + r) / p.G, jh = (w.row0 + r) % p.G;
    return ((long long)w.sg.q0 + i) * p.Hq + (long long)w.h * p.G + jh;
}
// One CTA held the whole range: its rows are final.
template <class C>
__device__ __forceinline__ void write_rows4(const Attend4Params &p, const Smem4<C> &sm, const Piece4 &w, int flags) {
    constexpr int D = C::D;
#pragma unroll 1
    for (int e = threadIdx.x; e < w.rows * (D / 4); e += C::kThreads) {
        const int r = e / (D / 4), c4 = e % (D / 4);
        float M, L;
        const float4 o = merge_warps<C>(sm, r, c4, M, L);
        const bool zero = flags || L == 0.f;  // a NaN sum stays: the row holds a NaN
        const float inv = 1.f / L;
        const long long row = out_row4(p, w, r);
        store_out4(p, row * D + 4 * c4, zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (c4 == 0 && p.lse) p.lse[row] = zero ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
    }
}
__device__ __forceinline__ void report4(const Attend4Params &p, int flags) {
    if (threadIdx.x == 0 && flags) atomicOr(p.err, ((flags & 1) ? PKV_ERR_BLOCK : 0u) | ((flags & 2) ? PKV_ERR_TIMEOUT : 0u));
}
template <class C>
__device__ __forceinline__ void init_bars4(const Smem4<C> &sm) {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll 1
        for (int i = 0; i < C::NST; ++i) mbar_init(sm.bars + (threadIdx.x >> 5) * C::NST + i, 2 * C::PP);  // one arrival a copy
        fence_barrier_init();
    }
}

// ---------------------------------------------------------------- one cluster per range

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) attend4_kernel(const __grid_constant__ Attend4Params p) {
    namespace cg = cooperative_groups;
    constexpr int D = C::D, R = C::R, NTHR = C::kThreads;
    extern __shared__ unsigned char smem_raw[];
    const Smem4<C> sm(smem_raw);
    const int tid = threadIdx.x, rank = blockIdx.x, ncta = gridDim.x;
    const int tile = blockIdx.y % p.row_tiles, s = blockIdx.z;
    depend4(p, false);
    auto leave = [&] {
        depend4(p, true);
        coverage4<D>(p);
    };
    if (p.S == 0) return leave();
    Piece4 w;
    w.h = blockIdx.y / p.row_tiles;
    w.sg = load_segment(p.seq_info, s);
    const unsigned fault = fault4(p, w.sg);
    w.row0 = tile * R;
    w.rows = fault ? 0 : min(R, w.sg.ql * p.G - w.row0);
    if (w.rows <= 0) {  // uniform across the cluster
        depend4(p, true);
        if (fault && rank == 0 && tile == 0) refuse4<D>(p, w.sg, fault, w.h, w.h + 1);
        coverage4<D>(p);
        return;
    }
    piece_bounds(p, w);
    // Short ranges take fewer CTAs than the cluster has: each gets a number of
    // pages that is worth its share of the merge.
    const int nblk = w.pages, ncl = min(ncta, max(1, (nblk + p.min_pages / 2) / p.min_pages));
    if (rank >= ncl) return leave();
    const int bps = (nblk + ncl - 1) / ncl;
    w.page0 += rank * bps;
    w.pages = max(0, min(bps, nblk - rank * bps));
    if (ncl > 1)  // announce this CTA to the cluster; waited on before any remote store
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    init_bars4<C>(sm);
    int ring = 0;
    const int flags = attend_piece<C>(p, sm, w, ring, true);
    report4(p, flags);
    if (ncl == 1) {
        write_rows4<C>(p, sm, w, flags);
        return;
    }
    // ---- merge across the cluster: every CTA pushes its merged partial of each
    // output slice to the CTA that finishes it
    cg::cluster_group cluster = cg::this_cluster();
    const int items = w.rows * (D / 4), per4 = (items + ncl - 1) / ncl;
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");  // every CTA of the cluster runs
    if (tid < ncl) *cluster.map_shared_rank(sm.all_flags + rank, tid) = flags;
#pragma unroll 1
    for (int e = tid; e < items; e += NTHR) {
        const int r = e / (D / 4), c4 = e % (D / 4), owner = e / per4;
        float M, L;
        const float4 o = merge_warps<C>(sm, r, c4, M, L);
        *cluster.map_shared_rank(reinterpret_cast<float4 *>(sm.recv) + rank * per4 + (e - owner * per4), owner) = o;
        if (c4 < ncl) *cluster.map_shared_rank(sm.stat + rank * R + r, c4) = make_float2(M, L);
    }
    cluster.sync();  // publishes every CTA's partials
    int poison = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) poison |= c < ncl ? sm.all_flags[c] : 0;
#pragma unroll 1
    for (int b = 0; b < R * 16; b += NTHR) {  // row, source CTA: normalised weights by 16-lane shuffles
        const int r = (b + tid) >> 4, c = tid & 15;
        const float2 stt = c < ncl && r < w.rows ? sm.stat[c * R + r] : make_float2(-CUDART_INF_F, 0.f);
        float M = stt.x;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float wt = stt.x == -CUDART_INF_F ? 0.f : ex2(stt.x - M);
        float W = wt * stt.y;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
        const bool zero = poison || W == 0.f;
        if (b + tid < R * 16) sm.w[r * 16 + c] = zero ? 0.f : wt / W;
        if (c == 0 && r < w.rows && rank == 0 && p.lse) p.lse[out_row4(p, w, r)] = zero ? -CUDART_INF_F : (M + log2f(W)) * 0.6931471805599453f;
    }
    __syncthreads();
#pragma unroll 1
    for (int e = tid; e < per4 && rank * per4 + e < items; e += NTHR) {
        const int r = (rank * per4 + e) / (D / 4), c4 = (rank * per4 + e) % (D / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < ncl; ++c) {
            const float wt = sm.w[r * 16 + c];
            const float4 v = reinterpret_cast<const float4 *>(sm.recv)[c * per4 + e];
            if (wt != 0.f) {  // a zero weight must not touch its partial: a poisoned one may hold NaN
                o.x = fmaf(wt, v.x, o.x);
                o.y = fmaf(wt, v.y, o.y);
                o.z = fmaf(wt, v.z, o.z);
                o.w = fmaf(wt, v.w, o.w);
            }
        }
        store_out4(p, out_row4(p, w, r) * D + 4 * c4, o);
    }
}

// ---------------------------------------------------------------- equal shares of all ranges

// With a workspace the ranges (one (kv head, row tile) each) are laid end to end, each
// as long as its pages and a few more for what a piece costs besides them (its
// first loads and its merge, about 4 us: short ranges would else make the
// CTAs that hold many of them late, 77 us against 58 on 32 sequences of up to
// 16384 keys).  The one wave of CTAs the device holds takes equal shares of
// the total T: CTA i [i T / N, (i + 1) T / N).  A range that one CTA holds whole is
// written at once; of a range that several share, each leaves its rows and
// (max, sum) in the workspace, slot 2 i + 1 where the range begins in CTA i and
// slot 2 i where it continues, and a second launch merges them.  Clusters
// need their CTAs free at the same time in one GPC, and a fixed number of
// them splits long and short ranges alike; shares have neither limit.

// A CTA's share, and a walk over its pieces.
// FAST: two paths for each division (a CTA of 640 threads, five roles of which
// walk their pieces, is faster with less code: 72 us against 75).
template <bool FAST>
struct Share4 {
    // a / b for a >= 0, b > 0; short where both fit 32 bits, as they mostly do.
    __device__ __forceinline__ static long long div4(long long a, long long b) {
        return !FAST || ((unsigned long long)(a | b) >> 32) ? a / b : (long long)((unsigned)a / (unsigned)b);
    }
    long long T;       // length of all ranges
    int N;             // CTAs that share them
    long long at, b;   // what is left of this CTA's share
    int s;             // the segment that holds `at`, and where it begins
    long long begin;

    // All rows of segment s.
    __device__ __forceinline__ static void segment(const Attend4Params &p, int s, Piece4 &w) {
        w.sg = load_segment(p.seq_info, s);
        w.row0 = 0;
        w.rows = fault4(p, w.sg) ? 0 : w.sg.ql * p.G;
        w.pages = 0;
        if (w.rows > 0) piece_bounds(p, w);
    }
    // Its (kv head, row tile) ranges, each as long as all its rows' range.
    __device__ __forceinline__ static long long length(const Attend4Params &p, const Piece4 &w, int R) {
        return w.pages ? (long long)(w.pages + p.piece_pages) * p.Hkv * ((w.rows + R - 1) / R) : 0ll;
    }
    // Every thread of the CTA calls it; NTHR threads, scratch of NTHR / 32 + 2 words of 8 bytes.
    template <int NTHR>
    __device__ __forceinline__ void find(const Attend4Params &p, int R, long long *scratch) {
        // prefix sum of the segments' lengths; thread t holds segments t per ..
        const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
        const int per = (p.S + NTHR - 1) / NTHR, s_lo = min(tid * per, p.S), s_hi = min(s_lo + per, p.S);
        long long mine = 0;
#pragma unroll 4
        for (int i = s_lo; i < s_hi; ++i) {
            Piece4 w;
            segment(p, i, w);
            mine += length(p, w, R);
        }
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) scratch[tid >> 5] = upto;
        __syncthreads();
        T = 0;
#pragma unroll
        for (int k = 0; k < NTHR / 32; ++k) {
            if (k < tid >> 5) upto += scratch[k];
            T += scratch[k];
        }
        N = (int)max(1ll, min((long long)gridDim.x, div4(T, p.min_pages)));
        at = div4(cta * T, N);
        b = cta < N ? div4((cta + 1) * T, N) : at;
        if (at < b && upto - mine <= at && at < upto) {
            long long x = upto - mine;
            int i = s_lo;
#pragma unroll 1
            for (; i + 1 < s_hi; ++i) {  // (the last one, where none before it does)
                Piece4 w;
                segment(p, i, w);
                const long long n = length(p, w, R);
                if (at < x + n) break;
                x += n;
            }
            scratch[NTHR / 32] = i;
            scratch[NTHR / 32 + 1] = x;
        }
        __syncthreads();
        s = (int)scratch[NTHR / 32];
        begin = scratch[NTHR / 32 + 1];
        __syncthreads();  // the scratch is free again
    }
    // The next piece: its rows, bounds and pages; from: pages of its range
    // before it, whole: it is all of the range.  last: the CTA that holds the
    // range's last page.  False when the share is done.
    __device__ __forceinline__ bool next(const Attend4Params &p, int R, Piece4 &w, int &tile, int &from, bool &whole, int &last) {
#pragma unroll 1
        while (at < b) {
            segment(p, s, w);
            const int nblk = w.pages, len = nblk + p.piece_pages;
            const long long n_seg = length(p, w, R);
            if (at >= begin + n_seg) {  // past this segment (or it has no pages)
                begin += n_seg;
                ++s;
                continue;
            }
            const int range = (int)div4(at - begin, len), tiles = (w.rows + R - 1) / R;
            tile = range % tiles;
            const long long first = begin + (long long)range * len, end = min(b, first + len);
            // the pages come after the piece's cost
            from = max(0, (int)(at - first) - p.piece_pages);
            const int n = max(0, (int)(end - first) - p.piece_pages) - from;
            at = end;
            if (n == 0) continue;
            const int page = w.page0 + from;
            w.h = range / tiles;
            w.row0 = tile * R;
            w.rows = min(R, w.rows - w.row0);
            if (tiles > 1) piece_bounds(p, w);  // the tile's own bounds: keys outside them are masked
            w.page0 = page;
            w.pages = n;
            whole = n == nblk;
            last = (int)div4((first + len) * N - 1, T);
            return true;
        }
        return false;
    }
};
// What a piece of a shared range leaves for the merge.
__device__ __forceinline__ int4 head4(const Piece4 &w, int tile, int last, int flags) {
    return make_int4(w.sg.q0, w.h | tile << 16, last, 1 | flags << 1 | w.rows << 4);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) balance4_kernel(const __grid_constant__ Attend4Params p) {
    constexpr int D = C::D, R = C::R, NTHR = C::kThreads;
    extern __shared__ unsigned char smem_raw[];
    const Smem4<C> sm(smem_raw);
    const int tid = threadIdx.x, cta = blockIdx.x;
    init_bars4<C>(sm);
    depend4(p, false);
    Share4<true> share;
    share.find<NTHR>(p, R, reinterpret_cast<long long *>(sm.recv));
    int ring = 0, left = 0;  // left: bit i, a piece in slot 2 cta + i
    bool waited = false;
    Piece4 w;
    int tile, from, last;
    bool whole;
#pragma unroll 1
    while (share.next(p, R, w, tile, from, whole, last)) {
        const int flags = attend_piece<C>(p, sm, w, ring, !waited);
        waited = true;
        report4(p, flags);
        if (whole) {
            write_rows4<C>(p, sm, w, flags);
        } else {
            const int slot = 2 * cta + (from == 0);
            left |= 1 << (from == 0);
            float *part = p.ws_part + (size_t)slot * R * D;
#pragma unroll 1
            for (int e = tid; e < w.rows * (D / 4); e += NTHR) {
                const int r = e / (D / 4), c4 = e % (D / 4);
                float M, L;
                reinterpret_cast<float4 *>(part)[e] = merge_warps<C>(sm, r, c4, M, L);
                if (c4 == 0) p.ws_stat[slot * R + r] = make_float2(M, L);
            }
            if (tid == 0) p.ws_head[slot] = head4(w, tile, last, flags);
        }
        __syncthreads();          // the partials are read
        fence_proxy_async();      // and the next copies may write over them
    }
    if (!waited) {
        depend4(p, true);
        coverage4<D>(p);
    }
    // (only after the dependency wait: the kernel before may be the last call's merge)
    if (tid < 2 && !(left >> tid & 1)) p.ws_head[2 * cta + tid].w = 0;
    // the refused segments, in turn
#pragma unroll 1
    for (int i = cta; i < p.S; i += gridDim.x) {
        const Segment sg = load_segment(p.seq_info, i);
        const unsigned fault = fault4(p, sg);
        if (fault) refuse4<D>(p, sg, fault, 0, p.Hkv);
    }
}

// Merge of the shared ranges: CTA (i, y) finishes rows y .. of the range that
// begins in slot 2 i + 1, from that slot and slots 2 (i + 1), .., 2 last.  TPR
// threads a row: a whole CTA where few rows have many slots, a warp where
// many rows have few.
template <int D, int R, int TPR>
__global__ void __launch_bounds__(kMerge4Threads) merge4_kernel(const __grid_constant__ Attend4Params p) {
    constexpr int Q = D / 4, GR = TPR > Q ? TPR / Q : 1, QL = TPR > Q ? 1 : Q / TPR;  // column quads; groups that share the slots; quads a thread
    constexpr int ROWS = kMerge4Threads / TPR;
    __shared__ float sWt[TPR == 32 ? 1 : kMerge4Slots];
    __shared__ float sRed[kMerge4Threads / 32][2];
    __shared__ float4 sAcc[TPR == 32 ? 1 : kMerge4Threads];
    const int tid = threadIdx.x, t = tid % TPR, cta = blockIdx.x, r = blockIdx.y * ROWS + tid / TPR;
    pdl_wait();
    pdl_trigger();
    const int4 hd = p.ws_head[2 * cta + 1];
    if (!(hd.w & 1)) return;
    Piece4 w;
    w.sg.q0 = hd.x;
    w.h = hd.y & 0xffff;
    w.row0 = (hd.y >> 16) * R;
    if (r >= hd.w >> 4) return;    // whole CTAs (TPR = CTA) or warps leave
    const int n = hd.z - cta + 1;  // slots, at most kMerge4Slots
    auto slot_of = [&](int k) { return k == 0 ? 2 * cta + 1 : 2 * (cta + k); };
    // max over the slots, then weights and their sum
    float M = -CUDART_INF_F;
    int poison = 0;
    for (int k = t; k < n; k += TPR) {
        M = fmaxf(M, p.ws_stat[(size_t)slot_of(k) * R + r].x);
        poison |= p.ws_head[slot_of(k)].w >> 1 & 3;
    }
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if constexpr (TPR == 32) {
        poison = __any_sync(0xffffffffu, poison);
    } else {
        if ((tid & 31) == 0) sRed[tid >> 5][0] = M;
        poison = __syncthreads_or(poison);
#pragma unroll
        for (int k = 0; k < kMerge4Threads / 32; ++k) M = fmaxf(M, sRed[k][0]);
    }
    float L = 0.f;
    for (int k = t; k < n; k += TPR) {
        const float2 st = p.ws_stat[(size_t)slot_of(k) * R + r];
        const float wt = st.x == -CUDART_INF_F ? 0.f : ex2(st.x - M);
        if constexpr (TPR != 32) sWt[k] = wt;
        L = fmaf(wt, st.y, L);
    }
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (TPR != 32) {
        if ((tid & 31) == 0) sRed[tid >> 5][1] = L;
        __syncthreads();
        L = 0.f;
#pragma unroll
        for (int k = 0; k < kMerge4Threads / 32; ++k) L += sRed[k][1];
    }
    const bool zero = poison || L == 0.f;
    const float inv = 1.f / L;
    const long long row = out_row4(p, w, r);
    const int c4 = t % Q, g = TPR > Q ? t / Q : 0;
    auto add = [](float4 &o, float wt, float4 v) {
        if (wt != 0.f) {  // a zero weight must not touch its partial: a poisoned one may hold NaN
            o.x = fmaf(wt, v.x, o.x);
            o.y = fmaf(wt, v.y, o.y);
            o.z = fmaf(wt, v.z, o.z);
            o.w = fmaf(wt, v.w, o.w);
        }
    };
    auto part = [&](int k, int q) { return reinterpret_cast<const float4 *>(p.ws_part)[((size_t)slot_of(k) * R + r) * Q + q]; };
    auto put = [&](int q, float4 o) {
        store_out4(p, row * D + 4 * q, zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    };
    float4 o[QL];
#pragma unroll
    for (int q = 0; q < QL; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (TPR == 32) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float x = p.ws_stat[(size_t)slot_of(k) * R + r].x, wt = x == -CUDART_INF_F ? 0.f : ex2(x - M);
#pragma unroll
            for (int q = 0; q < QL; ++q)
                if (t + q * TPR < Q) add(o[q], wt, part(k, t + q * TPR));
        }
#pragma unroll
        for (int q = 0; q < QL; ++q)
            if (t + q * TPR < Q) put(t + q * TPR, o[q]);
    } else {
#pragma unroll 4
        for (int k = g; k < n; k += GR) add(o[0], sWt[k], part(k, c4));
        sAcc[tid] = o[0];
        __syncthreads();
        if (g == 0) {
#pragma unroll
            for (int k = 1; k < GR; ++k) add(o[0], 1.f, sAcc[k * Q + c4]);
            put(c4, o[0]);
        }
    }
    if (t == 0 && p.lse) p.lse[row] = zero ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace pkv
