// Attention of packed prompts over their own rows on the tensor cores (sm_103a).
//
//   out[i] = sum_j softmax_j(scale q_i . k_j) v_j,   j in the row's window of its own segment
//
// q, k and v are rows of one projection (or of three), not pages: a prompt's rows
// are at hand when they are appended, and reading them needs no table.  A CTA takes
// one kv head of a segment and 128 (head_dim above 128) or 2 x 128 query rows, a
// token's G heads of the group side by side (row = token * G + head), so short
// prompts fill tiles and the causal edge of a tile is 128 / G tokens wide.  It walks over
// the keys that some row sees in blocks of 128.
//
// The grid has a CTA for every such item that the rows can make (the longest of 32 segments first), but a CTA that runs
// takes the items of CTAs that have not started (cluster launch control) instead of ending: one
// CTA an SM stays, dynamic balance without a counter in memory, and the next
// item's copies and products start while the rows of this one are written.  Which item a number is, one
// warp finds in the table as it goes along it.  (A CTA for each item that a segment could have at most: 128 prompts
// of 30 rows where 2048 were allowed 205 us, now 44; one of 4096 beside 63 of 30 rows 308, now 121.)
//
// Roles, meeting on mbarriers only, each walking through the items by itself:
//   softmax warps (four a tile; thread = row)  read S from TMEM, mask, take the
//       maximum, write P = 2^(S - reference) as bf16 to TMEM,
//       and at the end the normalised rows out.  The reference moves only when a score
//       passes it by 2^8 (then O is rescaled in TMEM; no product is in flight on it then);
//   MMA warps   S = Q K^T (M 128, N 128; Q and K in shared memory) and O += P V (P
//       from TMEM, V as an MN-major tile), a warp each; the second one then looks after rows of no
//       segment or of two, and refused segments;
//   copy warp   Q, then K and V blocks through a ring of stages
//       (TMA, 128-byte swizzle; rows past the tensor and columns past head_dim come as zeros);
//   dealer warp   asks for the next item, finds it in the table and works out its blocks for all.
// Where items are short a role's code is cold each time, some ten cycles an instruction: the kernel has to
// stay small (88 KB), what an item needs is worked out once, and the steps are spread over warps that
// wait anyway.  (Every role working items out for itself, 120 KB: 16 prompts of up to 301 rows 33 us, now 27;
// sliding windows at head_dim 256 248, then 209.)
// TMEM (512 columns): one S of 128, two P of 64, then O (256: two tiles up to head_dim 128,
// one above).  S is in registers some 200 cycles after it is there, and the next one is computed in its
// place: with two tiles that of the other tile, so that one tile's softmax runs beside the other's
// products; with one the next block's.  (S and P in one place for each tile, 2 x 128 columns, let the tiles fall into
// step, softmax and products in turn: 462 us for one prompt of 8192 rows, now 372.)
//
// P is rounded to bf16, as V is: half a step, 2^-8 of a weight, on sums
// whose result is rounded the same way or averaged over many keys; the sum of weights is
// taken from the unrounded ones in fp32, so a row that one key dominates is off by that key's half step.  (Sums of the
// rounded ones, by additions of bf16 to fp32: 386 us for one prompt of 8192 rows, not 370.)
//
// Keys that a row does not see have weight zero, and zero times a NaN or an
// infinity of such a key's V is NaN.  That shows in the row: items in which a row is
// not finite are kept in a list and run once more, carefully: V blocks that not every row sees have their
// non-finite values zeroed in shared memory, and the rows that do see
// such a key get its products at the end.  All waits are bounded; a
// timeout ends every role, rows not written yet read zero and PKV_ERR_TIMEOUT is set (but for an item that waits for the list
// to be run just then: it is not written).
#pragma once

#include <limits.h>
#include <math_constants.h>

#include "prompt_launch.h"
#include "verify.cuh"

namespace pkv {

template <int DP_>
struct PromptCfg {
    static constexpr int DP = DP_;                                  // head_dim, padded
    static constexpr int NT = DP <= 128 ? 2 : 1;                    // query tiles of a CTA
    static constexpr int kKeys = 128;                               // of a block
    static constexpr int kCols = DP < 128 ? DP : 128;               // columns of a stage
    static constexpr int SPB = DP / kCols;                          // stages of a block
    static constexpr unsigned kPart = 128 * 128;                    // 128 rows x 64 columns
    static constexpr unsigned kStage = kCols / 64 * kPart;
    static constexpr unsigned kQTile = DP / 64 * kPart;
    static constexpr int NST = DP == 64 ? 8 : 5;
    static constexpr int kSoftmaxWarps = 4 * NT;
    static constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
    // registers a thread: at launch, and of the softmax warps and of the others while the roles run (one tile leaves enough for all)
    static constexpr int kRegs = NT == 2 ? 168 : 0, kRegsSoftmax = NT == 2 ? 200 : 0, kRegsOthers = 104;
    static_assert(kSoftmaxWarps * 32 * kRegsSoftmax + 128 * kRegsOthers <= kThreads * kRegs || NT == 1, "the roles' registers fit the launch's");
    static constexpr int kSched = 1;                                // items dealt out and not taken by all roles (two: 4096 rows beside short ones 138 us, not 128)
    static constexpr int kOdd = 64;                                 // items to run again, at most before they are
    static constexpr int kBars = 2 * NST + 3 + 2 + 4 + 2 + 2 + 2 * kSched + 1;
    static constexpr size_t kSmem = 1024 + (size_t)NT * kQTile + (size_t)NST * kStage + 16 + kSched * 80 + kBars * 8 + kOdd * 8 + 64;
    static constexpr unsigned kColP = 128, kColO = 256;             // S at 0; two slots of P; O of tile t at kColO + t * DP
    static_assert(kSmem <= 232448, "exceeds the per-CTA shared memory limit");
};

constexpr float kNoScore = -3e38f;  // reference of a row that has seen no key
constexpr float kPromptLazy = 8.f;  // a reference moves when a score passes it by this (base 2)

// 32 columns of this thread's TMEM lane; the caller waits (tmem_wait_ld) before it uses them.
__device__ __forceinline__ void tmem_ld32_async(unsigned taddr, unsigned (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
// 3-D tiled TMA load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Why a segment is refused (PKV_ERR_*), or 0.  A prompt is whole: its keys are its own rows.
__device__ __forceinline__ unsigned prompt_fault(const PromptParams &p, const Segment &s) {
    if (s.q0 < 0 || s.ql < 0 || (long long)s.q0 + s.ql > p.total_rows || s.kend != s.ql) return PKV_ERR_SEGMENT;
    return s.ql > p.max_len ? PKV_ERR_QLEN : 0u;
}
__device__ __forceinline__ void prompt_store4(const PromptParams &p, long long at, float4 v) {
    if (p.out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + at) = v;
}
// Heads [h0, h0 + heads) of a row read zero (lanes of a warp, or threads of a CTA).
__device__ __forceinline__ void prompt_zero(const PromptParams &p, long long row, int h0, int heads, int t, int threads) {
    for (int e = t; e < heads * p.D / 4; e += threads) prompt_store4(p, (row * p.Hq + h0) * p.D + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse)
        for (int e = t; e < heads; e += threads) p.lse[row * p.Hq + h0 + e] = -CUDART_INF_F;
}
// Rows of no segment read zero, rows of two set PKV_ERR_OVERLAP: one warp takes the share of CTA number id.
// (Eight rows at a look at the table: row by row it held up everything else, 128 prompts of 30 rows took 42 us.)
__device__ __noinline__ void prompt_coverage(const PromptParams &p, int id, int lane) {
    const int end = (int)((long long)(id + 1) * p.total_rows / gridDim.x);
#pragma unroll 1
    for (int row = (int)((long long)id * p.total_rows / gridDim.x); row < end; row += 8) {
        int n[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 2
        for (int s = lane; s < p.S; s += 32) {
            const int4 v = p.seq_info[s];
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] += v.x >= 0 && v.x <= row + i && (long long)row + i < (long long)v.x + v.y;
        }
        unsigned none = 0, two = 0;  // rows of no segment, and of two
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = __reduce_add_sync(0xffffffffu, n[i]);
            none |= (k == 0) << i;
            two |= (k > 1) << i;
        }
        const unsigned rows = (1u << min(end - row, 8)) - 1u;
        if ((two & rows) && lane == 0) atomicOr(p.err, PKV_ERR_OVERLAP);
#pragma unroll 1
        for (none &= rows; none; none &= none - 1) prompt_zero(p, row + __ffs(none) - 1, 0, p.Hq, lane, 32);
    }
}
__device__ __forceinline__ bool not_finite(unsigned bf16_pair) { return (bf16_pair & 0x7f80u) == 0x7f80u || (bf16_pair & 0x7f800000u) == 0x7f800000u; }

// Products of the non-finite V values of one key that were zeroed, added to columns c0 .. c0 + 31 of a row.  (Rare, and short.)
__device__ __noinline__ void prompt_add_key(const PromptParams &p, long long key_row, long long q_row, int h, int hq, int c0, float m, float *o) {
    const __nv_bfloat16 *v = p.v + key_row * p.v_stride + (long long)h * p.D + c0;
    const int n = min(32, p.D - c0);
    bool some = false;
#pragma unroll 1
    for (int c = 0; c < n; ++c) some |= !isfinite(__bfloat162float(v[c]));
    if (!some) return;
    const __nv_bfloat16 *q = p.q + q_row * p.q_stride + (long long)hq * p.D, *k = p.k + key_row * p.k_stride + (long long)h * p.D;
    float s = 0.f;
#pragma unroll 1
    for (int d = 0; d < p.D; ++d) s = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), s);
    const float w = exp2_fast(fmaf(s, p.scale_log2, -m));
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
        const float x = __bfloat162float(v[c]);
        if (!isfinite(x)) o[c] = fmaf(w, x, o[c]);
    }
}

// One item: 2 (or 1) x 128 query rows of one (segment, kv head), and the blocks of keys they see.  One
// warp works it out, the others read it in shared memory (as each of them did that, the divisions' code alone was 50 KB).
struct PromptItem {
    int q0, ql;              // the segment's rows
    int token0, tokens;      // tokens of the segment; none: nothing to do
    int first[2], last[2];   // blocks of each tile
    int in_lo, in_hi;        // keys that every row sees
    int b0, b1;              // blocks of the item
    int kind, rows_of;       // kNoItem ..; the CTA number whose rows are looked after, or -1
    int s, place;            // segment (-1: none); item of the segment * Hkv + kv head
    int h, fault;            // kv head; why the segment is refused

    __device__ __forceinline__ void to(int4 *at) const {
        at[0] = make_int4(q0, ql, token0, tokens);
        at[1] = make_int4(first[0], last[0], first[1], last[1]);
        at[2] = make_int4(in_lo, in_hi, b0, b1);
        at[3] = make_int4(kind, rows_of, s, place);
        at[4] = make_int4(h, fault, 0, 0);
    }
    __device__ __forceinline__ void from(const int4 *at) {
        const int4 a = at[0], b = at[1], c = at[2], d = at[3], e = at[4];
        q0 = a.x; ql = a.y; token0 = a.z; tokens = a.w;
        first[0] = b.x; last[0] = b.y; first[1] = b.z; last[1] = b.w;
        in_lo = c.x; in_hi = c.y; b0 = c.z; b1 = c.w;
        kind = d.x; rows_of = d.y; s = d.z; place = d.w;
        h = e.x; fault = e.y;
    }
};
enum { kNoItem = 0, kItem = 1, kCarefulItem = 2 };

// Items of a segment for a kv head (a refused one has its rows to clear).
__device__ __forceinline__ int prompt_items(const PromptParams &p, const Segment &o, int tiles) {
    return prompt_fault(p, o) ? 1 : (o.ql + tiles * p.tokens - 1) / (tiles * p.tokens);
}
// Item `index` of segment s, which is sg, for kv head h.
template <int NT>
__device__ __forceinline__ void prompt_item(const PromptParams &p, PromptItem &w, const Segment &sg, int s, int index, int h) {
    w.q0 = sg.q0;
    w.ql = sg.ql;
    w.s = s;
    w.h = h;
    w.place = index * p.Hkv + h;
    w.fault = s >= 0 ? prompt_fault(p, sg) : 0u;
    w.token0 = index * NT * p.tokens;
    w.tokens = w.fault || s < 0 ? 0 : max(0, min(NT * p.tokens, sg.ql - w.token0));
    if (w.tokens == 0) return;
    int lo, hi, x;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int a = w.token0 + t * p.tokens, b = min(a + p.tokens, sg.ql) - 1;  // tokens of the tile
        w.first[t] = w.last[t] = 0;
        if (b >= a) {
            row_key_bounds(a, sg.ql, p.causal, p.window, 0, lo, x);
            row_key_bounds(b, sg.ql, p.causal, p.window, 0, x, hi);
            w.first[t] = lo / 128;
            w.last[t] = (hi + 127) / 128;
        }
    }
    row_key_bounds(w.token0, sg.ql, p.causal, p.window, 0, lo, w.in_hi);
    row_key_bounds(w.token0 + w.tokens - 1, sg.ql, p.causal, p.window, 0, w.in_lo, hi);
    w.b0 = lo / 128;
    w.b1 = (hi + 127) / 128;
}

// Ask for the item of a CTA that has not started: 16 bytes at `at`, completing on `bar`.
__device__ __forceinline__ void ask_next(uint4 *at, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(smem_u32(at)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The answer: the CTA's number, or -1 where none was left.
__device__ __forceinline__ int next_of(const uint4 *at) {
    unsigned got, x;
    asm volatile(
        "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(at))
        : "memory");
    return got ? (int)x : -1;
}
// Eight 32-bit words to global memory: one 32-byte store where the address allows it.
__device__ __forceinline__ void store32(void *at, const unsigned (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                     "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// 16 32-bit columns into this thread's TMEM lane; the caller waits (tmem_wait_st).
__device__ __forceinline__ void tmem_st16_async(unsigned taddr, const unsigned (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Whether the phase is over; does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, unsigned parity) {
    unsigned done;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done;
}

constexpr int kPromptProbes = 1 << 20;  // of one barrier phase before a wait is given up (a probe sleeps for a while)

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    constexpr int DP = C::DP, NT = C::NT, NST = C::NST, SPB = C::SPB, SCHED = C::kSched;
    constexpr int kWarpMma = C::kSoftmaxWarps, kWarpTma = kWarpMma + 2, kWarpDeal = kWarpMma + 3;
    using Item = PromptItem;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sQ = smem_raw + (-smem_u32(smem_raw) & 1023u);  // pointer arithmetic keeps the shared address space
    unsigned char *ring = sQ + NT * C::kQTile;
    uint4 *answer = reinterpret_cast<uint4 *>(ring + (size_t)NST * C::kStage);
    int4 *sItem = reinterpret_cast<int4 *>(answer + 1);  // [SCHED] items
    uint64_t *bars = reinterpret_cast<uint64_t *>(sItem + 5 * SCHED);
    uint64_t *full = bars, *empty = full + NST, *q_full = empty + NST, *q_empty = q_full + 1, *s_free = q_empty + 1, *s_full = s_free + 1;
    uint64_t *p_half = s_full + 2, *p_full = p_half + 2, *pv_done = p_full + 2, *drain = pv_done + 2;  // P of keys 0-63 and 64-127
    uint64_t *sched_full = drain + 2, *sched_empty = sched_full + SCHED, *asked = sched_empty + SCHED;
    int2 *sOdd = reinterpret_cast<int2 *>(bars + C::kBars);  // segment's number, item's place in it
    unsigned *tslot = reinterpret_cast<unsigned *>(sOdd + C::kOdd);
    volatile int *sAbort = reinterpret_cast<volatile int *>(tslot + 1), *sCount = sAbort + 1, *sNext = sAbort + 2;  // items to run again; the item after them
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < C::kBars; ++i) {
            uint64_t *b = bars + i;
            // P, and S once it is read: every warp of a tile; an item is released by every warp but the one that deals it out
            mbar_init(b, (b >= p_half && b < pv_done) || b == s_free ? 4 : b >= sched_empty && b < asked ? 3 + C::kSoftmaxWarps : 1);
        }
        fence_barrier_init();
        *sAbort = 0;
        *sCount = 0;
        *sNext = blockIdx.x;
    }
    Segment seen{0, 0, 0, 0};  // dealer: segment `lane`, on its way while the barriers and TMEM are set up
    if (warp == kWarpDeal) {
        pdl_wait();
        if (lane < p.S) seen = load_segment(p.seq_info, lane);
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = *tslot;
    pdl_wait();
    pdl_trigger();

    // Bounded wait of one thread on one phase; false on a timeout, here or in another role.  (The code of what
    // runs all the time has to stay small: with 250 KB of it the products' warp waited for instructions half its time.)
    auto wait_one = [&](uint64_t *bar, unsigned parity) -> bool {
        int left = kPromptProbes;
#pragma unroll 1
        while (!mbar_try_wait(bar, parity))
            if (--left == 0 || *sAbort) {
                *sAbort = 1;
                return false;
            }
        return true;
    };
    // The same of a whole warp.
    auto wait_bar = [&](uint64_t *bar, unsigned parity) -> bool { return __all_sync(0xffffffffu, wait_one(bar, parity)); };

    int stages = 0;             // stages used so far
    unsigned used = 0, phase = 0;  // bit slot: a P slot has been used; how often, modulo two (S products: of S itself)
    unsigned s_phase = 0;          // softmax: blocks of the tile so far, modulo two
    unsigned queries = 0;       // items with rows so far
    int nth = 0;                // items taken from the scheduler so far
    bool ok = true;
    unsigned answers = 0;

    // The copies of one item (a whole warp: lane c has stage c of every block; one thread for all of them takes 450 cycles a stage).
    auto copy_item = [&](const Item &w) {
        if (queries > 0) ok = ok && wait_bar(q_empty, (queries - 1) & 1);
        if (!ok) return;
        if (lane == 0) {
            unsigned bytes = 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) bytes += w.last[t] > w.first[t] ? DP / 64 * p.tokens * p.G * 128 : 0;
            mbar_expect_tx(q_full, bytes);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (w.last[t] > w.first[t])
#pragma unroll 1
                    for (int c = 0; c < DP / 64; ++c)
                        tma_load_3d(sQ + t * C::kQTile + c * C::kPart, &p.tmap_q, q_full, c * 64, w.h * p.G, w.q0 + w.token0 + t * p.tokens);
        }
        ++queries;
        // K(b0), K(b0 + 1), V(b0), K(b0 + 2), V(b0 + 1), ..: S is a block ahead
        const int n = w.b1 - w.b0;
#pragma unroll 1
        for (int i = 0; ok && i < 2 * n; ++i) {
            const bool k = i == 0 || ((i & 1) && i < 2 * n - 1);
            const int block = w.b0 + (k ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : i / 2 - 1);
            const int mine = stages + lane, st = mine % NST;
            bool todo = lane < SPB;
            int left = 64 * kPromptProbes;
#pragma unroll 1
            for (;; --left) {
                if (todo && (mine < NST || mbar_test_wait(empty + st, ((mine / NST) - 1) & 1))) {
                    todo = false;
                    mbar_expect_tx(full + st, C::kStage);
                    unsigned char *to = ring + (size_t)st * C::kStage;
#pragma unroll
                    for (int x = 0; x < C::kCols / 64; ++x)
                        tma_load_3d(to + x * C::kPart, k ? &p.tmap_k : &p.tmap_v, full + st, lane * C::kCols + x * 64, w.h, w.q0 + block * C::kKeys);
                }
                if (!__any_sync(0xffffffffu, todo)) break;
                if (__any_sync(0xffffffffu, left == 0 || *sAbort)) {  // (every lane leaves at the same vote)
                    *sAbort = 1;
                    ok = false;
                    break;
                }
            }
            stages += SPB;  // (some of them copied, where a wait ran out)
        }
    };
    // The products: one warp has S, one P V (one lane of each issues).  A look at an mbarrier takes 110 cycles even if
    // it is open, a commit 60, and an issuing warp waits behind its products: one warp for all of them left the tensor core
    // idle half the time (4700 cycles for the blocks of two tiles, 2050 of them products).
    const unsigned lead = lane == 0;
    unsigned ring_at = 0, ring_phase = 0;    // the stage to be read next
    // The stages of the next block, and the way over blocks that are the other warp's.
    auto next_block = [&](unsigned (&at)[SPB], unsigned (&ph)[SPB]) {
#pragma unroll
        for (int c = 0; c < SPB; ++c) {
            at[c] = ring_at;
            ph[c] = ring_phase;
            if (++ring_at == NST) {
                ring_at = 0;
                ring_phase ^= 1;
            }
        }
    };
    auto block_ready = [&](const unsigned (&at)[SPB], const unsigned (&ph)[SPB]) { return wait_bar(full + at[0], ph[0]); };
    auto release = [&](const unsigned (&at)[SPB]) { umma_commit_by(lead, empty + at[0]); };  // once what has been issued so far is done
    // S of tile t and the block in stages `at`; what was there has been read.  (Above head_dim 128 a block is two stages, and
    // the ring holds two blocks and a half: each, of K and of V, is waited for and given back by itself, so that the next one is on its
    // way while the other half is used; both at once: 209 us of sliding windows at head_dim 256, now 198.  Four stages of
    // 16 KB a block: 224 to 247, more waits, commits and copies than their earlier starts are worth.)
    auto issue_s = [&](int t, const unsigned (&at)[SPB], const unsigned (&ph)[SPB]) {
        const unsigned q_lo = UmmaDesc(smem_u32(sQ), 16).lo + t * (C::kQTile >> 4), k_lo = UmmaDesc(smem_u32(ring), 16).lo;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < SPB; ++c) {
            if (SPB > 1) {
                if (!wait_bar(full + at[c], ph[c])) return false;
                tc_fence_after();
            }
            const unsigned qd = q_lo + (c * (C::kCols / 64) * C::kPart >> 4), kd = k_lo + at[c] * (C::kStage >> 4);
#pragma unroll
            for (int k = 0; k < C::kCols / 16; ++k) {
                const unsigned off = ((k >> 2) * C::kPart + (k & 3) * 32) >> 4;
                umma_ss(lead, tmem, qd + off, kd + off, umma_idesc_bf16(128, 128, 0), c > 0 || k > 0);
            }
            if (SPB > 1) umma_commit_by(lead, empty + at[c]);
        }
        umma_commit_by(lead, s_full + t);
        return true;
    };
    // O of tile t += P in slot times the V block in stages `at` (two stages: the columns of one, then those of the other)
    auto issue_pv = [&](int t, const unsigned (&at)[SPB], const unsigned (&ph)[SPB], int slot, bool fresh) {
        const unsigned v_lo = UmmaDesc(smem_u32(ring), C::kPart).lo;
#pragma unroll
        for (int c = 0; c < SPB; ++c) {
            if (SPB > 1 && !wait_bar(full + at[c], ph[c])) return false;
            const unsigned vd = v_lo + at[c] * (C::kStage >> 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (c == 0 && !wait_bar((half ? p_full : p_half) + slot, phase >> slot & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int u = 4 * half; u < 4 * half + 4; ++u)
                    umma_ts(lead, tmem + C::kColO + t * DP + c * C::kCols, tmem + C::kColP + slot * 64 + u * 8, vd + (u * 2048 >> 4), umma_idesc_bf16(128, C::kCols, 1),
                            !fresh || u > 0);
            }
            if (SPB > 1) umma_commit_by(lead, empty + at[c]);
        }
        umma_commit_by(lead, pv_done + slot);
        phase ^= 1u << slot;
        return true;
    };
    // (copied in this order: K(b0), K(b0 + 1), V(b0), K(b0 + 2), V(b0 + 1), ..)
    auto scores_of_item = [&](const Item &w) {
        unsigned at[SPB], ph[SPB];
        ok = ok && wait_bar(q_full, queries & 1);
        ++queries;
#pragma unroll 1
        for (int j = w.b0; ok && j < w.b1; ++j) {
            if (j > w.b0 + 1) next_block(at, ph);  // V(j - 2)
            next_block(at, ph);
            if (SPB == 1) ok = block_ready(at, ph);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (ok && j >= w.first[t] && j < w.last[t]) {
                    if (used) ok = wait_bar(s_free, phase);  // the S before has been read
                    if (!ok) break;
                    phase ^= used;
                    used = 1;
                    ok = issue_s(t, at, ph);
                }
            if (SPB == 1 && ok) release(at);
        }
        if (!ok) return;
        umma_commit_by(lead, q_empty);
        if (w.b1 - w.b0 > 1) next_block(at, ph);  // the last two V
        next_block(at, ph);
    };
    auto sums_of_item = [&](const Item &w) {
        unsigned at[SPB], ph[SPB];
#pragma unroll 1
        for (int j = w.b0; ok && j < w.b1; ++j) {
            if (j == w.b0) next_block(at, ph);     // K(b0)
            if (j + 1 < w.b1) next_block(at, ph);  // K(j + 1)
            next_block(at, ph);
            if (SPB == 1) ok = block_ready(at, ph);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (ok && j >= w.first[t] && j < w.last[t]) ok = issue_pv(t, at, ph, NT == 2 ? t : (j - w.b0) & 1, j == w.first[t]);
            if (SPB == 1 && ok) release(at);
        }
    };
    // The rows of one item (a softmax warp).
    auto rows_of_item = [&](const Item &w, bool careful) {
        const int t = warp >> 2, r = tid & 127;  // tile, row of it
        const unsigned lane_off = (unsigned)(32 * (warp & 3)) << 16;
        const int token = w.token0 + t * p.tokens + r / p.G, begin = stages;
        const bool real = r < p.tokens * p.G && token < w.ql;
        stages += 2 * SPB * (w.b1 - w.b0);
        int lo_r = 0, hi_r = 0;
        if (real) row_key_bounds(token, w.ql, p.causal, p.window, 0, lo_r, hi_r);
        const float sc = p.scale_log2;
        float m = kNoScore, l = 0.f;
        // (no index of a run-time value: the item would live in local memory, 500 cycles a look where the products' warp asks between two of them)
        const int f = NT == 1 ? w.b0 : t ? w.first[NT - 1] : w.first[0], e = NT == 1 ? w.b1 : t ? w.last[NT - 1] : w.last[0];
        if (e <= f) return;
        // blocks that every row of the warp sees whole (rows that are none do not matter)
        const int in0 = __reduce_max_sync(0xffffffffu, real ? (lo_r + C::kKeys - 1) / C::kKeys : 0);
        const int in1 = __reduce_min_sync(0xffffffffu, real ? hi_r / C::kKeys : INT_MAX);
#pragma unroll 1
        for (int j = f; ok && j < e; ++j) {
            const int slot = NT == 2 ? t : (j - w.b0) & 1;
            const unsigned p_addr = tmem + lane_off + C::kColP + slot * 64;
            if (!(ok = wait_bar(s_full + t, s_phase))) break;
            s_phase ^= 1;
            tc_fence_after();
            unsigned x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_async(tmem + lane_off + 32 * c, x[c]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free);  // S is in registers: the next one may go over it
            __syncwarp();                        // (what follows is the whole warp's)
            // (P's slot: whether the product that read it is done, asked before it is needed; an answer takes 110 cycles)
            const bool p_free = !(used >> slot & 1) || mbar_try_wait(pv_done + slot, (phase >> slot & 1) ^ 1);
            used |= 1u << slot;
            const int pos0 = j * C::kKeys;
            if (j < in0 || j >= in1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // bits of the chunk's keys that the row sees
                    const int a = lo_r - pos0 - 32 * c, b = hi_r - pos0 - 32 * c;
                    const unsigned see = (b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u) & (a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a);
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[c][k] = see & (1u << k) ? x[c][k] : 0xff800000u;
                }
            }
            float mx;
            {   // row maximum as a tree of three-way maxima
                float y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float z[11];
#pragma unroll
                    for (int k = 0; k < 10; ++k)
                        z[k] = max3(__uint_as_float(x[c][3 * k]), __uint_as_float(x[c][3 * k + 1]), __uint_as_float(x[c][3 * k + 2]));
                    z[10] = fmaxf(__uint_as_float(x[c][30]), __uint_as_float(x[c][31]));
                    y[c] = max3(max3(max3(z[0], z[1], z[2]), max3(z[3], z[4], z[5]), max3(z[6], z[7], z[8])), z[9], z[10]);
                }
                mx = fmaxf(max3(y[0], y[1], y[2]), y[3]) * sc;
            }
            if (!__all_sync(0xffffffffu, p_free) && !(ok = wait_bar(pv_done + slot, (phase >> slot & 1) ^ 1))) break;
            const bool grow = mx > m + kPromptLazy;
            if (__any_sync(0xffffffffu, grow)) {
                const float m_new = grow ? mx : m, alpha = exp2_fast(m - m_new);
                if (j > f && __any_sync(0xffffffffu, grow && m != kNoScore)) {
                    // (no product is in flight on O: with one tile the last one was in the other slot)
                    if (NT == 1 && !(ok = wait_bar(pv_done + (slot ^ 1), (phase >> (slot ^ 1) & 1) ^ 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < DP; c0 += 32) {
                        float o[32];
                        tmem_ld32(tmem + lane_off + C::kColO + t * DP + c0, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= alpha;
                        tmem_st32(tmem + lane_off + C::kColO + t * DP + c0, o);
                    }
                }
                l *= alpha;
                m = m_new;
            }
            const uint64_t sc2 = f32x2(sc, sc), m2 = f32x2(-m, -m);
            uint64_t la = 0, lb = 0;
            const bool zero_v = careful && !(pos0 >= w.in_lo && pos0 + C::kKeys <= w.in_hi);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                unsigned pk[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float e0, e1;
                    f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[c][2 * k]), __uint_as_float(x[c][2 * k + 1])), sc2, m2), e0, e1);
                    e0 = exp2_fast(e0);
                    e1 = exp2_fast(e1);
                    if (k & 1) lb = add_f32x2(lb, f32x2(e0, e1));
                    else la = add_f32x2(la, f32x2(e0, e1));
                    pk[k] = pack_bf16x2(e0, e1);
                }
                tmem_st16_async(p_addr + 16 * c, pk);
                if (c == 1 && !zero_v) {  // the first keys' weights are there: their products may start
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_half + slot);
                    __syncwarp();
                }
            }
            {
                float l0, l1;
                f32x2_split(add_f32x2(la, lb), l0, l1);
                l += l0 + l1;
            }
            if (zero_v) {
                // V rows that not every row of the item sees: what is not finite reads zero
                const int i0 = begin + SPB * ((min(j + 1, w.b1 - 1) - w.b0 + 1) + (j - w.b0));
                const int key = pos0 + r;
#pragma unroll 1
                for (int c = 0; ok && c < SPB; ++c) {
                    ok = wait_bar(full + (i0 + c) % NST, ((i0 + c) / NST) & 1);
                    if (!ok || (key >= w.in_lo && key < w.in_hi)) continue;
#pragma unroll 1
                    for (int x8 = 0; x8 < C::kCols / 8; ++x8) {
                        uint4 *at = reinterpret_cast<uint4 *>(ring + (size_t)((i0 + c) % NST) * C::kStage + (x8 >> 3) * C::kPart + r * 128 + (x8 & 7) * 16);
                        uint4 v = *at;
                        unsigned u[4] = {v.x, v.y, v.z, v.w};
                        bool odd = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (!not_finite(u[i])) continue;
                            odd = true;
                            if ((u[i] & 0x7f80u) == 0x7f80u) u[i] &= 0xffff0000u;
                            if ((u[i] & 0x7f800000u) == 0x7f800000u) u[i] &= 0xffffu;
                        }
                        if (odd) *at = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                __syncwarp();
                fence_proxy_async();
                if (!ok) break;
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (zero_v) mbar_arrive(p_half + slot);
                mbar_arrive(p_full + slot);
            }
            phase ^= 1u << slot;
        }
        // ---- the rows' ends: the last product has landed
        const int slot = NT == 2 ? t : (e - 1 - w.b0) & 1;
        if (ok) ok = wait_bar(pv_done + slot, (phase >> slot & 1) ^ 1);
        tc_fence_after();
        const long long row = (long long)w.q0 + (real ? token : 0);
        const int hq = w.h * p.G + (real ? r % p.G : 0);
        const bool zero = !ok || l == 0.f;
        const float inv = zero ? 0.f : 1.f / l;
        const long long at = (row * p.Hq + hq) * p.D;
        bool odd = false;
#pragma unroll 1
        for (int c0 = 0; c0 < DP; c0 += 32) {
            unsigned x[32];
            __syncwarp();  // lanes without a row are ahead of the others' stores; the load is the whole warp's
            tmem_ld32_async(tmem + lane_off + C::kColO + t * DP + c0, x);
            tmem_wait_ld();
            float o[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(x[k]);
            if (!real) continue;
            if (careful) {
                float y[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = o[k];
#pragma unroll 1
                for (int key = lo_r; key < hi_r; ++key) {
                    if (key >= w.in_lo && key < w.in_hi) key = w.in_hi;  // (those every row sees were not touched)
                    if (key < hi_r) prompt_add_key(p, (long long)w.q0 + key, row, w.h, hq, c0, m, y);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = y[k];
            }
            float test[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                test[k & 3] = fmaf(o[k], 0.f, test[k & 3]);  // NaN where one is not finite
                o[k] = zero ? 0.f : o[k] * inv;
            }
            odd |= (test[0] + test[1]) + (test[2] + test[3]) != 0.f;
            if (p.out_bf16) {
                __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(p.out) + at + c0;
                if (c0 + 32 <= p.D) {
                    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {
                        unsigned v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(o[k + 2 * i], o[k + 2 * i + 1]);
                        store32(dst + k, v, wide);
                    }
                    continue;
                }
            } else if (c0 + 32 <= p.D) {
                float *dst = reinterpret_cast<float *>(p.out) + at + c0;
                const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    unsigned v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(o[k + i]);
                    store32(dst + k, v, wide);
                }
                continue;
            }
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                if (c0 + k < p.D) prompt_store4(p, at + c0 + k, make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]));
        }
        if (real && p.lse) p.lse[row * p.Hq + hq] = zero ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
        // (a row with a NaN sum has one among its own scores)
        if (!careful && ok && __any_sync(0xffffffffu, odd && l == l) && lane == 0) {
            const int n = atomicAdd(const_cast<int *>(sCount), 1);
            sOdd[n % C::kOdd] = make_int2(w.s, w.place);  // (never that many: see below)
        }
        __syncwarp();
        tc_fence_before();
    };

    // What a CTA does: items until none is left, or until the list of those to run again is nearly
    // full (the items on their way may each add one a softmax warp); then that list.
    constexpr int kListRoom = C::kOdd - (SCHED + 2) * C::kSoftmaxWarps;  // (asked before the slot is free: a slow warp may be two items behind)
    static_assert(kListRoom > 0, "the list holds what the items on their way may add");
    // Waits on the scheduler last as long as an item may take, and end whatever has happened to the others.
    auto wait_long = [&](uint64_t *bar, unsigned parity) -> bool {
        int left = 64 * kPromptProbes;
#pragma unroll 1
        while (!mbar_try_wait(bar, parity))
            if (--left == 0) {
                *sAbort = 1;
                return false;
            }
        return true;
    };
    // The next item of a role, into w (a whole warp); false where there is none.
    Item w;
    auto take = [&](bool) -> bool {
        const int i = nth++ % SCHED;
        const bool got = __all_sync(0xffffffffu, wait_long(sched_full + i, ((nth - 1) / SCHED) & 1));
        w.from(sItem + 5 * i);
        __syncwarp();
        if (got && lane == 0) mbar_arrive(sched_empty + i);
        ok = ok && got;
        return got && w.kind != kNoItem;
    };
    // A role's items: those of the grid, then, where all roles have come to the end of
    // them, those of the list, and so on until none is left.
    auto all_items = [&](auto &&next, auto &&run) {
        bool careful = false;
#pragma unroll 1
        for (;;) {
            if (next(careful)) {
                run();
                __syncwarp();
                continue;
            }
            __syncthreads();
            careful = !careful && *sCount > 0;
            if (careful) continue;
            const bool done = *sNext < 0 || *sAbort;
            __syncthreads();
            if (tid == 0) *sCount = 0;
            __syncthreads();
            if (done) return;
        }
    };
    if (warp < C::kSoftmaxWarps) {
        if constexpr (C::kRegsSoftmax > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegsSoftmax));
        all_items(take, [&]() {
            if (w.tokens > 0) rows_of_item(w, w.kind == kCarefulItem);
        });
    } else {
        if constexpr (C::kRegsSoftmax > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsOthers));
        if (warp < kWarpTma) {
            all_items(take, [&]() {
                if (w.tokens > 0) {
                    if (warp == kWarpMma) scores_of_item(w);
                    else sums_of_item(w);
                }
                if (warp == kWarpMma) return;
                if (w.rows_of >= 0) prompt_coverage(p, w.rows_of, lane);
                if (w.fault && w.place < p.Hkv) {  // (one warp writes its rows)
                    if (lane == 0) atomicOr(p.err, w.fault);
                    if (w.q0 >= 0)           // a negative q_start covers nothing
                        for (long long r = w.q0; r < min((long long)w.q0 + w.ql, (long long)p.total_rows); ++r)
                            prompt_zero(p, r, w.h * p.G, p.G, lane, 32);
                }
            });
        } else if (warp == kWarpTma) {
            all_items(take, [&]() {
                if (w.tokens > 0 && ok) copy_item(w);
            });
        } else {
            int id = blockIdx.x;
            bool asking = false, held = true, cover = true;  // an answer is to come; the item is still to be given out; its number's rows too
            long long unit = id / p.Hkv, units = -1;         // the item's place among those of a kv head; how many there are
            // ---- units to items: lane i has segment s0 + i of the table and its n items; those of 32 segments come the last ones first
            int s0 = 0, n = 0, all = 0, top = 0, passed = 0;  // items of the 32; the item of each segment looked at, and those of the 32 before it
            long long before = 0;                             // items before s0
            bool loaded = false, again = false;
            Segment o = seen;
            auto seek = [&](Segment &g, int &index) -> int {  // the segment of `unit`, or -1
                if (unit < before + passed) {
                    if (unit < before) {
                        s0 = 0;
                        before = 0;
                    }
                    loaded = false;
                }
#pragma unroll 1
                for (;;) {
                    if (!loaded) {
                        if (again) o = s0 + lane < p.S ? load_segment(p.seq_info, s0 + lane) : Segment{0, 0, 0, 0};
                        again = true;
                        n = s0 + lane < p.S ? prompt_items(p, o, NT) : 0;
                        all = __reduce_add_sync(0xffffffffu, n);
                        top = __reduce_max_sync(0xffffffffu, n) - 1;
                        passed = 0;
                        loaded = true;
                    }
                    if (unit < before + all) break;
                    if (s0 + 32 >= p.S) return -1;
                    before += all;
                    s0 += 32;
                    loaded = false;
                }
                const int at = (int)(unit - before);
                unsigned m;
#pragma unroll 1
                for (;;) {
                    m = __ballot_sync(0xffffffffu, n > top);
                    const int c = __popc(m);
                    if (at - passed < c) break;
                    // as many of a segment's items as the same segments have
                    const int down = min((at - passed) / c, top + 1 - __reduce_max_sync(0xffffffffu, n > top ? 0 : n));
                    passed += down * c;
                    top -= down;
                }
                for (int l = at - passed; l; --l) m &= m - 1;
                const int l = __ffs(m) - 1;  // the one of them
                g.q0 = __shfl_sync(0xffffffffu, o.q0, l);
                g.ql = __shfl_sync(0xffffffffu, o.ql, l);
                g.kend = __shfl_sync(0xffffffffu, o.kend, l);
                index = top;
                return s0 + l;
            };
            int done = 0;  // of the list
            all_items([&](bool careful) -> bool {
                Segment g{0, 0, 0, 0};
                int s = -1, index = 0, h = 0;
                bool now = false;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (careful) {
                    const int listed = min(*sCount, C::kOdd);
                    int2 e = make_int2(0, 0);
#pragma unroll 1
                    for (; !now && done < listed; ++done) {  // (each warp of an item may have put it there)
                        e = sOdd[done];
                        now = true;
#pragma unroll 1
                        for (int k = 0; k < done; ++k) now = now && !(sOdd[k].x == e.x && sOdd[k].y == e.y);
                    }
                    now = __shfl_sync(0xffffffffu, now && !*sAbort, 0);
                    if (now) {
                        s = e.x;
                        g = load_segment(p.seq_info, s);
                        index = e.y / p.Hkv;
                        h = e.y % p.Hkv;
                    }
                } else {
                    done = 0;
                    if (!held) {
                        if (units < 0) {  // (asked while the first item is on its way)
                            units = 0;
#pragma unroll 4
                            for (int i = lane; i < p.S; i += 32) units += prompt_items(p, load_segment(p.seq_info, i), NT);
#pragma unroll
                            for (int d = 16; d; d >>= 1) units += __shfl_xor_sync(0xffffffffu, units, d);
                        }
                        cover = id < 0 || unit + p.units >= units;
                        if (!cover) {  // segments that overlap may have more items than the grid
                            unit += p.units;
                        } else {
                            id = -1;
                            if (lane == 0 && asking) {  // the item after the last one
                                if (wait_long(asked, answers & 1)) id = next_of(answer);
                                else ok = false;
                                ++answers;
                            }
                            asking = false;
                            id = __shfl_sync(0xffffffffu, id, 0);
                            unit = id / p.Hkv;
                        }
                    }
                    held = id >= 0 && __shfl_sync(0xffffffffu, *sCount, 0) >= kListRoom;  // the list is run first
                    now = id >= 0 && !held;
                    if (now) {
                        h = id % p.Hkv;
                        s = seek(g, index);
                    }
                }
                prompt_item<NT>(p, w, g, s, index, h);
                w.kind = !now ? kNoItem : careful ? kCarefulItem : kItem;
                w.rows_of = now && !careful && cover ? id : -1;
                const int i = nth % SCHED;
                if (lane == 0) {
                    if (nth >= SCHED) ok = wait_long(sched_empty + i, ((nth / SCHED) - 1) & 1) && ok;
                    if (!careful) *sNext = id;
                    w.to(sItem + 5 * i);
                    mbar_arrive(sched_full + i);
                }
                ++nth;
                if (now && !careful && !asking) {  // for the item after this one: the answer is there when this one is on its way
                    asking = __shfl_sync(0xffffffffu, ok && !*sAbort, 0);  // (after a timeout the others still write this item's zeros)
                    if (asking && lane == 0) {
                        fence_proxy_async();  // the answer before has been read
                        mbar_expect_tx(asked, 16);
                        ask_next(answer, asked);
                    }
                }
                return now;
            }, [&]() {});
        }
    }
    if (*sAbort) {
        // what is on its way gets a bounded chance to land: copies, then products, before TMEM is freed
        if (warp == kWarpTma && lane == 0)
#pragma unroll 1
            for (int i = max(0, stages - NST); i < stages; ++i)
                mbar_wait_ns(full + i % NST, (i / NST) & 1);
        if ((warp == kWarpMma || warp == kWarpMma + 1) && lane == 0) {
            umma_commit(drain + (warp - kWarpMma));
            mbar_wait_ns(drain + (warp - kWarpMma), 0);
        }
        if (tid == 0) atomicOr(p.err, PKV_ERR_TIMEOUT);
        __syncthreads();
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");
    }
}

}  // namespace pkv
