// Append to an 8-bit cache, with per-head norm and rotary position of q and k (sm_103a).
//
// A page and kv head share a scale, so the unit of work is a page, not a row: a
// CTA takes one page of a segment's new rows, forms the rows' angles once, and its
// warps take heads (of q, then k, then v).  A warp holds the page's new rows of a head
// in registers, 16-byte loads all in flight together, turns them as the row kernel
// does (rope.cuh: same order of operations, so k is the row that a bf16 cache would
// hold; the queries of a long step go through that kernel itself), takes the largest magnitude of all of them, and writes codes, the scale and
// the rows as they are held.  Tokens that are in the page already keep the scale
// from shrinking; where it grows, their codes are brought to it.
//
// In a ring a scale is left over once the tokens that made it are overwritten or behind the
// window, or are those of an earlier sequence.  Where it is far (kScaleSlack8) above what the new rows need,
// the codes of the tokens that some row may still see are looked at, and where it is as far above theirs it comes down to the larger
// of both, which is exact for them.  Older tokens stay until they are overwritten (a rewind may bring them back), and saturate;
// a slot that the sequence has not come to holds nothing.  (A kernel of its own: with the look in the
// one of flat caches, 256 sequences of a row each took 9.8 us there, not 9.3, 12.9, not 11.3, at head_dim 256.)
//
// The tokens of one page may come from several segments of a call (pieces of one
// sequence, a padded batch that holds a segment twice).  The scale is theirs in
// common, so the lowest of them writes the page for all.  A row's queries are turned once, for the lowest
// segment that holds it (they may be turned in place).  Where the table's columns and rows
// ascend, as a step's mostly do, or no other valid segment names the same ones, none of that is asked.
//
// How many pages there are only the table says: every CTA sums it (a thread some
// segments) and takes every n-th page of all segments end to end.  (A CTA for each page that a
// segment could have at most was 13,000 CTAs for a step of 256 sequences, 18.6 us.)
#pragma once

#include "fp8.cuh"
#include "rope.cuh"

namespace pkv {

constexpr int kAppend8Warps = 4, kAppend8Threads = kAppend8Warps * 32;
// Doublings by which a ring's page may have too large a scale: of the 14.8 from 448 down to the first value that loses
// bits, so that rows of less than 2^-6 of the scale's largest start it anew.  (With four, pages of ordinary rows are looked at now and then, a microsecond each.)
constexpr unsigned kScaleSlack8 = 6;
constexpr int kPlainRows = 3;  // beside RopePair: rows that are neither normalised nor turned, and no queries

struct Append8Params {
    RopeParams r;     // rows, rope, cache (lanes_log2, slices, row_ctas and page_warps unused)
    int page_ctas;    // CTAs that share the pages
    int head_ctas;    // and those that share a page's heads
};

// The kernel for how column pairs meet (RopePair, kPlainRows), one unit per head_dim.
const void *pick_append8_64(int pair, bool ring);
const void *pick_append8_128(int pair, bool ring);
const void *pick_append8_256(int pair, bool ring);

// Pages that a segment's new rows go to; none for an empty or refused one.
__device__ __forceinline__ int new_pages(const RopeParams &p, const Segment &sg) {
    if (sg.ql <= 0 || segment_fault(sg, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window)) return 0;
    const int n = (sg.kend + kPage - 1) / kPage - (sg.kend - sg.ql) / kPage;
    return p.ring_rows ? min(n, p.ring_rows / kPage) : n;  // (a step as long as the ring: its last page is its first one too)
}

// Row and position of slot `slot` (of the table's columns laid end to end) in segment o, or row -1.
__device__ __forceinline__ int row_of_slot(const Segment &o, int slot, int ring_rows, int &pos) {
    const int first = o.kend - o.ql;
    long long at = slot;
    if (ring_rows) {
        const int d = (slot - first) % ring_rows;
        at = (long long)first + (d < 0 ? d + ring_rows : d);
    }
    pos = (int)at;
    return at >= first && at < o.kend ? o.q0 + (int)(at - first) : -1;
}

// Which rows the page `tp` of segment s's column gets from all segments of the table,
// later ones before earlier ones where two write a slot, and the lowest segment that
// writes it.  One warp; lane j < 16 has slot j's row and position.  first, kend: of all segments that
// write this column, the lowest first position and the highest end.
static __device__ __noinline__ int merge_page_rows(const RopeParams &p, const Segment &sg, int tp, int lane, int &row, int &pos, int &first, int &kend) {
    int owner = -1;
    row = -1;
    pos = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < p.S; s0 += 32) {
        const Segment a = load_segment(p.seq_info, min(s0 + lane, p.S - 1));
        unsigned m = __ballot_sync(0xffffffffu, s0 + lane < p.S && a.col == sg.col && a.ql > 0 &&
                                                    !segment_fault(a, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window));
#pragma unroll 1
        for (; m; m &= m - 1) {
            const int s = s0 + __ffs(m) - 1;
            const Segment o = load_segment(p.seq_info, s);
            if (!new_pages_ok(p, o, lane)) continue;
            first = min(first, o.kend - o.ql);
            kend = max(kend, o.kend);
            int at;
            const int r = row_of_slot(o, tp * kPage + (lane & 15), p.ring_rows, at);
            if (!__any_sync(0xffffffffu, r >= 0)) continue;
            if (owner < 0) owner = s;
            if (r >= 0) {
                row = r;
                pos = at;
            }
        }
    }
    return owner;
}

// Slots whose row a segment below s, segment sg, holds as well: bit j for slot j.  One warp, lane j < 16 has slot j's row.
static __device__ __noinline__ unsigned rows_of_lower(const RopeParams &p, const Segment &sg, int s, int row, int lane) {
    unsigned taken = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < s; s0 += 32) {
        const Segment a = load_segment(p.seq_info, min(s0 + lane, s - 1));
        unsigned m = __ballot_sync(0xffffffffu, s0 + lane < s && overlap(a, sg) && new_pages(p, a) > 0);
#pragma unroll 1
        for (; m; m &= m - 1) {
            const Segment o = load_segment(p.seq_info, s0 + __ffs(m) - 1);
            if (!new_pages_ok(p, o, lane)) continue;
            taken |= __ballot_sync(0xffffffffu, lane < kPage && row >= o.q0 && (long long)row < (long long)o.q0 + o.ql);
        }
    }
    return taken;
}

// Which slots of a ring's page `tp` without a new row (`fresh`) hold a token, and, in the upper 16 bits, which of those some row may still see.
// One warp, lane j < 16: slot j.  first, kend: of the column's new rows.
__device__ __forceinline__ unsigned kept_tokens(const RopeParams &p, int tp, unsigned fresh, int first, int kend, int lane) {
    // the slot's token is the last one before kend
    const int back = (kend - 1 - (tp * kPage + (lane & 15))) % p.ring_rows;
    const long long at = (long long)kend - 1 - (back < 0 ? back + p.ring_rows : back);
    const bool there = lane < kPage && !(fresh >> (lane & 15) & 1u) && at >= 0;
    const unsigned m = __ballot_sync(0xffffffffu, there);
    return m | __ballot_sync(0xffffffffu, there && at > (long long)first - p.window) << 16;
}

// The scale that the tokens `count` of block `at` need, which are held under b0.
template <int D>
__device__ __noinline__ unsigned scale_needed(const unsigned char *at, unsigned count, unsigned b0, int lane) {
    unsigned top = 0;  // largest code
#pragma unroll 1
    for (int i = lane; i < kPage * D / 16; i += 32) {
        if (!(count >> (i / (D / 16)) & 1u)) continue;
        const uint4 w = reinterpret_cast<const uint4 *>(at)[i];
        const unsigned m = __vmaxu4(__vmaxu4(w.x & 0x7f7f7f7fu, w.y & 0x7f7f7f7fu), __vmaxu4(w.z & 0x7f7f7f7fu, w.w & 0x7f7f7f7fu));
        top = max(top, max(max(m & 0xffu, m >> 8 & 0xffu), max(m >> 16 & 0xffu, m >> 24)));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    unsigned lo, hi;
    unpack_e4m3x4(lo, hi, top);
    return scale8_of(__float_as_uint(half2_floats(lo).x * scale8_value(b0)));
}

// One head of one page: kind 0 q, 1 k, 2 v.  rows: the page's new rows by slot, -1: none.  tokens: kept_tokens of a ring's page.  angles: [16][rot_dim / 2].
template <int D, int PAIR, bool RING>
__device__ __forceinline__ void append8_head(const RopeParams &p, int kind, int h, const int *rows, unsigned tokens, const float2 *angles, long long block,
                                             float *stage, int lane) {
    constexpr int L = D / 8, TPI = 32 / L, IT = kPage / TPI;  // lanes a row, rows at once, turns
    using T = __nv_bfloat16;
    const int sub = lane / L, c = lane % L, half = p.rot_dim / 2;
    const T *src = reinterpret_cast<const T *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + h * D + c * 8;
    const long long src_stride = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    T *dst = reinterpret_cast<T *>(kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out);
    const long long dst_stride = kind == 0 ? p.q_out_stride : kind == 1 ? p.k_out_stride : p.v_out_stride;
    if (dst) dst += h * D + c * 8;
    const unsigned fresh = __ballot_sync(0xffffffffu, lane < kPage && rows[lane & 15] >= 0);  // bit j: slot j has a new row
    auto some = [&](int it) { return (fresh >> (it * TPI)) & ((1u << TPI) - 1u); };
    unsigned char *out = reinterpret_cast<unsigned char *>(kind == 1 ? p.k_pool : p.v_pool) + (block * p.Hkv + h) * block8_bytes(D);
    const unsigned kept = RING ? tokens & 0xffffu : ~fresh & ((1u << (31 - __clz(fresh))) - 1u);
    unsigned word = 0;  // the page's scale and NaN tokens, on their way with the rows
    if (kind && kept) word = *reinterpret_cast<const unsigned *>(out + 16 * D);
    Raw8<T> x[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        x[it].clear();
        if (!some(it)) continue;
        const int row = rows[it * TPI + sub];
        if (row >= 0) x[it].load(src + row * src_stride);
    }
    const T *weight = reinterpret_cast<const T *>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
    const bool turn = kind < 2 && p.rot_dim > 0;
    if (PAIR != kPlainRows && (weight || turn)) {
        const int left = p.rot_dim - c * 8;  // rotated columns from this lane's first on
        const unsigned turned = !turn ? 0u : left >= 8 ? 0xffu : left <= 0 ? 0u : (1u << left) - 1u;
        int partner = lane;
        if (PAIR == kByShuffle && c < half / 4) partner = lane + (c < half / 8 ? half / 8 : -(half / 8));
        float wt[8], wz[8];  // the columns' weights, and their partners'
#pragma unroll
        for (int e = 0; e < 8; ++e) wt[e] = wz[e] = 1.f;
        if (weight) {
            Raw8<T> r;
            r.load(weight + c * 8);
            r.get(wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (PAIR == kInLane) {
                    wz[e] = wt[e ^ 1];
                } else if constexpr (PAIR == kByShuffle) {
                    wz[e] = __shfl_sync(0xffffffffu, wt[e], partner);
                } else {
                    const int d = c * 8 + e, o = d < half ? d + half : d - half;
                    if (turned >> e & 1u) wz[e] = __bfloat162float(weight[o]);
                }
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            if (!some(it)) continue;
            float v[8], y[8], ca[8], sb[8], rinv = 1.f;
            x[it].get(v);
            if (weight) {
                uint64_t s2 = 0;
#pragma unroll
                for (int e = 0; e < 8; e += 2) s2 = fma_f32x2(f32x2(v[e], v[e + 1]), f32x2(v[e], v[e + 1]), s2);
                float ss, st;
                f32x2_split(s2, ss, st);
                ss += st;
#pragma unroll
                for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                rinv = rsqrtf(fmaf(ss, 1.f / D, p.eps));
            }
            const float2 *ang = angles + (it * TPI + sub) * half;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ca[e] = wt[e];
                sb[e] = 0.f;
                if (turned >> e & 1u) {
                    const int d = c * 8 + e, i = PAIR == kInLane ? d / 2 : d < half ? d : d - half;
                    const float2 t = ang[i];
                    ca[e] = t.x * wt[e];
                    sb[e] = ((PAIR == kInLane ? e & 1 : d >= half) ? t.y : -t.y) * wz[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) f32x2_split(mul_f32x2(f32x2(v[e], v[e + 1]), f32x2(ca[e], ca[e + 1])), y[e], y[e + 1]);
            if (turn) {
                float z[8];  // the partner columns' values
                if constexpr (PAIR == kInLane) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = v[e ^ 1];
                } else if constexpr (PAIR == kByShuffle) {
                    Raw8<T> o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o.w[e] = __shfl_sync(0xffffffffu, x[it].w[e], partner);
                    o.get(z);
                } else {
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) stage[e * 32 + lane] = v[e];
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = c * 8 + e, o = d < half ? d + half : d - half;
                        z[e] = d < p.rot_dim ? stage[(o & 7) * 32 + sub * L + (o >> 3)] : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)  // (columns that are not rotated never meet a partner's infinity)
                    if (turned >> e & 1u) y[e] = fmaf(z[e], sb[e], y[e]);
            }
            if (weight)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= rinv;
            x[it].set(y);
            if (rows[it * TPI + sub] < 0) x[it].clear();  // (a slot without a new row has no angles, and 1 / sqrt(eps) may be infinite)
        }
    }
    if (kind == 0) {
#pragma unroll
        for (int it = 0; it < IT; ++it)
            if (some(it)) {
                const int row = rows[it * TPI + sub];
                if (row >= 0) x[it].store(dst + row * dst_stride);
            }
        return;
    }
    // ---- the largest magnitude, NaN apart
    __nv_bfloat162 top = __float2bfloat162_rn(0.f), with_nan = top;
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 a = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x[it].w[e]));
            top = __hmax2(top, a);  // (takes the number of a number and a NaN)
            with_nan = __hmax2_nan(with_nan, a);
        }
    const unsigned tb = *reinterpret_cast<const unsigned *>(&top), nb = *reinterpret_cast<const unsigned *>(&with_nan);
    const unsigned amax = __reduce_max_sync(0xffffffffu, max(tb << 16, tb & 0xffff0000u));
    unsigned nan = 0;  // tokens that hold one
    if (__any_sync(0xffffffffu, max(nb << 16, nb & 0xffff0000u) > 0x7f800000u)) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            bool mine = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                unsigned &w = x[it].w[e];
                if ((w & 0x7fffu) > 0x7f80u) { mine = true; w &= 0xffff0000u; }
                if ((w & 0x7fff0000u) > 0x7f800000u) { mine = true; w &= 0xffffu; }
            }
            const unsigned m = __ballot_sync(0xffffffffu, mine);
#pragma unroll
            for (int r = 0; r < TPI; ++r)
                if (m >> (r * L) & (L == 32 ? 0xffffffffu : (1u << (L & 31)) - 1u)) nan |= 1u << (it * TPI + r);
        }
    }
    // ---- the page's scale: that of the tokens it keeps, or more
    unsigned b = scale8_of(amax);
    if (kept) {
        const unsigned b0 = min(word & 0xffu, kScaleMax8);
        nan |= (word >> 16) & kept;
        unsigned least = b0;
        if (RING && b0 > b + kScaleSlack8) {
            const unsigned theirs = scale_needed<D>(out, tokens >> 16, b0, lane);
            if (max(theirs, b) + kScaleSlack8 < b0) least = max(theirs, 1u);
        }
        b = max(b, least);
        if ((RING ? b != b0 : b > b0) && b0) {
            // to a larger scale: what is 2^-18 of 2^-9 or less reads zero anyway; to a smaller one: what is too large saturates
            float by = b - b0 < 32 ? __uint_as_float((127u + b0 - b) << 23) : 0.f;
            if (RING && b < b0) by = __uint_as_float((127u + min(b0 - b, 127u)) << 23);
#pragma unroll 1
            for (int it = 0; it < IT; ++it) {
                const int tok = it * TPI + sub;
                if (!(kept >> tok & 1u)) continue;
                uint2 *a = reinterpret_cast<uint2 *>(out + tok * D + 16 * place8(tok, c >> 1, D) + 8 * (c & 1));
                const uint2 w = *a;
                *a = make_uint2(scale_e4m3x4(w.x, by), scale_e4m3x4(w.y, by));
            }
        }
    }
    const float inv = scale8_inverse(b), scale = scale8_value(b);
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        if (!some(it)) continue;
        const int tok = it * TPI + sub, row = rows[tok];
        if (row < 0) continue;
        float v[8];
        x[it].get(v);
        uint2 w;
        w.x = pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        w.y = pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
        *reinterpret_cast<uint2 *>(out + tok * D + 16 * place8(tok, c >> 1, D) + 8 * (c & 1)) = w;
        if (dst) {
            unsigned q[4];
            unpack_e4m3x4(q[0], q[1], w.x);
            unpack_e4m3x4(q[2], q[3], w.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // (four significant bits: exact in bf16)
                const float2 f = half2_floats(q[e]);
                x[it].w[e] = nan >> tok & 1u ? 0x7fff7fffu : pack_bf16x2(f.x * scale, f.y * scale);
            }
            x[it].store(dst + row * dst_stride);
        }
    }
    if (lane == 0) *reinterpret_cast<unsigned *>(out + 16 * D) = b | nan << 16;
}

// The stored values of flat rows 0 .. n - 1 (pages in the order of the pool), [kv_heads][n][D]: D / 8 lanes a row, K then V.
struct Read8Params {
    const unsigned char *pool[2];
    __nv_bfloat16 *out[2];
    long long n;
    int Hkv, D;
};
static __global__ void __launch_bounds__(256) read8_kernel(const __grid_constant__ Read8Params p) {
    const int L = p.D / 8;
    const long long rows = 2ll * p.Hkv * p.n, step = (long long)gridDim.x * blockDim.x / L;
    const int c = threadIdx.x % L;
    for (long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / L; i < rows; i += step) {
        const long long tok = i % p.n;
        const int h = (int)(i / p.n % p.Hkv), side = i >= rows / 2, t = (int)(tok % kPage);
        const unsigned char *block = p.pool[side] + (tok / kPage * p.Hkv + h) * block8_bytes(p.D);
        const unsigned word = *reinterpret_cast<const unsigned *>(block + 16 * p.D);
        const uint2 w = *reinterpret_cast<const uint2 *>(block + t * p.D + 16 * place8(t, c >> 1, p.D) + 8 * (c & 1));
        const float scale = scale8_value(word & 0xffu);
        unsigned q[4];
        unpack_e4m3x4(q[0], q[1], w.x);
        unpack_e4m3x4(q[2], q[3], w.y);
        Raw8<__nv_bfloat16> x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = half2_floats(q[e]);
            x.w[e] = word >> (16 + t) & 1u ? 0x7fff7fffu : pack_bf16x2(f.x * scale, f.y * scale);
        }
        x.store(p.out[side] + (h * p.n + tok) * p.D + c * 8);
    }
}

template <int D, int PAIR, bool RING>
__global__ void __launch_bounds__(kAppend8Threads, D == 256 ? 3 : PAIR == kPlainRows && !(RING && D == 128) ? 5 : 4) append8_kernel(const __grid_constant__ Append8Params a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int sRow[2][kPage], sPos[2][kPage], sOwner;  // own rows (apart: queries'); those of every segment
    __shared__ unsigned sKept;  // (ring)
    __shared__ long long sSum[kAppend8Warps], sFirst;
    __shared__ int sSegment;
    const RopeParams &p = a.r;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pairs = PAIR == kPlainRows ? 0 : p.rot_dim / 2;
    float *stage = reinterpret_cast<float *>(smem) + warp * 256;                                                    // (kByShared)
    float2 *angles = reinterpret_cast<float2 *>(smem + (PAIR == kByShared ? kAppend8Warps * 1024 : 0));             // [16][pairs]
    const int hc = blockIdx.x % a.head_ctas, pc = blockIdx.x / a.head_ctas, ring_pages = p.ring_rows / kPage;
    pdl_wait();
    pdl_trigger();
    // ---- the pages of all segments: thread t sums segments t per .. (a table of one needs no sum)
    const int per = (p.S + kAppend8Threads - 1) / kAppend8Threads, s_lo = min(tid * per, p.S), s_hi = min(s_lo + per, p.S);
    long long mine = 0, upto, total;
    const bool queries = PAIR != kPlainRows && p.q;
    bool may_share = false;  // columns or rows that do not ascend
    Segment sg{0, 0, 0, 0};
    if (p.S > 1) {
        int last = -1;
        long long rows_to = INT32_MIN;  // end of the last one's rows
        if (s_lo > 0 && s_lo < s_hi) {
            const Segment o = load_segment(p.seq_info, s_lo - 1);
            last = o.col;
            rows_to = o.ql > 0 ? (long long)o.q0 + o.ql : INT32_MAX;
        }
#pragma unroll 4
        for (int i = s_lo; i < s_hi; ++i) {
            const Segment o = load_segment(p.seq_info, i);
            mine += new_pages(p, o);
            may_share |= o.col <= last;
            last = o.col;
            if (PAIR != kPlainRows) {
                may_share |= queries && o.ql > 0 && o.q0 < rows_to;
                rows_to = o.ql > 0 ? (long long)o.q0 + o.ql : INT32_MAX;
            }
            const unsigned fault = segment_fault(o, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
            if (fault && blockIdx.x == 0) atomicOr(p.err, fault);
        }
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) sSum[warp] = upto;
        may_share = __syncthreads_or(may_share);
        total = 0;
#pragma unroll
        for (int k = 0; k < kAppend8Warps; ++k) {
            if (k < warp) upto += sSum[k];
            total += sSum[k];
        }
    } else {
        sg = load_segment(p.seq_info, 0);
        total = new_pages(p, sg);
        const unsigned fault = segment_fault(sg, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
        if (fault && blockIdx.x == 0 && tid == 0) atomicOr(p.err, fault);
    }
    const int nq = p.q ? p.Hq : 0, items = nq + 2 * p.Hkv;
    long long end = 0, first = 0;  // pages before the segment's end, and before it
    int s = 0, p0 = 0;
    bool fine = false, shared = false, twice = false;
#pragma unroll 1
    for (long long at = pc; at < total; at += a.page_ctas) {
        if (at >= end) {  // another segment
            if (p.S > 1) {
                __syncthreads();
                if (upto - mine <= at && at < upto) {
                    long long x = upto - mine;
                    int i = s_lo;
#pragma unroll 1
                    for (;; ++i) {
                        const int n = new_pages(p, load_segment(p.seq_info, i));
                        if (at < x + n) break;
                        x += n;
                    }
                    sSegment = i;
                    sFirst = x;
                }
                __syncthreads();
                s = sSegment;
                first = sFirst;
                sg = load_segment(p.seq_info, s);
            }
            end = first + new_pages(p, sg);
            p0 = (sg.kend - sg.ql) / kPage;
            fine = new_pages_ok(p, sg, lane);  // (every warp sees the same)
            if (!fine && hc == 0 && tid == 0) atomicOr(p.err, PKV_ERR_BLOCK);
            shared = twice = false;  // another segment writes this column; a lower one has some of these rows
            if (may_share) {
#pragma unroll 4
                for (int t = tid; t < p.S; t += kAppend8Threads) {
                    const Segment o = load_segment(p.seq_info, t);
                    const bool writes = t != s && new_pages(p, o) > 0;
                    shared |= writes && o.col == sg.col;
                    if (PAIR != kPlainRows) twice |= writes && t < s && overlap(o, sg);
                }
                shared = __syncthreads_or(shared);
                if (queries) twice = __syncthreads_or(twice);
            }
        }
        if (!fine) continue;
        const int u = (int)(at - first);
        const int tp = ring_pages ? (p0 + u) % ring_pages : p0 + u;
        const long long block = p.block_table[(long long)sg.col * p.mbps + tp];
        __syncthreads();
        if (warp == 0) {
            int pos, row = row_of_slot(sg, tp * kPage + (lane & 15), p.ring_rows, pos), owner = s, from = sg.kend - sg.ql, to = sg.kend;
            const unsigned taken = queries && twice ? rows_of_lower(p, sg, s, row, lane) : 0u;
            if (lane < kPage) {
                sRow[0][lane] = taken >> lane & 1u ? -1 : row;
                sPos[0][lane] = pos;
            }
            if (shared) owner = merge_page_rows(p, sg, tp, lane, row, pos, from, to);
            const unsigned tokens = RING ? kept_tokens(p, tp, __ballot_sync(0xffffffffu, lane < kPage && row >= 0), from, to, lane) : 0u;
            if (lane < kPage) {
                sRow[1][lane] = row;
                sPos[1][lane] = pos;
            }
            if (lane == 0) {
                sOwner = owner;
                sKept = tokens;
            }
        }
        // Own rows serve q, those of every segment k and v; they are the same but where segments share a column or rows.
        const bool apart = shared || (queries && twice);
#pragma unroll 1
        for (int pass = 0; pass < (apart ? 2 : 1); ++pass) {
            const int i0 = pass ? nq : 0, i1 = apart && !pass ? nq : items;
            __syncthreads();
            if (pass && sOwner != s) break;
            if constexpr (PAIR != kPlainRows) {
                // a thread keeps to one pair, and takes every n-th slot
                const int width = pairs <= 32 ? 32 : pairs <= 64 ? 64 : 128, e = tid & (width - 1);
                if (e < pairs) {
                    const unsigned long long turn = p.turns[e];
                    const int axis = p.axis ? min((int)p.axis[e], p.axes - 1) : 0;
#pragma unroll 4
                    for (int j = tid / width; j < kPage; j += kAppend8Threads / width) {
                        const int row = sRow[pass][j];
                        if (row < 0) continue;
                        unsigned pos = (unsigned)sPos[pass][j];
                        if (p.positions) pos = (unsigned)p.positions[p.axis ? (long long)row * p.axes + axis : row];
                        angles[j * pairs + e] = angle_of(pos, turn, p.mscale);
                    }
                }
                __syncthreads();
            }
#pragma unroll 1
            for (int it = i0 + hc * kAppend8Warps + warp; it < i1; it += a.head_ctas * kAppend8Warps) {
                const int kind = it < nq ? 0 : it < nq + p.Hkv ? 1 : 2;
                append8_head<D, PAIR, RING>(p, kind, kind == 0 ? it : kind == 1 ? it - nq : it - nq - p.Hkv, sRow[pass], RING ? sKept : 0u, angles, block, stage, lane);
            }
        }
    }
}

}  // namespace pkv
