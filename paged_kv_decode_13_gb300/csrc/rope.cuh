// Per-head norm, rotary position and append of this step's rows (sm_103a).
//
// One pass over q, k and v: y = R(pos) (x * rsqrt(mean(x^2) + eps) * w) for q
// and k heads, q to its output rows, k and v to their cache slots.  Every value
// is read once and written once, about a dozen flops each.
//
// A warp takes one row (token) and a slice of its heads: lanes own 8 columns
// of a head, D / 8 lanes (rounded up to a power of two) a head, 32 / that many
// heads at once.  The row's angles are the same for every head: the lanes form
// them once a row, in shared memory of the warp's own, and keep those of their 8 columns,
// with the head weights folded in, in registers; the norm's sum and the
// rotation partner come by shuffles (or through shared memory where a
// half of rot_dim is no whole number of lanes).  No barrier.  With few rows
// several warps share a row's heads; with many, one wave of warps takes rows in
// turn.
//
// Small calls are a launch: one token of 32 + 8 + 8 heads 4.1 us, 256 tokens 7.0 us.
// Long ones should be bound by HBM and are bound by issue and latency: 16,400
// tokens of 32 + 8 + 8 heads of 128 (330 MB), norm and half the head rotated,
// 76 us, 4.3 TB/s, against 49 us at the rate of a copy; 2,800 instructions a token
// keep the schedulers 52 % busy, at 20 warps an SM (96 registers): four heads are
// loaded together but handled one behind the other, each a chain of a sum, shuffles and a
// root.  Three
// heads' loads in flight or six, more warps with fewer registers, prefetches,
// loads rolling from row to row (85 us) and a version fed by bulk copies through shared memory (95 us) were slower.
//
// Angles: turn_i = frequency / 2 pi as a 64-bit fraction of a turn, formed in
// double: off by at most 2^-55 of a turn a position for frequencies up to 1.  position *
// turn_i modulo 2^64 is its exact product, whose top 32 bits (2^-32) become a
// float of half turns (2^-26 of a turn) that sinpif / cospif take as it is: the angle
// is off by |position| 2^-55 + 2^-25.9 of a turn.
// (A float product pos * freq is off by 0.008 rad at position 131072.)
//
// The 4-bit cache stores V by token pairs, two tokens to a byte, so its V pages
// are written by page: a warp takes one (segment, kv head, page), gathers the
// page's new rows and merges their nibbles into the old ones.  K needs no
// merge (a byte is two columns of one token) and is quantised by the row warps.
// 16,600 tokens of 8 heads of 128: 49 us, 24 at the rate of a copy: the quantiser's
// instructions (maximum, scale, eight products rounded to codes, the byte
// exchange; 46 % of issue slots) and its shuffles' latency bound it.  A page's
// rows are loaded together first (loads one by one behind the stores: 98 us).
#pragma once

#include "fp4.cuh"

namespace pkv {

constexpr int kRopeWarps = 4;    // warps of a CTA
constexpr int kRopeUnroll = 4;   // head loads in flight per lane

enum RopeCache { kNoCache = 0, kSameType = 1, kFp4 = 2 };
enum RopePair { kInLane = 0, kByShuffle = 1, kByShared = 2 };

struct RopeParams {
    const void *q, *k, *v;            // rows; q may be null (no query heads), k and v null without a cache or k rows
    void *q_out, *k_out, *v_out;      // q_out null without q; k_out / v_out optional with a cache
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride, v_out_stride;  // elements between rows
    const int *positions;             // [rows] or null: the row's cache position
    const unsigned long long *turns;  // [rot_dim / 2]
    const void *q_weight, *k_weight;  // [D] or null
    float eps, mscale;
    int rot_dim, interleaved;
    int rows, Hq, Hkv, D;
    int lanes_log2;                   // lanes of a head
    int slices;                       // warps of a row
    int row_ctas;                     // CTAs of row warps; the rest write 4-bit V pages
    // cache
    void *k_pool, *v_pool;
    const int *block_table;
    const int4 *seq_info;
    unsigned *err;
    long long num_blocks;
    int S, max_seqs, mbps, ring_rows, window;
    int page_warps;                   // 4-bit cache: warps that share one (segment, kv head)'s new pages
};

// Every page the segment's new rows go to is inside the pool (the whole warp asks).
__device__ __forceinline__ bool new_pages_ok(const RopeParams &p, const Segment &sg, int lane) {
    const int *bt = p.block_table + (long long)sg.col * p.mbps;
    const int p0 = (sg.kend - sg.ql) / kPage, p1 = (sg.kend + kPage - 1) / kPage;
    bool ok = true;
    if (sg.ql > 0)
        for (int pb = p0 + lane; pb < p1; pb += 32) {
            const int b = bt[table_page(pb, p.ring_rows)];
            ok &= b >= 0 && (long long)b < p.num_blocks;
        }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool holds_row(const RopeParams &p, const Segment &sg, int row) {
    return sg.q0 <= row && (long long)row < (long long)sg.q0 + sg.ql &&
           !segment_fault(sg, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
}

// Lowest valid segment from `from` on that holds `row`, or -1 (the whole warp asks).
__device__ __forceinline__ int next_segment(const RopeParams &p, int row, int from, int lane) {
    for (int s0 = from; s0 < p.S; s0 += 32) {
        const int s = s0 + lane;
        const bool hit = s < p.S && holds_row(p, load_segment(p.seq_info, min(s, p.S - 1)), row);
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m) return s0 + __ffs(m) - 1;
    }
    return -1;
}

// A valid segment that holds `row`, or -1 (the whole warp asks): the lowest, but
// segment i for row i, as a decode step's table has it, is looked at first.
__device__ __forceinline__ int segment_of_row(const RopeParams &p, int row, int lane) {
    if (row < p.S && holds_row(p, load_segment(p.seq_info, row), row)) return row;
    return next_segment(p, row, 0, lane);
}

// Whether segments may share rows (the whole CTA asks): not where each begins at or past the end of the one
// before it, with empty ones only at the table's end, as steps mostly have
// them.  Asked once a CTA of a long table (place_row knows of a short one): a warp that asks for
// each segment (shares_rows) took 8 us of 53 for 4096 tokens of as many sequences.
__device__ __forceinline__ bool may_share_rows(const RopeParams &p) {
    if (p.S <= 32) return false;
    bool odd = false;
#pragma unroll 4
    for (int t = threadIdx.x + 1; t < p.S; t += kRopeWarps * 32) {
        const Segment a = load_segment(p.seq_info, t - 1), b = load_segment(p.seq_info, t);
        odd |= b.ql > 0 && (a.ql <= 0 || b.q0 < (long long)a.q0 + a.ql);
    }
    return __syncthreads_or(odd);
}
__device__ __forceinline__ bool overlap(const Segment &a, const Segment &b) {
    return a.q0 < (long long)b.q0 + b.ql && b.q0 < (long long)a.q0 + a.ql;
}
// Whether a segment but s has a row of sg, segment s (the whole warp asks).
__device__ __forceinline__ bool shares_rows(const RopeParams &p, const Segment &sg, int s, int lane) {
    bool any = false;
#pragma unroll 4
    for (int t = lane; t < p.S; t += 32) {
        any |= t != s && overlap(load_segment(p.seq_info, t), sg);
    }
    return __any_sync(0xffffffffu, any);
}

// Eight elements of a row as they are in memory.
template <typename T>
struct Raw8 {
    unsigned w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T *dst) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
            else x[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) {
                if (i & 1) w[i / 2] = pack_bf16x2(x[i - 1], x[i]);
            } else {
                w[i] = __float_as_uint(x[i]);
            }
        }
    }
};

// Quantise 8 columns of a bf16 row (half a scale group: lanes 2j and 2j + 1
// hold one).  Returns the codes; stored: x becomes the stored values.
//
// x / s: s has 4 significant bits and x 8, so the quotient is either exactly
// on a border b between two codes (a multiple of 1/4) or at least b 2^-8 away from
// it, 2^-10 at the lowest, 1/4.  x * (1 / s), whose error is below 2^-21 of it, is rounded to a
// multiple of 2^-11 by adding and taking off 3 * 2^11, which moves it by at most 2^-12: it
// stays on the same side, and is exactly on the border where x / s is.  The code
// is that of the exact quotient.
__device__ __forceinline__ unsigned quantise8(Raw8<__nv_bfloat16> &x, unsigned &scale, bool stored) {
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x.w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x.w[i])));
    unsigned amax = *reinterpret_cast<const unsigned *>(&m);
    amax = max(amax << 16, amax & 0xffff0000u);  // a NaN's bits are above all others
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    scale = scale4_of(amax);
    const float inv = scale4_inverse(scale);  // a zero scale: codes 0 with the signs of x
    float v[8];
    x.get(v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float a, b;
        f32x2_split(add_f32x2(fma_f32x2(f32x2(v[i], v[i + 1]), f32x2(inv, inv), f32x2(6144.f, 6144.f)), f32x2(-6144.f, -6144.f)), a, b);
        v[i] = copysignf(a, v[i]);
        v[i + 1] = copysignf(b, v[i + 1]);
    }
    const unsigned codes = pack_e2m1x8(v);
    if (stored) {
        unsigned h[4];
        unpack_e2m1x8(h, codes);
        const unsigned s2 = scale4_both(scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // exact in fp16, and in bf16
            const unsigned y = hmul2(h[i], s2);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
            x.w[i] = pack_bf16x2(f.x, f.y);
        }
    }
    return codes;
}

// One row warp's cache slot.
struct RopeSlot {
    long long block;  // page id
    int token;        // slot in the page
};

// The heads [h0, h1) of one kind (q, k or v) of a row.  ca, sb: this lane's
// factors of its own and its partner's columns; norm, turn: what is done to
// them; turned: bit e set where column e of the lane is rotated.
template <typename T, int CACHE, int PAIR>
__device__ __forceinline__ void rope_heads(const RopeParams &p, const T *src, T *dst, unsigned char *pool,
                                           const RopeSlot &slot, int h0, int h1, const float (&ca)[8],
                                           const float (&sb)[8], bool norm, bool turn, unsigned turned, int partner, float *stage, int lane) {
    const int per = 1 << p.lanes_log2, sub = lane >> p.lanes_log2, c = lane & (per - 1), heads = 32 >> p.lanes_log2;
    const bool col_ok = c * 8 < p.D;
    const bool whole = (p.rot_dim & 7) == 0;  // a lane's columns are all rotated or none
    const float inv_d = 1.f / (float)p.D;
    src += (h0 + sub) * p.D + c * 8;
    if (dst) dst += (h0 + sub) * p.D + c * 8;
    const int step = heads * p.D;
    if (CACHE == kSameType && pool)
        pool += (((slot.block * kPage + slot.token) * p.Hkv + h0 + sub) * p.D + c * 8) * (long long)sizeof(T);
    if (CACHE == kFp4 && pool) pool += (slot.block * p.Hkv + h0 + sub) * block4_bytes(p.D);
    const int pool_step = CACHE == kFp4 ? heads * block4_bytes(p.D) : step * (int)sizeof(T);
#pragma unroll 1
    for (int hb = h0 + sub; hb - sub < h1; hb += heads * kRopeUnroll) {
        Raw8<T> raw[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            raw[u].clear();
            if (col_ok && hb + u * heads < h1) raw[u].load(src + u * step);
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (hb - sub + u * heads >= h1) break;  // uniform
            const bool mine = col_ok && hb + u * heads < h1;
            if (norm || turn) {
                float x[8], y[8];
                raw[u].get(x);
                float rinv = 1.f;
                if (norm) {
                    uint64_t s2 = 0;
#pragma unroll
                    for (int e = 0; e < 8; e += 2) s2 = fma_f32x2(f32x2(x[e], x[e + 1]), f32x2(x[e], x[e + 1]), s2);
                    float ss, st;
                    f32x2_split(s2, ss, st);
                    ss += st;
                    for (int o = per >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    rinv = rsqrtf(fmaf(ss, inv_d, p.eps));
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    f32x2_split(mul_f32x2(f32x2(x[e], x[e + 1]), f32x2(ca[e], ca[e + 1])), y[e], y[e + 1]);
                if (turn) {
                    float z[8];  // the partner columns' values
                    if constexpr (PAIR == kInLane) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] = x[e ^ 1];
                    } else if constexpr (PAIR == kByShuffle) {
                        Raw8<T> o;
#pragma unroll
                        for (int e = 0; e < 2 * (int)sizeof(T); ++e) o.w[e] = __shfl_sync(0xffffffffu, raw[u].w[e], partner);
                        o.get(z);
                    } else {
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e) stage[e * 32 + lane] = x[e];
                        __syncwarp();
                        const int half = p.rot_dim / 2;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int d = c * 8 + e, o = d < half ? d + half : d - half;
                            z[e] = d < p.rot_dim ? stage[(o & 7) * 32 + (sub << p.lanes_log2) + (o >> 3)] : 0.f;
                        }
                    }
                    // Columns that are not rotated never meet a partner's infinity.
                    if (whole) {
                        if (turned)
#pragma unroll
                            for (int e = 0; e < 8; e += 2)
                                f32x2_split(fma_f32x2(f32x2(z[e], z[e + 1]), f32x2(sb[e], sb[e + 1]), f32x2(y[e], y[e + 1])), y[e], y[e + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (turned >> e & 1u) y[e] = fmaf(z[e], sb[e], y[e]);
                    }
                }
                if (norm)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) f32x2_split(mul_f32x2(f32x2(y[e], y[e + 1]), f32x2(rinv, rinv)), y[e], y[e + 1]);
                raw[u].set(y);
            }
            if constexpr (CACHE == kFp4) {
                if (pool) {  // the row as it would be handed on (bf16), quantised
                    unsigned scale;
                    const unsigned codes = quantise8(raw[u], scale, dst != nullptr);
                    if (mine) {
                        unsigned char *b = pool + u * pool_step;
                        *reinterpret_cast<unsigned *>(b + slot.token * (p.D / 2) + c * 4) = codes;
                        if ((c & 1) == 0) b[8 * p.D + slot.token * (p.D / 16) + c / 2] = (unsigned char)scale;
                    }
                }
            } else if (CACHE == kSameType && pool && mine) {
                raw[u].store(reinterpret_cast<T *>(pool + u * pool_step));
            }
            if (dst && mine) raw[u].store(dst + u * step);
        }
        src += kRopeUnroll * step;
        if (dst) dst += kRopeUnroll * step;
        if (CACHE != kNoCache && pool) pool += kRopeUnroll * pool_step;
    }
}

// What a row warp knows of the segment of its last row.
struct RowSegment {
    Segment sg{0, 0, 0, 0};
    int s = 0;             // its index, where `shared`
    bool pages_ok = false;
    bool may_share = false;  // 4-bit caches: segments of this table may share rows
    bool shared = false;     // and others have some of this one's
};
__device__ __forceinline__ void locate_row(const RopeParams &p, const Segment &sg, int row, RopeSlot &slot, long long &place) {
    place = (long long)sg.kend - sg.ql + (row - sg.q0);
    slot.block = p.block_table[(long long)sg.col * p.mbps + table_page((int)(place / kPage), p.ring_rows)];
    slot.token = (int)(place % kPage);
}
__device__ __forceinline__ bool ask_pages(const RopeParams &p, const Segment &sg, int lane) {
    const bool ok = new_pages_ok(p, sg, lane);
    if (!ok && lane == 0) atomicOr(p.err, PKV_ERR_BLOCK);
    return ok;
}
// Where a row goes; false where it goes nowhere (no valid segment, or a bad
// page).  c: the segment of the row before, looked up again when the row is
// past it.  The whole warp asks.  The V pages of a 4-bit cache are written for every
// segment of a row, and so is its K: the lowest segment that takes the row places it
// here, copy_k4_to_others the rest.
template <int CACHE>
__device__ __forceinline__ bool place_row(const RopeParams &p, int row, RowSegment &c, RopeSlot &slot, long long &place, int lane) {
    if (c.shared || !(c.sg.q0 <= row && (long long)row < (long long)c.sg.q0 + c.sg.ql)) {
        c.shared = false;
        if (CACHE == kFp4 && p.S <= 32) {  // a lane has a segment: one load answers both questions
            const Segment o = load_segment(p.seq_info, min(lane, p.S - 1));
            const unsigned m = __ballot_sync(0xffffffffu, lane < p.S && holds_row(p, o, row));
            if (!m) {
                c.sg.ql = 0;
                return false;
            }
            const int s = __ffs(m) - 1;
            c.sg.q0 = __shfl_sync(0xffffffffu, o.q0, s);
            c.sg.ql = __shfl_sync(0xffffffffu, o.ql, s);
            c.sg.col = __shfl_sync(0xffffffffu, o.col, s);
            c.sg.kend = __shfl_sync(0xffffffffu, o.kend, s);
            c.shared = __any_sync(0xffffffffu, lane < p.S && lane != s && overlap(o, c.sg));
        } else {
            const int s = segment_of_row(p, row, lane);
            if (s < 0) {
                c.sg.ql = 0;
                return false;
            }
            c.sg = load_segment(p.seq_info, s);
            if (CACHE == kFp4 && c.may_share) c.shared = shares_rows(p, c.sg, s, lane);
        }
        if (c.shared) {
            c.pages_ok = false;
#pragma unroll 1
            for (c.s = next_segment(p, row, 0, lane); c.s >= 0 && !c.pages_ok;) {
                c.sg = load_segment(p.seq_info, c.s);
                c.pages_ok = ask_pages(p, c.sg, lane);
                if (!c.pages_ok) c.s = next_segment(p, row, c.s + 1, lane);
            }
        } else {
            c.pages_ok = ask_pages(p, c.sg, lane);
        }
    }
    if (!c.pages_ok) return false;
    locate_row(p, c.sg, row, slot, place);
    return true;
}

// Cosine and sine (times mscale) of position `pos` at a pair of `turn`.
__device__ __forceinline__ float2 angle_of(unsigned pos, unsigned long long turn, float mscale) {
    const unsigned f = pos * (unsigned)(turn >> 32) + __umulhi(pos, (unsigned)turn) -
                       ((int)pos < 0 ? (unsigned)turn : 0u);  // (pos mod 2^64) * turn, bits 32..63
    float si, co;
    sincospif((float)(int)f * 4.656612873077393e-10f, &si, &co);  // 2^-31: half turns in [-1, 1]
    return make_float2(co * mscale, si * mscale);
}

// The heads of one row that groups [f0, f1) name (q, then k, then v), from
// `rows[kind]` (global or shared memory); angles: the row's pairs.
struct RopeWork {
    int f0, f1, nq, nk, all;   // groups of heads: this warp's, and of each kind
    unsigned turned;           // columns of this lane that are rotated
    int partner;               // lane of the partner columns (by shuffle)
};
template <typename T, int CACHE, int PAIR>
__device__ __forceinline__ void rope_row(const RopeParams &p, int row, const RopeSlot &slot, const float2 *angles, const T *const (&rows)[3],
                                         const RopeWork &w, float *stage, int lane) {
    const int per = 1 << p.lanes_log2, c = lane & (per - 1), half = p.rot_dim / 2, heads = 32 >> p.lanes_log2;
    int first = 0;
#pragma unroll 1
    for (int kind = 0; kind < (CACHE == kSameType ? 3 : 2); ++kind) {  // q, k, v
        const int H = kind == 0 ? p.Hq : p.Hkv, groups = kind == 0 ? w.nq : kind == 1 ? w.nk : w.all - w.nq - w.nk;
        const int h0 = max(w.f0 - first, 0) * heads, h1 = min(max(w.f1 - first, 0) * heads, H);
        first += groups;
        if (groups == 0 || h0 >= h1) continue;
        const T *src = kind == 0 ? rows[0] : kind == 1 ? rows[1] : rows[2];
        T *dst = reinterpret_cast<T *>(kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out);
        if (dst) dst += row * (kind == 0 ? p.q_out_stride : kind == 1 ? p.k_out_stride : p.v_out_stride);
        unsigned char *pool = reinterpret_cast<unsigned char *>(kind == 0 ? nullptr : kind == 1 ? p.k_pool : p.v_pool);
        const T *weight = reinterpret_cast<const T *>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
        // this lane's columns: cosine and signed sine, then the head weights
        const bool turn = kind < 2 && p.rot_dim > 0;
        float ca[8], sb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ca[e] = 1.f;
            sb[e] = 0.f;
        }
        if (turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = c * 8 + e, i = PAIR == kInLane ? d / 2 : d < half ? d : d - half;
                if (w.turned >> e & 1u) {
                    const float2 t = angles[i];
                    ca[e] = t.x;
                    sb[e] = (PAIR == kInLane ? e & 1 : d >= half) ? t.y : -t.y;
                }
            }
        }
        if (weight) {
            Raw8<T> r;
            r.clear();
            if (c * 8 < p.D) r.load(weight + c * 8);
            float wt[8], wz[8];  // the columns' weights, and their partners'
            r.get(wt);
            if constexpr (PAIR == kInLane) {
#pragma unroll
                for (int e = 0; e < 8; ++e) wz[e] = wt[e ^ 1];
            } else if constexpr (PAIR == kByShuffle) {
#pragma unroll
                for (int e = 0; e < 8; ++e) wz[e] = __shfl_sync(0xffffffffu, wt[e], w.partner);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = c * 8 + e, o = d < half ? d + half : d - half;
                    wz[e] = 1.f;
                    if (w.turned >> e & 1u) {
                        if constexpr (sizeof(T) == 2) wz[e] = __bfloat162float(weight[o]);
                        else wz[e] = weight[o];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ca[e] *= wt[e];
                sb[e] *= wz[e];
            }
        }
        rope_heads<T, CACHE, PAIR>(p, src, dst, pool, slot, h0, h1, ca, sb, weight != nullptr, turn, w.turned, w.partner,
                                   stage, lane);
    }
}

// Part `slice` of `slices` of a row's groups of heads (q, then k, then v, cut evenly).
template <int CACHE, int PAIR>
__device__ __forceinline__ RopeWork rope_work(const RopeParams &p, int slice, int slices, int lane) {
    const int per = 1 << p.lanes_log2, c = lane & (per - 1), half = p.rot_dim / 2, heads = 32 >> p.lanes_log2;
    RopeWork w;
    w.partner = lane;
    if (PAIR == kByShuffle && c < half / 4) w.partner = lane + (c < half / 8 ? half / 8 : -(half / 8));  // the halves are whole lanes
    const int left = p.rot_dim - c * 8;  // rotated columns from this lane's first on
    w.turned = left >= 8 ? 0xffu : left <= 0 ? 0u : (1u << left) - 1u;
    w.nq = p.q ? (p.Hq + heads - 1) / heads : 0;
    w.nk = p.k ? (p.Hkv + heads - 1) / heads : 0;
    w.all = w.nq + w.nk + (CACHE == kSameType ? (p.Hkv + heads - 1) / heads : 0);
    w.f0 = (int)((long long)w.all * slice / slices);
    w.f1 = (int)((long long)w.all * (slice + 1) / slices);
    return w;
}

// The K heads of this warp's part of a row, as they are in the slot `from` of
// segment s, to the row's slots in the segments after it.  (A lane copies what it wrote.)
static __device__ __noinline__ void copy_k4_to_others(const RopeParams &p, int row, int s, RopeSlot from, int f0, int f1, int nq, int lane) {
    const int per = 1 << p.lanes_log2, sub = lane >> p.lanes_log2, c = lane & (per - 1), heads = 32 >> p.lanes_log2, block = block4_bytes(p.D);
    const int h0 = max(f0 - nq, 0) * heads, h1 = min(max(f1 - nq, 0) * heads, p.Hkv);
    unsigned char *pool = reinterpret_cast<unsigned char *>(p.k_pool);
    for (s = next_segment(p, row, s + 1, lane); s >= 0; s = next_segment(p, row, s + 1, lane)) {
        const Segment sg = load_segment(p.seq_info, s);
        if (!ask_pages(p, sg, lane)) continue;
        RopeSlot to;
        long long place;
        locate_row(p, sg, row, to, place);
        for (int h = h0 + sub; h < h1; h += heads) {  // D is a power of two: every lane has columns
            const unsigned char *a = pool + (from.block * p.Hkv + h) * block;
            unsigned char *b = pool + (to.block * p.Hkv + h) * block;
            *reinterpret_cast<unsigned *>(b + to.token * (p.D / 2) + c * 4) = *reinterpret_cast<const unsigned *>(a + from.token * (p.D / 2) + c * 4);
            if ((c & 1) == 0) b[8 * p.D + to.token * (p.D / 16) + c / 2] = a[8 * p.D + from.token * (p.D / 16) + c / 2];
        }
    }
}

// Write the 4-bit V page `pb` of kv head h from the segment's new rows.
template <int D>
__device__ __forceinline__ void write_v4_page(const RopeParams &p, const Segment &sg, int h, int pb, unsigned char *codes,
                                              unsigned char *scales, int lane) {
    constexpr int L = D / 8, TPI = 32 / L;  // lanes a row, rows at once
    const int start = sg.kend - sg.ql, sub = lane / L, c = lane % L;
    const int a = max(start - pb * kPage, 0), b = min(sg.kend - pb * kPage, kPage);  // new tokens of the page
    const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(p.v);
    __syncwarp();
    constexpr int B = 16 / TPI < 8 ? 16 / TPI : 8;  // rows of the lane that are loaded together
#pragma unroll 1
    for (int tb = 0; tb < kPage; tb += B * TPI) {
        Raw8<__nv_bfloat16> x[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int tok = tb + i * TPI + sub;
            x[i].clear();
            if (tok >= a && tok < b) x[i].load(v + ((long long)sg.q0 + (pb * kPage + tok - start)) * p.v_stride + h * D + c * 8);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int t0 = tb + i * TPI, tok = t0 + sub;
            if (t0 + TPI <= a || t0 >= b) continue;  // uniform
            const bool mine = tok >= a && tok < b;
            unsigned scale;
            const unsigned w = quantise8(x[i], scale, p.v_out != nullptr);
            if (mine) {
                // one code a byte, for the exchange below
                const unsigned lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
                *reinterpret_cast<uint2 *>(codes + tok * D + c * 8) =
                    make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
                if ((c & 1) == 0) scales[tok * (D / 16) + c / 2] = (unsigned char)scale;
                if (p.v_out)
                    x[i].store(reinterpret_cast<__nv_bfloat16 *>(p.v_out) + ((long long)sg.q0 + (pb * kPage + tok - start)) * p.v_out_stride + h * D + c * 8);
            }
        }
    }
    __syncwarp();
    const long long blk = p.block_table[(long long)sg.col * p.mbps + table_page(pb, p.ring_rows)];
    unsigned char *out = reinterpret_cast<unsigned char *>(p.v_pool) + (blk * p.Hkv + h) * block4_bytes(D);
    const int g = lane >> 2, t = lane & 3;
    auto fresh = [&](int tok) { return tok >= a && tok < b; };
    const unsigned m0 = (fresh(2 * t) ? 0x0fu : 0u) | (fresh(2 * t + 1) ? 0xf0u : 0u);
    const unsigned m1 = (fresh(2 * t + 8) ? 0x0fu : 0u) | (fresh(2 * t + 9) ? 0xf0u : 0u);
    const unsigned mask = (m0 | m1 << 8) * 0x10001u;
    if (mask) {
#pragma unroll
        for (int pl = 0; pl < D / 64; ++pl) {
            auto pair = [&](int tok) {  // tokens tok and tok + 1 of 8 columns, one byte a column
                const unsigned char *s = codes + tok * D + g * (D / 8) + pl * 8;
                const uint2 lo = *reinterpret_cast<const uint2 *>(s), hi = *reinterpret_cast<const uint2 *>(s + D);
                return make_uint2((lo.x & 0x0f0f0f0fu) | (hi.x & 0x0f0f0f0fu) << 4, (lo.y & 0x0f0f0f0fu) | (hi.y & 0x0f0f0f0fu) << 4);
            };
            const uint2 x = pair(2 * t), y = pair(2 * t + 8);
            uint4 w = make_uint4(__byte_perm(x.x, y.x, 0x5140), __byte_perm(x.x, y.x, 0x7362),
                                 __byte_perm(x.y, y.y, 0x5140), __byte_perm(x.y, y.y, 0x7362));
            uint4 *d = reinterpret_cast<uint4 *>(out + pl * 512 + lane * 16);
            if (mask == 0xffffffffu) {
                *d = w;
            } else {
                // Other tokens of the page may be written at the same time (a
                // ring's last page is its first one too, another segment goes
                // on in the page): only these tokens' bits are cleared and set.  The same
                // segment twice, as padded batches have it, still leaves its values.
                atomicAnd(&d->x, ~mask); atomicOr(&d->x, w.x & mask);
                atomicAnd(&d->y, ~mask); atomicOr(&d->y, w.y & mask);
                atomicAnd(&d->z, ~mask); atomicOr(&d->z, w.z & mask);
                atomicAnd(&d->w, ~mask); atomicOr(&d->w, w.w & mask);
            }
        }
    }
    for (int i = lane; i < (b - a) * (D / 16); i += 32) {
        const int tok = a + i / (D / 16), G = i % (D / 16);
        out[8 * D + (G * 4 + (tok % 8) / 2) * 4 + (tok / 8) * 2 + (tok & 1)] = scales[tok * (D / 16) + G];
    }
}

// The V pages of one (segment, kv head, page warp) unit, page warps fastest.
__device__ __forceinline__ void write_v4_pages(const RopeParams &p, long long unit, unsigned char *codes, int lane) {
    const int pw = (int)(unit % p.page_warps), h = (int)(unit / p.page_warps % p.Hkv);
    const long long s = unit / p.page_warps / p.Hkv;
    if (s >= p.S) return;
    const Segment sg = load_segment(p.seq_info, (int)s);
    if (segment_fault(sg, p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window) || sg.ql == 0) return;
    if (!new_pages_ok(p, sg, lane)) return;
    unsigned char *scales = codes + kPage * p.D;
    const int p1 = (sg.kend + kPage - 1) / kPage;
    for (int pb = (sg.kend - sg.ql) / kPage + pw; pb < p1; pb += p.page_warps) {
        if (p.D == 64) write_v4_page<64>(p, sg, h, pb, codes, scales, lane);
        else if (p.D == 128) write_v4_page<128>(p, sg, h, pb, codes, scales, lane);
        else write_v4_page<256>(p, sg, h, pb, codes, scales, lane);
    }
}
// The errors of the refused segments (one CTA).
__device__ __forceinline__ void report_segments(const RopeParams &p) {
    for (int s = threadIdx.x; s < p.S; s += blockDim.x) {
        const unsigned f = segment_fault(load_segment(p.seq_info, s), p.rows, p.max_seqs, p.mbps, p.ring_rows, p.window);
        if (f) atomicOr(p.err, f);
    }
}

template <typename T, int CACHE, int PAIR>
__global__ void __launch_bounds__(kRopeWarps * 32, sizeof(T) == 2 ? 5 : 4) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (CACHE == kFp4 && (int)blockIdx.x >= p.row_ctas) {
        write_v4_pages(p, (long long)(blockIdx.x - p.row_ctas) * kRopeWarps + warp, smem + (size_t)warp * kPage * (p.D + p.D / 16), lane);
        return;
    }
    RowSegment seg;
    if (CACHE == kFp4) seg.may_share = may_share_rows(p);
    if (CACHE != kNoCache && blockIdx.x == 0) report_segments(p);
    // Few rows: `slices` warps share a row's heads.  Many: a warp takes rows of
    // its own, one after the other, and looks their segment up once.
    const long long w = (long long)blockIdx.x * kRopeWarps + warp;
    const int slice = (int)(w % p.slices);
    const long long warps = (long long)p.row_ctas * kRopeWarps / p.slices, wr = w / p.slices;
    if (wr >= warps) return;
    const int row0 = (int)(wr * p.rows / warps), row1 = (int)((wr + 1) * p.rows / warps);
    float2 *angles = reinterpret_cast<float2 *>(smem) + warp * 128;                       // cosine and sine of each pair
    float *stage = reinterpret_cast<float *>(smem) + kRopeWarps * 256 + warp * 256;
    const RopeWork work = rope_work<CACHE, PAIR>(p, slice, p.slices, lane);
#pragma unroll 1
    for (int row = row0; row < row1; ++row) {
        RopeSlot slot{0, 0};
        long long place = 0;
        if (CACHE != kNoCache && !place_row<CACHE>(p, row, seg, slot, place, lane)) continue;
        if (p.rot_dim) {
            __syncwarp();
            const unsigned pos = (unsigned)(p.positions ? p.positions[row] : (int)place);
            for (int i = lane; i < p.rot_dim / 2; i += 32) angles[i] = angle_of(pos, p.turns[i], p.mscale);
            __syncwarp();
        }
        const T *const rows[3] = {reinterpret_cast<const T *>(p.q) + row * p.q_stride, reinterpret_cast<const T *>(p.k) + row * p.k_stride,
                                  reinterpret_cast<const T *>(p.v) + row * p.v_stride};
        rope_row<T, CACHE, PAIR>(p, row, slot, angles, rows, work, stage, lane);
        if (CACHE == kFp4 && seg.shared) copy_k4_to_others(p, row, seg.s, slot, work.f0, work.f1, work.nq, lane);
    }
}

}  // namespace pkv
