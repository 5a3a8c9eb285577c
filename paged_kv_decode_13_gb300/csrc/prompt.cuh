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
// Roles, meeting on mbarriers:
//   softmax warps (four a tile; thread = row)  read S from TMEM, mask, take the
//       maximum, write P = 2^(S - reference) as bf16 over the S columns read,
//       and at the end the normalised rows out.  The reference moves only when a score
//       passes it by 2^8 (then O is rescaled in TMEM; no product is in flight on it then);
//   MMA warp    S = Q K^T (M 128, N 128; Q and K in shared memory) and O += P V (P
//       from TMEM, V as an MN-major tile);
//   copy warp   Q once, then K and V blocks through a ring of stages (TMA, 128-byte
//       swizzle; rows past the tensor and columns past head_dim come as zeros).
// TMEM (512 columns): two S / P slots of 128, then O.  Up to head_dim 128 the two
// slots are the CTA's two tiles, whose softmax and products alternate: each tile's
// next S waits for its own P V, and the tensor core works on the other's meanwhile.
// Above, O of one tile takes 256 columns and the slots are two blocks in turn.
//
// P is rounded to bf16, as V is: half a step, 2^-8 of a weight, on sums
// whose result is rounded the same way or averaged over many keys; the sum of weights is
// taken from the unrounded ones in fp32.
//
// Keys that a row does not see have weight zero, and zero times a NaN or an
// infinity of such a key's V is NaN.  That shows in the row: a CTA that finds a row
// not finite runs its item once more, carefully: V blocks that not every row sees have their
// non-finite values zeroed in shared memory, and the rows that do see
// such a key get its products at the end.  All waits are bounded; a
// timeout ends every role, the rows read zero and PKV_ERR_TIMEOUT is set.
#pragma once

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
    static constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
    static constexpr int kBars = 2 * NST + 1 + 2 + 2 + 2 + 1;
    static constexpr size_t kSmem = 1024 + (size_t)NT * kQTile + (size_t)NST * kStage + kBars * 8 + 64;
    static constexpr unsigned kColO = 256;                          // O of tile t at kColO + t * DP
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
// Rows of no segment read zero, rows of two set PKV_ERR_OVERLAP: one warp of every CTA takes its share of the rows.
__device__ __noinline__ void prompt_coverage(const PromptParams &p, int lane) {
    for (long long row = blockIdx.x; row < p.total_rows; row += gridDim.x) {
        int n = 0;
        for (int s = lane; s < p.S; s += 32) {
            const int4 v = p.seq_info[s];
            n += v.x >= 0 && v.x <= row && row < (long long)v.x + v.y;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (n == 0) prompt_zero(p, row, 0, p.Hq, lane, 32);
        if (n > 1 && lane == 0) atomicOr(p.err, PKV_ERR_OVERLAP);
    }
}
__device__ __forceinline__ bool not_finite(unsigned bf16_pair) { return (bf16_pair & 0x7f80u) == 0x7f80u || (bf16_pair & 0x7f800000u) == 0x7f800000u; }

// Products of the non-finite V values of one key that were zeroed, added to columns c0 .. c0 + 31 of a row.
__device__ __noinline__ void prompt_add_key(const PromptParams &p, long long key_row, long long q_row, int h, int hq, int c0, float m, float (&o)[32]) {
    const __nv_bfloat16 *v = p.v + key_row * p.v_stride + (long long)h * p.D + c0;
    float w = 0.f;
    bool known = false;
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        if (c0 + c >= p.D) break;
        const uint4 x = *reinterpret_cast<const uint4 *>(v + c);
        const unsigned u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!not_finite(u[e])) continue;
            if (!known) {
                float s = 0.f;
                for (int d = 0; d < p.D; ++d)
                    s = fmaf(__bfloat162float(p.q[q_row * p.q_stride + (long long)hq * p.D + d]), __bfloat162float(p.k[key_row * p.k_stride + (long long)h * p.D + d]), s);
                w = exp2_fast(fmaf(s, p.scale_log2, -m));
                known = true;
            }
            const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
            if (!isfinite(lo)) o[c + 2 * e] = fmaf(w, lo, o[c + 2 * e]);
            if (!isfinite(hi)) o[c + 2 * e + 1] = fmaf(w, hi, o[c + 2 * e + 1]);
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    constexpr int DP = C::DP, NT = C::NT, NST = C::NST, SPB = C::SPB;
    constexpr int kWarpMma = C::kSoftmaxWarps, kWarpTma = kWarpMma + 1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sQ = smem_raw + (-smem_u32(smem_raw) & 1023u);  // pointer arithmetic keeps the shared address space
    unsigned char *ring = sQ + NT * C::kQTile;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + (size_t)NST * C::kStage);
    uint64_t *full = bars, *empty = full + NST, *q_full = empty + NST, *s_full = q_full + 1, *p_full = s_full + 2, *pv_done = p_full + 2, *drain = pv_done + 2;
    unsigned *tslot = reinterpret_cast<unsigned *>(bars + C::kBars);
    volatile int *sAbort = reinterpret_cast<volatile int *>(tslot + 1), *sOdd = sAbort + 1;  // a wait ran out; a row is not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- this CTA's item: the longest (the last tiles) first
    const int per = max(p.S, 1) * p.Hkv, order = blockIdx.x / per, s = blockIdx.x % per / p.Hkv, h = blockIdx.x % p.Hkv;
    const int item = p.items - 1 - order;
    pdl_wait();
    pdl_trigger();
    const Segment sg = p.S ? load_segment(p.seq_info, s) : Segment{0, 0, 0, 0};
    const unsigned fault = p.S ? prompt_fault(p, sg) : 0u;
    const int token0 = item * NT * p.tokens, tokens = min(NT * p.tokens, sg.ql - token0);  // of this item
    if (fault || tokens <= 0) {
        if (fault && item == 0) {
            if (tid == 0) atomicOr(p.err, fault);
            if (sg.q0 >= 0)  // a negative q_start covers nothing
                for (long long r = sg.q0; r < min((long long)sg.q0 + sg.ql, (long long)p.total_rows); ++r)
                    prompt_zero(p, r, h * p.G, p.G, tid, C::kThreads);
        }
        if (warp == kWarpTma) prompt_coverage(p, lane);
        return;
    }
    // keys of each tile: [lo, hi) that some row sees; of the item: [in_lo, in_hi) that every row does
    int first[NT], last[NT];  // blocks of each tile
    int in_lo, in_hi, lo, hi;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int a = token0 + t * p.tokens, b = min(a + p.tokens, sg.ql) - 1;  // tokens of the tile
        first[t] = last[t] = 0;
        if (b >= a) {
            int x;
            row_key_bounds(a, sg.ql, p.causal, p.window, 0, lo, x);
            row_key_bounds(b, sg.ql, p.causal, p.window, 0, x, hi);
            first[t] = lo / C::kKeys;
            last[t] = (hi + C::kKeys - 1) / C::kKeys;
        }
    }
    row_key_bounds(token0, sg.ql, p.causal, p.window, 0, lo, in_hi);
    row_key_bounds(token0 + tokens - 1, sg.ql, p.causal, p.window, 0, in_lo, hi);
    const int b0 = lo / C::kKeys, b1 = (hi + C::kKeys - 1) / C::kKeys;

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < C::kBars; ++i) mbar_init(bars + i, bars + i >= p_full && bars + i < p_full + 2 ? 4 : 1);
        fence_barrier_init();
        *sAbort = 0;
        *sOdd = 0;
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = *tslot;

    // Bounded wait of a whole warp on one phase; false on a timeout, here or in another role.
    auto wait_bar = [&](uint64_t *bar, unsigned parity) -> bool {
        bool ok = mbar_try_wait(bar, parity);
        if (!ok) {
            const unsigned long long t0 = global_ns();
#pragma unroll 1
            while (!ok) {
                ok = mbar_try_wait(bar, parity);
                if (!ok && (*sAbort || global_ns() - t0 > kWaitNs)) break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *sAbort = 1;
        return ok;
    };

    int stages = 0;             // stages used so far
    unsigned uses[2] = {0, 0};  // S / P slots: blocks so far
    bool covered = false;
#pragma unroll 1
    for (int careful = 0; careful < 2; ++careful) {
        const int begin = stages;
        if (warp == kWarpTma) {
            // ---------------- copies
            if (!careful && lane == 0) {
                unsigned bytes = 0;
#pragma unroll
                for (int t = 0; t < NT; ++t) bytes += last[t] > first[t] ? DP / 64 * p.tokens * p.G * 128 : 0;
                mbar_expect_tx(q_full, bytes);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (last[t] > first[t])
                        for (int c = 0; c < DP / 64; ++c)
                            tma_load_3d(sQ + t * C::kQTile + c * C::kPart, &p.tmap_q, q_full, c * 64, h * p.G, sg.q0 + token0 + t * p.tokens);
            }
            __syncwarp();
            bool ok = true;
            auto load = [&](const CUtensorMap *map, int block) {
#pragma unroll 1
                for (int c = 0; ok && c < SPB; ++c) {
                    const int st = stages % NST;
                    if (stages >= NST) ok = wait_bar(empty + st, ((stages / NST) - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_expect_tx(full + st, C::kStage);
#pragma unroll
                        for (int x = 0; x < C::kCols / 64; ++x)
                            tma_load_3d(ring + (size_t)st * C::kStage + x * C::kPart, map, full + st, c * C::kCols + x * 64, h, sg.q0 + block * C::kKeys);
                    }
                    __syncwarp();
                    ++stages;
                }
            };
            load(&p.tmap_k, b0);
#pragma unroll 1
            for (int j = b0; ok && j < b1; ++j) {
                // the order in which the products take them
                if (NT == 1 && j + 1 < b1) load(&p.tmap_k, j + 1);
                load(&p.tmap_v, j);
                if (NT == 2 && j + 1 < b1) load(&p.tmap_k, j + 1);
            }
            if (!ok) {  // copies in flight get a bounded chance to land
                if (lane == 0)
#pragma unroll 1
                    for (int i = max(0, stages - NST); i < stages; ++i)
                        if (!mbar_wait_ns(full + i % NST, (i / NST) & 1)) break;
                __syncwarp();
            }
            if (!covered) prompt_coverage(p, lane);
            covered = true;
        } else if (warp == kWarpMma) {
            // ---------------- products
            const uint32_t id_s = umma_idesc_bf16(128, 128, 0), id_o = umma_idesc_bf16(128, C::kCols, 1);
            const unsigned q_addr = smem_u32(sQ), ring_addr = smem_u32(ring);
            bool ok = careful || wait_bar(q_full, 0);
            auto stage_ready = [&](int i) { return wait_bar(full + i % NST, (i / NST) & 1); };
            // S of tile t and the block whose stages begin at i, into slot
            auto issue_s = [&](int t, int i, int slot) {
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        const unsigned k_addr = ring_addr + (unsigned)((i + k / (C::kCols / 16)) % NST) * C::kStage;
                        umma_bf16(tmem + slot * 128, umma_desc(q_addr + t * C::kQTile + (k >> 2) * C::kPart + (k & 3) * 32, 16, 1024),
                                  umma_desc(k_addr + (k % (C::kCols / 16) >> 2) * C::kPart + (k & 3) * 32, 16, 1024), id_s, k > 0 ? 1 : 0);
                    }
                    umma_commit(s_full + slot);
                }
                __syncwarp();
            };
            // O of tile t += P in slot times the V block whose stages begin at i
            auto issue_pv = [&](int t, int i, int slot, bool fresh) {
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < SPB; ++c) {
                        const unsigned v_addr = ring_addr + (unsigned)((i + c) % NST) * C::kStage;
#pragma unroll
                        for (int u = 0; u < C::kKeys / 16; ++u)
                            umma_bf16_ts(tmem + C::kColO + t * DP + c * C::kCols, tmem + slot * 128 + u * 8, umma_desc(v_addr + u * 2048, C::kPart, 1024),
                                         id_o, (!fresh || u > 0) ? 1 : 0);
                    }
                    umma_commit(pv_done + slot);
                }
                __syncwarp();
                ++uses[slot];
            };
            auto release = [&](int i) {  // once what has been issued so far is done
                if (lane == 0)
#pragma unroll
                    for (int c = 0; c < SPB; ++c) umma_commit(empty + (i + c) % NST);
                __syncwarp();
            };
            auto block_ready = [&](int i) {
                bool r = true;
                for (int c = 0; r && c < SPB; ++c) r = stage_ready(i + c);
                return r;
            };
            ok = ok && block_ready(stages);
            if (ok) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (b0 >= first[t] && b0 < last[t]) issue_s(t, stages, t);
                release(stages);
            }
            stages += SPB;
#pragma unroll 1
            for (int j = b0; ok && j < b1; ++j) {
                const bool more = j + 1 < b1;
                if constexpr (NT == 2) {
                    const int v = stages, k = stages + SPB;
                    ok = block_ready(v);
                    bool k_ready = false;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const bool here = j >= first[t] && j < last[t], next = more && j + 1 >= first[t] && j + 1 < last[t];
                        if (ok && here) {
                            ok = wait_bar(p_full + t, uses[t] & 1);
                            if (ok) issue_pv(t, v, t, j == first[t]);
                        }
                        if (ok && next) {
                            if (!k_ready) ok = block_ready(k);
                            k_ready = true;
                            if (ok && here) ok = wait_bar(pv_done + t, (uses[t] - 1) & 1);  // P is read: S may go over it
                            if (ok) issue_s(t, k, t);
                        }
                    }
                    if (ok) {
                        release(v);
                        if (more) release(k);
                    }
                    stages += more ? 2 * SPB : SPB;
                } else {
                    const int slot = (j - b0) & 1;
                    if (more) {
                        ok = block_ready(stages);
                        if (ok && j > b0) ok = wait_bar(pv_done + (slot ^ 1), (uses[slot ^ 1] - 1) & 1);
                        if (ok) {
                            issue_s(0, stages, slot ^ 1);
                            release(stages);
                        }
                        stages += SPB;
                    }
                    ok = ok && block_ready(stages) && wait_bar(p_full + slot, uses[slot] & 1);
                    if (ok) {
                        issue_pv(0, stages, slot, j == b0);
                        release(stages);
                    }
                    stages += SPB;
                }
            }
            if (!ok && lane == 0) {  // every product issued has completed before TMEM is freed
                umma_commit(drain);
                mbar_wait_ns(drain, 0);
            }
            __syncwarp();
        } else {
            // ---------------- softmax
            const int t = warp >> 2, r = tid & 127;  // tile, row of it
            const unsigned lane_off = (unsigned)(32 * (warp & 3)) << 16;
            const int token = token0 + t * p.tokens + r / p.G;
            const bool real = r < p.tokens * p.G && token < sg.ql;
            int lo_r = 0, hi_r = 0;
            if (real) row_key_bounds(token, sg.ql, p.causal, p.window, 0, lo_r, hi_r);
            const float sc = p.scale_log2;
            float m = kNoScore, l = 0.f;
            bool ok = true;
            const int f = NT == 2 ? first[t] : b0, e = NT == 2 ? last[t] : b1;
#pragma unroll 1
            for (int j = f; ok && j < e; ++j) {
                const int slot = NT == 2 ? t : (j - b0) & 1;
                const unsigned s_addr = tmem + lane_off + slot * 128;
                if (!(ok = wait_bar(s_full + slot, uses[slot] & 1))) break;
                tc_fence_after();
                unsigned x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(s_addr + 32 * c, x[c]);
                tmem_wait_ld();
                const int pos0 = j * C::kKeys;
                if (!__all_sync(0xffffffffu, !real || (pos0 >= lo_r && pos0 + C::kKeys <= hi_r))) {
                    const int a = lo_r - pos0, b = hi_r - pos0;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k < a || 32 * c + k >= b) x[c][k] = 0xff800000u;
                }
                float mx = -CUDART_INF_F;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float y[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = fmaxf(y[i], __uint_as_float(x[c][k + i]));
                    mx = fmaxf(mx, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
                }
                mx *= sc;
                const bool grow = mx > m + kPromptLazy;
                if (__any_sync(0xffffffffu, grow)) {
                    const float m_new = grow ? mx : m, alpha = exp2_fast(m - m_new);
                    if (j > f && __any_sync(0xffffffffu, grow && m != kNoScore)) {
                        // the product before is done: with two tiles S came after it, with two slots it is waited for
                        if (NT == 1 && !(ok = wait_bar(pv_done + (slot ^ 1), (uses[slot ^ 1] - 1) & 1))) break;
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
                    tmem_st16(s_addr + 16 * c, pk);
                }
                {
                    float l0, l1;
                    f32x2_split(add_f32x2(la, lb), l0, l1);
                    l += l0 + l1;
                }
                if (careful && !(pos0 >= in_lo && pos0 + C::kKeys <= in_hi)) {
                    // V rows that not every row of the item sees: what is not finite reads zero
                    const int i0 = begin + SPB * (NT == 2 ? 2 * (j - b0) + 1 : (min(j + 1, b1 - 1) - b0 + 1) + (j - b0));
                    const int key = pos0 + r;
#pragma unroll 1
                    for (int c = 0; ok && c < SPB; ++c) {
                        ok = wait_bar(full + (i0 + c) % NST, ((i0 + c) / NST) & 1);
                        if (!ok || (key >= in_lo && key < in_hi)) continue;
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
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + slot);
                ++uses[slot];
            }
            // ---- the rows' ends: the last product has landed
            if (e > f) {
                const int slot = NT == 2 ? t : (e - 1 - b0) & 1;
                if (ok) ok = wait_bar(pv_done + slot, (uses[slot] - 1) & 1);
                tc_fence_after();
                const long long row = (long long)sg.q0 + (real ? token : 0);
                const int hq = h * p.G + (real ? r % p.G : 0);
                const bool zero = !ok || l == 0.f;
                const float inv = 1.f / l;
                bool odd = false;
#pragma unroll 1
                for (int c0 = 0; c0 < DP; c0 += 32) {
                    float o[32];
                    tmem_ld32(tmem + lane_off + C::kColO + t * DP + c0, o);
                    if (!real) continue;
                    if (careful) {
                        float y[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) y[k] = o[k];
#pragma unroll 1
                        for (int key = lo_r; key < hi_r; ++key) {
                            if (key >= in_lo && key < in_hi) key = in_hi;  // (those every row sees were not touched)
                            if (key < hi_r) prompt_add_key(p, (long long)sg.q0 + key, row, h, hq, c0, m, y);
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = y[k];
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) sum += o[k] * 0.f;  // NaN where one is not finite
                    odd |= sum != 0.f;
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (c0 + k < p.D)
                            prompt_store4(p, (row * p.Hq + hq) * p.D + c0 + k,
                                          zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[k] * inv, o[k + 1] * inv, o[k + 2] * inv, o[k + 3] * inv));
                }
                if (real && p.lse) p.lse[row * p.Hq + hq] = zero ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
                if (odd && l == l) *sOdd = 1;  // (a NaN sum: its own scores hold one)
                tc_fence_before();
            }
            stages += 2 * SPB * (b1 - b0);
        }
        __syncthreads();
        if (careful || *sAbort || !*sOdd) break;
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");
    }
    if (*sAbort) {  // every row of the item reads zero
        for (int i = warp; i < tokens; i += C::kThreads / 32) prompt_zero(p, (long long)sg.q0 + token0 + i, h * p.G, p.G, lane, 32);
        if (tid == 0) atomicOr(p.err, PKV_ERR_TIMEOUT);
    }
}

}  // namespace pkv
