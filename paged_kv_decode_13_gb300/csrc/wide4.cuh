// Tensor-core (tcgen05) attention over a quantised cache (4 or 8 bits) for wide
// query groups (sm_103a, head_dim 128).
//
// The row class of draft verification and chunked steps: 128 query rows of
// one (segment, kv head) against its pages, as equal shares of all ranges
// (Share4: one CTA an SM, several pieces each, merge4_kernel after it).  The
// mma.sync tile dequantises a page once for every 32 rows and is bound by the
// warps' own matrix instructions; here a page is dequantised once for 128 rows
// into shared memory and tcgen05.mma takes it from there.
//
// Per CTA (640 threads; the softmax warpgroups take registers from the others), the roles meeting on mbarriers only, so that each
// runs ahead across pieces:
//   warp 18     bulk copies of the raw page blocks, a ring of NR groups of 4
//               pages (a dequantising warp that issued its own waited for the
//               issue: 420 of 2000 cycles a group);
//   warps 8-11, page u = warp % 4 of every group: K (the first four) and V (the
//   12-15       others) as fp16 (exact) into the group's operand tiles, in an
//               order that keeps both the reads (fp4.cuh) and the swizzled
//               writes wide and off each other's banks: token 8 hi + 2 t + n
//               of a page sits at 4 t + 2 hi + n, V column 16 g + i at row
//               8 i + turn(g);
//   warp 16     S(j) = Q K_j^T (M 128, N 64, K 128), Q from TMEM (from shared memory its
//               reads met the dequantising warps' traffic: 89 us of 8-bit drafts
//               against 86 then), K from shared memory, into one of NB buffers of TMEM;
//   warps 0-7   softmax: row t belongs to warps t / 32 and t / 32 + 4, each with
//               32 of a group's 64 keys, its own running maximum and sum and
//               its own O, as in the bf16 tile; P (fp16) over the S columns read;
//               at a piece's end they combine the halves and write the rows,
//               or leave them for the merge;
//   warp 17     O_h += P_h(j) V_j (A from TMEM, K-major V^T, N 128).
//
// 16 sequences of up to 8192 keys, 8 kv heads, up to 128 rows each: 65 us with
// the merge, where the bytes take 12 us, the products (of full tiles) at the
// measured bf16 rate 19, and the mma.sync tiles 179; in 8 bits 84, the bytes 22 (halves of a lane's
// two pieces exchanged as codes and masked only in edge pages: 86.5 before).  In 8 bits the tensor cores are 21 %
// busy, the schedulers 45 %, HBM 28 %: nothing is full, a group's chain of copy, conversion, scores,
// softmax and product is waited for, and so is the change from piece to piece.  Registers 128 / 72 (136 / 64 and 144 / 64: the same time), and a
// piece counted as 36 pages (10: 82 us, 24: 73) in the shares.
// All waits are bounded (kWaitNs); a timeout ends every role, the rows not
// written yet read zero, and PKV_ERR_TIMEOUT is set.
#pragma once

#include "attend4.cuh"
#include "verify.cuh"

namespace pkv {

template <int BITS_>
struct Wide4 {
    static constexpr int BITS = BITS_, D = 128, R = 128, kThreads = 640, PG = 4;
    static constexpr int NK = 3, NV = 3, NB = 3, NR = BITS == 4 ? 8 : 7;  // K, V tiles; S / P buffers; raw groups
    static constexpr int NS = 8;                                    // 8 bits: groups whose pages' scales are kept (the copies are 6 ahead of the softmax at most)
    static constexpr int kBlock = BITS == 4 ? block4_bytes(D) : block8_bytes(D), kRaw = 2 * kBlock;
    static constexpr unsigned kTile = 64 * 256;                     // K: two halves of 64 tokens x 64 columns; V^T: 128 columns x 64 tokens
    static constexpr size_t kRawBytes = (size_t)PG * NR * kRaw;
    // registers a thread: at launch, of the softmax warps and of the others while the roles run
    static constexpr int kRegs = 96, kRegsSoftmax = 128, kRegsOthers = 72;
    static constexpr int kBars = 2 * NK + 2 * NV + 3 * NB + 2 + 2 * NR + (BITS == 8 ? NS : 0), kPieces = 16;
    static constexpr size_t kSmem = 1024 + (size_t)(NK + NV) * kTile + kRawBytes + (BITS == 8 ? 8 : 6) * R * 4 + kBars * 8 + (BITS == 8 ? 2 * NS * PG * 4 : 0) + 256;
    static constexpr unsigned kColO = 64 * NB, kColQ = kColO + 256; // O_h at kColO + 128 h; Q as fp16 pairs
    static_assert(kColQ + 64 <= 512, "the columns of TMEM");
    static_assert(kSmem <= 232448, "exceeds the per-CTA shared memory limit");
    static_assert(256 * kRegsSoftmax + 384 * kRegsOthers <= kThreads * kRegs, "the roles' registers fit the launch's");
    static_assert(kBlock % 16 == 0, "copies stay 16-byte aligned");
    static_assert(NR + NV < kPieces, "the copies are ahead of the softmax by fewer pieces than there are flag words");
};

// V^T's row within 8 of column group g: three bits turned, so that the rows of
// four neighbouring groups differ where the swizzle's low bit does not.
__device__ __forceinline__ int v_turn(int g) { return ((g << 1) & 6) | (g >> 2); }

// kind::f16 with fp16 A and B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A place in a ring of N, and the parity of its phase: carried along, as a division between two waits is on the groups' critical path.
template <int N>
struct RingAt {
    int i = 0;
    unsigned phase = 0;
    bool again = false;  // not the first time round
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
            again = true;
        }
    }
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) wide4_kernel(const __grid_constant__ Attend4Params p) {
    constexpr bool k8 = C::BITS == 8;
    constexpr int D = C::D, R = C::R, PG = C::PG, NK = C::NK, NV = C::NV, NB = C::NB, NR = C::NR;
    constexpr int kWarpS = 16, kWarpPv = 17, kWarpRaw = 18;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sK = smem_raw + (-smem_u32(smem_raw) & 1023u);  // pointer arithmetic keeps the shared address space (a cast would lose it)
    unsigned char *sV = sK + (size_t)NK * C::kTile;
    unsigned char *raw = sV + (size_t)NV * C::kTile;                // [NR][PG] raw pages
    float *sQm = reinterpret_cast<float *>(raw + C::kRawBytes);     // [2][R] largest query magnitude of each half
    float *sXm = sQm + 2 * R, *sXl = sXm + 2 * R, *sXu = sXl + 2 * R;  // [2][R] each half's maximum and sum; 8 bits: what its O counts in
    uint64_t *bars = reinterpret_cast<uint64_t *>(k8 ? sXu + 2 * R : sXu);
    uint64_t *k_full = bars, *k_empty = k_full + NK, *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *s_full = v_empty + NV, *p_full = s_full + NB, *pv_done = p_full + NB;
    uint64_t *q_full = pv_done + NB, *drain = q_full + 1, *raw_full = drain + 1, *raw_empty = raw_full + NR;
    uint64_t *sc_full = raw_empty + NR;                             // 8 bits: the scales of group J are in slot J % NS
    unsigned *sWord = reinterpret_cast<unsigned *>(bars + C::kBars);  // [K, V][NS][PG] scale and NaN tokens of the pages
    unsigned *tslot = sWord + (k8 ? 2 * C::NS * PG : 0);
    volatile int *sAbort = reinterpret_cast<volatile int *>(tslot + 1);
    int *sPiece = reinterpret_cast<int *>(tslot + 2);               // [kPieces] flags of piece i % kPieces: 1 bad page, 2 NaN in an edge page's V

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3, cta = blockIdx.x;
    const int quad = warp & 3, half = (warp >> 2) & 1, r = quad * 32 + lane;  // softmax: TMEM lanes, key half, row of the tile

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < C::kBars; ++i) {
            const bool four = (i < NK) || (i >= 2 * NK && i < 2 * NK + NV) ;                                     // k_full, v_full: the dequantising warps
            const bool eight = (bars + i >= p_full && bars + i < p_full + NB) || bars + i == q_full;           // every softmax warp
            mbar_init(bars + i, four ? 4 : eight || bars + i >= raw_full ? 8 : 1);                             // raw_full: two copies a page; raw_empty: both of its readers; sc_full: K and V of each page
        }
        fence_barrier_init();
        *sAbort = 0;
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) sPiece[i] = 0;
    }
    if (warp == kWarpS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = *tslot, lane_off = (unsigned)(32 * quad) << 16;
    depend4(p, false);
    Share4<false> share;
    share.find<C::kThreads>(p, R, reinterpret_cast<long long *>(sQm));
    depend4(p, true);

    // Bounded wait of a whole warp on one phase; false on a timeout, here or in
    // another role.
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

    Piece4 w;
    int tile, from, last, left = 0;
    bool whole, timed_out = false;
    int gbase = 0, issued = 0;  // groups before this piece; of them, copied
    static_assert(NK == NV && NV == NB, "one place serves the tiles and the buffers");
    RingAt<NK> tile3;           // group gbase + j's tiles and buffer
    RingAt<NR> raws;            // and its raw pages
    if (warp >= 8 && warp < 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsOthers));
        // ---------------- raw pages to operand tiles
        const int u = warp & 3;
        const bool is_v = warp >= 12;
#pragma unroll 1
        for (int piece = 0; !timed_out && share.next(p, R, w, tile, from, whole, last); ++piece) {
            const int ngr = (w.pages + PG - 1) / PG;
#pragma unroll 1
            for (int j = 0; j < ngr; ++j, tile3.next(), raws.next()) {
                const int J = gbase + j, ks = tile3.i, vs = tile3.i, rs = raws.i, li = j * PG + u;
                const bool mine = li < w.pages;
                const unsigned char *st = raw + (size_t)(rs * PG + u) * C::kRaw;
                const bool free_now = !tile3.again || mbar_try_wait((is_v ? v_empty : k_empty) + tile3.i, tile3.phase ^ 1);  // (asked before it is needed: an answer takes 110 cycles)
                if (!wait_bar(raw_full + rs, raws.phase)) { timed_out = true; break; }
                auto tile_free = [&] { return __all_sync(0xffffffffu, free_now) || wait_bar((is_v ? v_empty : k_empty) + tile3.i, tile3.phase ^ 1); };
                if constexpr (k8) {
                    // Tokens l / 8 + 4 i, chunk l % 8 of 16 columns (K and V alike: both tiles have a token's columns side by side).
                    // Lanes of the second column half store their two 16-byte pieces the other way round: the writes meet no bank twice.
                    const unsigned char *src = st + (is_v ? C::kBlock : 0);
                    uint4 cw[4];
                    unsigned word = 0;
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int tok = (lane >> 3) + 4 * i;
                            cw[i] = *reinterpret_cast<const uint4 *>(src + tok * D + 16 * place8(tok, lane & 7, D));
                        }
                        word = *reinterpret_cast<const unsigned *>(src + 16 * D);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_empty + rs);
                    // (slot J % NS is free: its group's P V is done before the tile of group J - 3 is)
                    if (!tile_free()) { timed_out = true; break; }
                    if (lane == 0) {
                        sWord[((is_v ? C::NS : 0) + J % C::NS) * PG + u] = word;
                        if (is_v && word >> 16) atomicOr(sPiece + piece % C::kPieces, 2);
                        mbar_arrive(sc_full + J % C::NS);
                    }
                    const int pos0 = (w.page0 + li) * kPage, half64 = (lane >> 2) & 1;
                    unsigned char *tile64 = (is_v ? sV + (size_t)vs * C::kTile : sK + (size_t)ks * C::kTile) + half64 * (64 * 128);
                    if (is_v && !(mine && pos0 >= w.lo_u && pos0 + kPage <= w.hi_u)) {  // keys that no row sees may hold anything
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = pos0 + (lane >> 3) + 4 * i;
                            if (!mine || key < w.lo_u || key >= w.hi_u) cw[i] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (mine || is_v) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = u * 16 + (lane >> 3) + 4 * i, c = 2 * (lane & 3);
                            unsigned x[8];
                            unpack_e4m3x4(x[0], x[1], half64 ? cw[i].z : cw[i].x);
                            unpack_e4m3x4(x[2], x[3], half64 ? cw[i].w : cw[i].y);
                            unpack_e4m3x4(x[4], x[5], half64 ? cw[i].x : cw[i].z);
                            unpack_e4m3x4(x[6], x[7], half64 ? cw[i].y : cw[i].w);
                            *reinterpret_cast<uint4 *>(tile64 + swz_row(row, c + half64)) = make_uint4(x[0], x[1], x[2], x[3]);
                            *reinterpret_cast<uint4 *>(tile64 + swz_row(row, c + (half64 ^ 1))) = make_uint4(x[4], x[5], x[6], x[7]);
                        }
                    }
                    fence_proxy_async();  // the tensor core reads through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(is_v ? v_full + vs : k_full + ks);
                } else if (!is_v) {
                    // K: two tokens a lane, 32 columns each.  The block goes to registers
                    // first: the stores then wait for no load, and the slot is free early.
                    const int swap = (tq >> 1) * 8;  // lanes of the second column half go the other way round: the writes meet no bank twice
                    unsigned kw[2][4], ks0[2], ks1[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {  // tokens g and g + 8
                        const unsigned char *cs = st + (gq + 8 * k) * (D / 2) + tq * (D / 8), *ss = st + 8 * D + (gq + 8 * k) * (D / 16) + tq * (D / 64);
                        const uint2 lo = *reinterpret_cast<const uint2 *>(cs + swap), hi = *reinterpret_cast<const uint2 *>(cs + (swap ^ 8));
                        kw[k][0] = lo.x; kw[k][1] = lo.y; kw[k][2] = hi.x; kw[k][3] = hi.y;
                        ks0[k] = ss[tq >> 1];        // of words 0, 1 as loaded
                        ks1[k] = ss[(tq >> 1) ^ 1];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_empty + rs);
                    if (!tile_free()) { timed_out = true; break; }
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int row = u * 16 + (gq >> 1) * 4 + (gq & 1) + 2 * k;
                            const unsigned s0 = scale4_both(ks0[k]), s1 = scale4_both(ks1[k]);
                            unsigned char *dst = sK + (size_t)ks * C::kTile + (tq >> 1) * (64 * 128) + row * 128;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int c = (tq & 1) * 4 + (i ^ ((tq >> 1) * 2));  // 16-byte chunk of the row
                                unsigned x[4];
                                unpack_e2m1x8(x, kw[k][i]);
                                const unsigned s = i < 2 ? s0 : s1;
                                *reinterpret_cast<uint4 *>(dst + ((c ^ (row & 7)) << 4)) =
                                    make_uint4(hmul2(x[0], s), hmul2(x[1], s), hmul2(x[2], s), hmul2(x[3], s));
                            }
                        }
                    }
                    fence_proxy_async();  // the tensor core reads through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(k_full + ks);
                } else {
                    // V: 16 columns a lane, four tokens each
                    unsigned vw[2][4] = {}, sw = 0;
                    if (mine) {
                        lds_words<4>(vw[0], st + C::kBlock + lane * 16);
                        lds_words<4>(vw[1], st + C::kBlock + 512 + lane * 16);
                        sw = *reinterpret_cast<const unsigned *>(st + C::kBlock + 8 * D + lane * 4);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_empty + rs);
                    const int pos0 = (w.page0 + li) * kPage;
                    if (!mine || !(pos0 >= w.lo_in && pos0 + kPage <= w.hi_in)) {
                        // keys that no row sees read zero, and so does a NaN that only some
                        // rows may see (they are set at the end)
                        unsigned keep = 0, nan = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = pos0 + 2 * tq + (i >> 1) * 8 + (i & 1);
                            const unsigned m = 0xffu << (8 * i);
                            if (mine && key >= w.lo_u && key < w.hi_u) {
                                if ((sw & m) >= (0xf8u << (8 * i))) nan |= m;
                                else keep |= m;
                            }
                        }
                        sw &= keep;
                        if (__any_sync(0xffffffffu, nan != 0) && lane == 0) atomicOr(sPiece + piece % C::kPieces, 2);
                    }
                    if (!tile_free()) { timed_out = true; break; }
                    const unsigned fa = scale4_pair(sw, 0), fb = scale4_pair(sw, 2);
                    unsigned char *dst = sV + (size_t)vs * C::kTile + v_turn(gq) * 128 + (((u * 2 + (tq >> 1)) ^ v_turn(gq)) << 4) + (tq & 1) * 8;
#pragma unroll
                    for (int pl = 0; pl < 2; ++pl) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            unsigned x[4];
                            unpack_e2m1x8(x, vw[pl][k]);
                            const int col = pl * 8 + 2 * k;
                            *reinterpret_cast<uint2 *>(dst + col * 1024) = make_uint2(hmul2(x[0], fa), hmul2(x[1], fb));
                            *reinterpret_cast<uint2 *>(dst + (col + 1) * 1024) = make_uint2(hmul2(x[2], fa), hmul2(x[3], fb));
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_full + vs);
                }
            }
            gbase += ngr;
        }
    } else if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsOthers));
        if (warp == kWarpRaw) {
            // ---------------- raw copies: lane 2 u copies page u's K block, lane 2 u + 1 its V block
#pragma unroll 1
            for (int piece = 0; !timed_out && share.next(p, R, w, tile, from, whole, last); ++piece) {
                const int ngr = (w.pages + PG - 1) / PG;
                const int *bt_row = p.block_table + (long long)w.sg.col * p.mbps;
                const unsigned char *copy_base = ((lane & 1) ? p.v : p.k) + (size_t)w.h * C::kBlock;
                const size_t block_stride = (size_t)p.Hkv * C::kBlock;
                int id_reg = -1;  // page j0 + lane of the window of 32 pages
#pragma unroll 1
                for (int j = 0; j < ngr; ++j, raws.next()) {
                    const int J = gbase + j, rs = raws.i, j0 = j * PG;
                    if ((j0 & 31) == 0) id_reg = j0 + lane < w.pages ? bt_row[table_page(w.page0 + j0 + lane, p.ring_rows)] : -1;
                    const int bid = __shfl_sync(0xffffffffu, id_reg, (j0 + (lane >> 1)) & 31);
                    if (raws.again && !wait_bar(raw_empty + rs, raws.phase ^ 1)) { timed_out = true; break; }
                    if (lane < 2 * PG) {
                        const bool some = j0 + (lane >> 1) < w.pages, ok = (unsigned)bid < (unsigned)p.num_blocks;
                        if (some && ok) {
                            mbar_expect_tx(raw_full + rs, C::kBlock);
                            bulk_load(raw + (size_t)rs * PG * C::kRaw + lane * C::kBlock, copy_base + (unsigned)bid * block_stride, C::kBlock, raw_full + rs);
                        } else {
                            if (some) atomicOr(sPiece + piece % C::kPieces, 1);
                            mbar_arrive(raw_full + rs);
                        }
                    }
                    __syncwarp();
                    issued = J + 1;
                }
                gbase += ngr;
            }
            // copies in flight get a bounded chance to land (all have, unless a wait ran out)
            if (lane == 0)
#pragma unroll 1
                for (int J = max(0, issued - NR); J < issued; ++J)
                    if (!mbar_wait_ns(raw_full + J % NR, (J / NR) & 1)) break;
            __syncwarp();
        } else if (warp == kWarpS) {
            // ---------------- S products
            const uint32_t idesc = umma_idesc_f16(128, 64);
            const unsigned lead = lane == 0, k_first = UmmaDesc(smem_u32(sK), 16).lo;
            int piece = 0;
#pragma unroll 1
            for (; !timed_out && share.next(p, R, w, tile, from, whole, last); ++piece) {
                const int ngr = (w.pages + PG - 1) / PG;
                if (!wait_bar(q_full, piece & 1)) { timed_out = true; break; }
#pragma unroll 1
                for (int j = 0; j < ngr; ++j, tile3.next()) {
                    const int ks = tile3.i, b = tile3.i;
                    const bool read = !tile3.again || mbar_try_wait(pv_done + b, tile3.phase ^ 1);
                    if (!wait_bar(k_full + ks, tile3.phase)) { timed_out = true; break; }
                    // S(J) goes over buffer b, which P V(J - NB) reads P(J - NB) from
                    if (!__all_sync(0xffffffffu, read) && !wait_bar(pv_done + b, tile3.phase ^ 1)) { timed_out = true; break; }
                    tc_fence_after();
                    const unsigned k_lo = k_first + ks * (C::kTile >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_ts(lead, tmem + b * 64, tmem + C::kColQ + k * 8, k_lo + (((k >> 2) * (64 * 128) + (k & 3) * 32) >> 4), idesc, k > 0);
                    umma_commit_by(lead, s_full + b);
                    umma_commit_by(lead, k_empty + ks);
                }
                gbase += ngr;
            }
            if (lane == 0) {  // every product this thread issued has completed before TMEM is freed
                umma_commit(drain);
                mbar_wait_ns(drain, 0);
            }
            __syncwarp();
        } else if (warp == kWarpPv) {
            // ---------------- P V products
            const uint32_t idesc = umma_idesc_f16(128, 128) | (k8 ? 1u << 16 : 0u);  // 8 bits: V with its columns side by side (MN-major)
            const unsigned lead = lane == 0, v_first = UmmaDesc(smem_u32(sV), k8 ? 64 * 128 : 16).lo;
            int done = -1;
#pragma unroll 1
            while (!timed_out && share.next(p, R, w, tile, from, whole, last)) {
                const int ngr = (w.pages + PG - 1) / PG;
#pragma unroll 1
                for (int j = 0; j < ngr; ++j, tile3.next()) {
                    const int J = gbase + j, vs = tile3.i, b = tile3.i;
                    const bool weights = mbar_try_wait(p_full + b, tile3.phase);
                    if (!wait_bar(v_full + vs, tile3.phase)) { timed_out = true; break; }
                    if (!__all_sync(0xffffffffu, weights) && !wait_bar(p_full + b, tile3.phase)) { timed_out = true; break; }
                    tc_fence_after();
                    const unsigned v_lo = v_first + vs * (C::kTile >> 4);
#pragma unroll
                    for (int k = 0; k < PG; ++k) {
                        const int h = k >> 1;  // keys 0-31 -> O_0 (P of half 0), 32-63 -> O_1
                        umma_ts(lead, tmem + C::kColO + h * 128, tmem + b * 64 + h * 32 + (k & 1) * 8, v_lo + (k * (k8 ? 2048 : 32) >> 4), idesc, j > 0 || (k & 1));
                    }
                    umma_commit_by(lead, v_empty + vs);
                    umma_commit_by(lead, pv_done + b);
                    done = J;
                }
                gbase += ngr;
            }
            if (lane == 0 && done >= 0) mbar_wait_ns(pv_done + done % NB, (done / NB) & 1);
            __syncwarp();
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegsSoftmax));
        // ---------------- softmax and the rows' ends.  A warp that has timed out
        // still keeps the others' barriers.
#pragma unroll 1
        for (int piece = 0; share.next(p, R, w, tile, from, whole, last); ++piece) {
            const int ngr = (w.pages + PG - 1) / PG;
            const bool real = r < w.rows;
            const int first = first_valid_of(p.first_valid, w.sg.col);
            // ---- this row's half of the query, brought into fp16's range (and the scale's sign with it)
            float sc;
            {
                const int i = (w.row0 + (real ? r : 0)) / p.G, jh = (w.row0 + (real ? r : 0)) % p.G;
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (((long long)w.sg.q0 + i) * p.Hq + (long long)w.h * p.G + jh) * D + half * 64);
                uint4 qv[8];
                unsigned mx = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    qv[c] = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    const unsigned v[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx = max(mx, max((v[k] << 16) & 0x7fffffffu, v[k] & 0x7fff0000u));
                }
                sQm[half * R + r] = __uint_as_float(mx);
                named_barrier(1, 256);
                mx = max(__float_as_uint(sQm[r]), __float_as_uint(sQm[R + r]));
                const int k2 = mx ? min(141 - (int)(mx >> 23), 100) : 0;
                const float up = copysignf(__uint_as_float((unsigned)(127 + k2) << 23), p.scale_log2);
                // (never 0: a masked score times it has to stay -inf)
                sc = fmaxf(fabsf(p.scale_log2) * __uint_as_float((unsigned)(127 - k2) << 23), 1e-38f);
#pragma unroll
                for (int c = 0; c < 8; c += 4) {  // (the products of the piece before are done: its last S has been read)
                    unsigned v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint4 &y = qv[c + (k >> 2)];
                        const unsigned x = (k & 3) == 0 ? y.x : (k & 3) == 1 ? y.y : (k & 3) == 2 ? y.z : y.w;
                        v[k] = pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
                    }
                    tmem_st16(tmem + lane_off + C::kColQ + half * 32 + c * 4, v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            int lo_r = 0, hi_r = 0;
            if (real) row_key_bounds(w.sg.kend - w.sg.ql + (w.row0 + r) / p.G, w.sg.kend, p.causal, p.window, first, lo_r, hi_r);
            const int hi_k = min(hi_r, (w.page0 + w.pages) * kPage);  // of this piece
            float m = kNoMax, l = 0.f;
            float wref = kNoMax;  // 8 bits: the reference of the weights of the product with V, which O_half counts in (attend4.cuh)
#pragma unroll 1
            for (int j = 0; j < ngr && !timed_out; ++j, tile3.next()) {
                const int J = gbase + j, b = tile3.i;
                // (an mbarrier's answer takes 110 cycles: both are asked before either is looked at)
                const bool scaled = !k8 || mbar_try_wait(sc_full + J % C::NS, (J / C::NS) & 1), there = mbar_try_wait(s_full + b, tile3.phase);
                if (!__all_sync(0xffffffffu, scaled && there) &&
                    ((k8 && !wait_bar(sc_full + J % C::NS, (J / C::NS) & 1)) || !wait_bar(s_full + b, tile3.phase))) { timed_out = true; break; }
                tc_fence_after();
                float x[32];
                tmem_ld32(tmem + lane_off + b * 64 + half * 32, x);
                float f[2] = {sc, sc};           // of the scores of each of the half's two pages
                float ve[2] = {0.f, 0.f};        // 8 bits: log2 of the pages' V scales, -inf: every value is zero
                if constexpr (k8) {
                    const unsigned *kw = sWord + (J % C::NS) * PG + half * 2;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[i] = fmaxf(sc * scale8_value(kw[i] & 0xffu), 1e-38f);
                        const unsigned b8 = kw[C::NS * PG + i] & 0xffu;
                        ve[i] = b8 ? (float)((int)b8 - 127) : -CUDART_INF_F;
                    }
                    if ((kw[0] | kw[1]) >> 16) {  // tokens that hold a NaN
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (kw[k >> 4] >> (16 + (k & 15)) & 1u) x[k] = CUDART_NAN_F;
                    }
                }
                // (unsigned: a group's missing last pages may lie past 2^31)
                const unsigned pos0 = (unsigned)(w.page0 + j * PG) * kPage + half * 32, lo_u = lo_r, hi_u = hi_k;
                // Key bounds per score only where some real row of the warp does not see all 32.
                if (!__all_sync(0xffffffffu, !real || (pos0 >= lo_u && pos0 + 32 <= hi_u))) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const unsigned pos = k8 ? pos0 + k : pos0 + (k & 16) + 2 * ((k & 15) >> 2) + (k & 1) + 8 * ((k >> 1) & 1);  // the token at column k
                        if (pos < lo_u || pos >= hi_u) x[k] = -CUDART_INF_F;
                    }
                }
                float mx, wx = 0.f;  // wx, 8 bits: the largest exponent of a weight of the product
                if constexpr (k8) {  // the pages' maxima each as a tree of three-way maxima
                    float t[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float *y = x + 16 * i;
                        const float a = max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), max3(y[6], y[7], y[8]));
                        t[i] = fmaxf(max3(a, max3(y[9], y[10], y[11]), max3(y[12], y[13], y[14])), y[15]) * f[i];
                    }
                    mx = fmaxf(t[0], t[1]);
                    wx = fmaxf(t[0] + ve[0], t[1] + ve[1]);
                } else {  // row maximum of the 32 scores as a tree of three-way maxima
                    float t[11];
#pragma unroll
                    for (int k = 0; k < 10; ++k) t[k] = max3(x[3 * k], x[3 * k + 1], x[3 * k + 2]);
                    t[10] = fmaxf(x[30], x[31]);
                    const float a = max3(t[0], t[1], t[2]), b3 = max3(t[3], t[4], t[5]), c3 = max3(t[6], t[7], t[8]);
                    mx = max3(max3(a, b3, c3), t[9], t[10]) * sc;
                }
                const bool grow = mx > m + kLazy4, raise = k8 && wx > wref + kLazy4;
                if (__any_sync(0xffffffffu, grow || raise)) {
                    const float m_new = grow ? mx - kLift4 : m, alpha = ex2(m - m_new), w_new = raise ? wx - kLift4 : wref;
                    const float all = k8 ? ex2(wref - w_new) : alpha;
                    if (j > 0 && __any_sync(0xffffffffu, k8 ? raise && wref != kNoMax : grow && m != kNoMax)) {
                        // O_half holds P V up to the group before against the old reference
                        if (!wait_bar(pv_done + (b ? b - 1 : NB - 1), b ? tile3.phase : tile3.phase ^ 1)) { timed_out = true; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            float o[32];
                            tmem_ld32(tmem + lane_off + C::kColO + half * 128 + c0, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= all;
                            tmem_st32(tmem + lane_off + C::kColO + half * 128 + c0, o);
                        }
                    }
                    l *= alpha;
                    m = m_new;
                    wref = w_new;
                }
                unsigned pk[16];
                // 8 bits: a weight of the product is that of the sum times 2^up of its page.  A page whose scale is 2^127 and
                // more above the reference has small weights alone: they are raised by 2^far beforehand.
                float far = 0.f;
                uint64_t fv[2];
                if constexpr (k8) {
                    const float up[2] = {ve[0] + (m - wref), ve[1] + (m - wref)};
                    far = fminf(fmaxf(fmaxf(up[0], up[1]) - 127.f, 0.f), 100.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float v = ex2(fminf(up[i] - far, 127.f));
                        fv[i] = f32x2(v, v);
                    }
                }
                const uint64_t mm2 = f32x2(far - m, far - m);
                uint64_t la = 0, lb = 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float e0, e1;
                    f32x2_split(fma_f32x2(f32x2(x[2 * k], x[2 * k + 1]), f32x2(f[k >> 3], f[k >> 3]), mm2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    if (k & 1) lb = add_f32x2(lb, f32x2(e0, e1));
                    else la = add_f32x2(la, f32x2(e0, e1));
                    if constexpr (k8) f32x2_split(mul_f32x2(f32x2(e0, e1), fv[k >> 3]), e0, e1);
                    pk[k] = pack_f16x2(e0, e1);
                }
                {
                    float l0, l1;
                    f32x2_split(add_f32x2(la, lb), l0, l1);
                    l = k8 ? fmaf(l0 + l1, ex2(-far), l) : l + (l0 + l1);
                }
                // P(j) as fp16 pairs over the first 16 of this half's S columns (read above)
                tmem_st16(tmem + lane_off + b * 64 + half * 32, pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + b);
            }
            gbase += ngr;
            // ---- the piece's end: the last product has landed
            if (!timed_out && !wait_bar(pv_done + (tile3.i ? tile3.i - 1 : NB - 1), tile3.i ? tile3.phase : tile3.phase ^ 1)) timed_out = true;
            tc_fence_after();
            sXm[half * R + r] = m == kNoMax ? (l != l ? 0.f : -CUDART_INF_F) : m;  // a row of NaN scores keeps its NaN sum
            sXl[half * R + r] = l;
            if (k8) sXu[half * R + r] = wref == kNoMax ? 0.f : ex2(wref - m);
            const int flags = *reinterpret_cast<volatile int *>(sPiece + piece % C::kPieces);
            named_barrier(1, 256);
            if (timed_out) continue;
            if (tid == 0) sPiece[piece % C::kPieces] = 0;
            report4(p, flags & 1);
            // the row's two halves against one reference
            const float m0 = sXm[r], m1 = sXm[R + r], M = fmaxf(m0, m1);
            const float w0 = m0 == -CUDART_INF_F ? 0.f : ex2(m0 - M), w1 = m1 == -CUDART_INF_F ? 0.f : ex2(m1 - M);
            const float L = w0 * sXl[r] + w1 * sXl[R + r];
            const float v0 = k8 ? w0 * sXu[r] : w0, v1 = k8 ? w1 * sXu[R + r] : w1;  // of the halves' columns
            // A NaN in V (4 bits: on a page that not every row sees) was left out: the rows that see it get it here.
            unsigned nan = 0;  // bit g: columns 16 g ..
            if (flags & 2)
#pragma unroll 1
                for (int li = 0; li < w.pages; ++li) {
                    const int pos0 = (w.page0 + li) * kPage;
                    const int bid = p.block_table[(long long)w.sg.col * p.mbps + table_page(w.page0 + li, p.ring_rows)];
                    if ((!k8 && pos0 >= w.lo_in && pos0 + kPage <= w.hi_in) || (unsigned)bid >= (unsigned)p.num_blocks) continue;
                    if constexpr (k8) {  // the whole token
                        const unsigned odd = *reinterpret_cast<const unsigned *>(p.v + ((size_t)bid * p.Hkv + w.h) * C::kBlock + 16 * D) >> 16;
                        for (int k = max(lo_r - pos0, 0); k < min(hi_r - pos0, kPage); ++k)
                            if (odd >> k & 1u) nan = 0xffu;
                        continue;
                    }
                    const unsigned char *ss = p.v + ((size_t)bid * p.Hkv + w.h) * C::kBlock + 8 * D;
                    for (int k = max(lo_r - pos0, 0); k < min(hi_r - pos0, kPage); ++k)
                        for (int g = 0; g < 8; ++g)
                            if (ss[(g * 4 + (k & 7) / 2) * 4 + (k >> 3) * 2 + (k & 1)] >= 0xf8u) nan |= 1u << g;
                }
            const int slot = 2 * cta + (from == 0);
            const bool zero = (flags & 1) || L == 0.f;
            const float inv = 1.f / L;
            const long long row = out_row4(p, w, real ? r : 0);
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
                float o[32], o1[32];
                __syncwarp();  // lanes without a row are ahead of the others' stores; the loads are the whole warp's
                tmem_ld32(tmem + lane_off + C::kColO + half * 64 + c0, o);
                tmem_ld32(tmem + lane_off + C::kColO + 128 + half * 64 + c0, o1);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = (w0 != 0.f ? v0 * o[e] : 0.f) + (w1 != 0.f ? v1 * o1[e] : 0.f);
                if (real)
#pragma unroll
                    for (int g = 0; g < 8; ++g) {  // 4 bits: O's column 8 i + turn(g) is V's column 16 g + i
                        const int tg = v_turn(g);
                        float4 v = k8 ? make_float4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]) : make_float4(o[tg], o[8 + tg], o[16 + tg], o[24 + tg]);
                        if (nan >> g & 1u) v = make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F);
                        const int d = k8 ? half * 64 + c0 + 4 * g : g * 16 + half * 8 + c0 / 8;
                        if (whole)
                            store_out4(p, row * D + d, zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                        else
                            *reinterpret_cast<float4 *>(p.ws_part + ((size_t)slot * R + r) * D + d) = v;
                    }
            }
            if (whole) {
                if (half == 0 && real && p.lse) p.lse[row] = zero ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
            } else {
                left |= 1 << (from == 0);
                if (half == 0 && real) p.ws_stat[(size_t)slot * R + r] = make_float2(M, L);
                if (tid == 0) p.ws_head[slot] = head4(w, tile, last, flags & 1);
            }
            tc_fence_before();  // O is read: the next piece's first product may overwrite it
        }
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegs));
    }
    tc_fence_before();
    // The others take their registers back only here, after the softmax warps
    // have given theirs up: a role without work would else take them before the
    // softmax warps ever had them, and both would wait.
    __syncthreads();
    if (warp >= 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegs));
    if (warp == kWarpS) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");
    }
    if (*sAbort) {  // every row of the share reads zero, here or in the merge
        share.find<C::kThreads>(p, R, reinterpret_cast<long long *>(sQm));
        left = 0;
#pragma unroll 1
        while (share.next(p, R, w, tile, from, whole, last)) {
            if (whole) {
#pragma unroll 1
                for (int i = warp; i < w.rows; i += C::kThreads / 32) {
                    const long long row = out_row4(p, w, i);
                    store_out4(p, row * D + lane * 4, make_float4(0.f, 0.f, 0.f, 0.f));
                    if (lane == 0 && p.lse) p.lse[row] = -CUDART_INF_F;
                }
            } else {
                left |= 1 << (from == 0);
                if (tid == 0) p.ws_head[2 * cta + (from == 0)] = head4(w, tile, last, 2);
            }
        }
        report4(p, 2);
    }
    // slots without a piece (thread 0 is a softmax thread and knows)
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (!(left >> i & 1)) p.ws_head[2 * cta + i].w = 0;
    }
#pragma unroll 1
    for (int i = cta; i < p.S; i += gridDim.x) {  // the refused segments, in turn
        const Segment sg = load_segment(p.seq_info, i);
        const unsigned fault = fault4(p, sg);
        if (fault) refuse4<D>(p, sg, fault, 0, p.Hkv);
    }
    coverage4<D>(p);
}

}  // namespace pkv
