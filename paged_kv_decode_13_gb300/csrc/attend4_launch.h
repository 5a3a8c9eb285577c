// Host-side view of the 4-bit attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <stddef.h>

#include "common.cuh"

namespace pkv {

// Everything one launch reads; passed by value as a grid constant.
struct Attend4Params {
    const unsigned char *k, *v;   // this layer's pools, [num_blocks][Hkv][9 D]
    const __nv_bfloat16 *q;       // [rows][Hq][D]
    const int *block_table;       // [max_seqs][mbps]
    const int4 *seq_info;         // [S]
    const int *first_valid;       // [max_seqs] or null
    void *out;                    // [rows][Hq][D], fp32 or bf16
    float *lse;                   // [rows][Hq] or null
    unsigned *err;
    long long num_blocks;
    int Hq, Hkv, G;
    int total_rows, S, max_seqs, mbps, ring_rows, max_q_len;
    int row_tiles;                // CTAs along the rows of one (segment, kv head)
    int min_pages;                // pages of a range worth a CTA of the cluster
    int causal, window, out_bf16;
    int early;                    // PKV_FLAG_PDL: the tables and old pages may be read before the dependency wait
    float scale_log2;             // softmax scale * log2(e)
    // equal shares (balance4_kernel)
    int piece_pages;              // what a piece of a range costs besides its pages, in pages
    // what shared ranges leave for the merge
    int4 *ws_head;                // [2 N] (first row, kv head | tile << 16, last CTA, 1 | flags << 1 | rows << 4); w = 0: no piece
    float2 *ws_stat;              // [2 N][R] (max, sum)
    float *ws_part;               // [2 N][R][D]
};

constexpr int kMerge4Threads = 256;
constexpr int kMerge4Slots = 2048;  // CTAs of a wave, at most

struct Attend4Kernel {
    const void *fn;
    const void *balance, *merge;  // equal shares and their merge
    int threads;
    size_t smem;
    int rows;   // query rows of a CTA
    int warps;
    int ctas;   // CTAs an SM holds
    int page_ns;  // what a CTA alone on its SM takes for a page of its range, and
    int full;     // what it takes on a full one, in 1 / 20 of that (both measured)
    int regs;   // registers a thread the kernel has to be launched with (it hands them between its warps), or 0
};

// The kernel for head_dim D and at most `rows` query rows a (segment, kv head);
// few: there are few ranges, and a CTA has twice the warps.
Attend4Kernel pick4_64(int rows, bool few);
Attend4Kernel pick4_128(int rows, bool few);
Attend4Kernel pick4_256(int rows, bool few);
// The tcgen05 kernel of wide groups (head_dim 128, equal shares only: fn is null).
Attend4Kernel pick4_wide();

}  // namespace pkv
