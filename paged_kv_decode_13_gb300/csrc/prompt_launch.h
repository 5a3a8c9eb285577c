// Host-side view of the prompt attention kernel.
#pragma once

#include "common.cuh"

namespace pkv {

// Everything one launch reads; passed by value as a grid constant.
struct PromptParams {
    CUtensorMap tmap_q;           // (D, Hq, rows), box: 64 columns x the group's heads x the tile's tokens
    CUtensorMap tmap_k, tmap_v;   // (D, Hkv, rows), box: 64 columns x 1 head x 128 rows
    const __nv_bfloat16 *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // elements from row to row
    const int4 *seq_info;         // [S]
    void *out;                    // [rows][Hq][D], fp32 or bf16
    float *lse;                   // [rows][Hq] or null
    unsigned *err;
    int Hq, Hkv, G, D, total_rows, S, max_len;
    int tokens;                   // of a tile of 128 query rows: 128 / G
    int units;                    // of a kv head, in the grid: tile groups of all segments, at most
    int causal, window, out_bf16;
    float scale_log2;             // softmax scale * log2(e), positive
};

struct PromptKernel {
    const void *fn;
    int threads;
    size_t smem;
    int tiles;  // query tiles of a CTA
    int regs;   // registers a thread the kernel has to be launched with (it hands them between its warps), or 0
};
// The kernel for head_dim D (a multiple of 8, at most 256).
PromptKernel pick_prompt(int head_dim);

}  // namespace pkv
