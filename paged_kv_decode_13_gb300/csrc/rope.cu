// Instantiations and launch of the norm + rotary + append kernel.
#include <algorithm>

#include "rope.cuh"
#include "rope_launch.h"

namespace pkv {

template <typename T, int CACHE>
static const void *pick_pair(int pair) {
    switch (pair) {
        case kInLane: return reinterpret_cast<const void *>(&rope_kernel<T, CACHE, kInLane>);
        case kByShuffle: return reinterpret_cast<const void *>(&rope_kernel<T, CACHE, kByShuffle>);
        default: return reinterpret_cast<const void *>(&rope_kernel<T, CACHE, kByShared>);
    }
}

cudaError_t launch_rope(RopeParams &p, int cache, bool f32, int sms, cudaStream_t stream) {
    const int chunks = p.D / 8;
    p.lanes_log2 = 0;
    while ((1 << p.lanes_log2) < chunks) ++p.lanes_log2;
    const int heads = 32 >> p.lanes_log2;  // heads a warp takes at once
    // In the half layout a column's partner is rot_dim / 2 columns away: whole
    // lanes away when that is a multiple of 8, else through shared memory.
    const int pair = p.rot_dim == 0 || p.interleaved ? kInLane : p.rot_dim % 16 == 0 ? kByShuffle : kByShared;
    const auto groups = [&](int H) { return (H + heads - 1) / heads; };
    const int all = std::max(1, (p.q ? groups(p.Hq) : 0) + (p.k ? groups(p.Hkv) : 0) + (cache == kSameType ? groups(p.Hkv) : 0));
    // Few rows: a row's heads are spread over warps until there are about
    // kRopeFill warps an SM.  Many rows: about kRopeFill warps an SM take them
    // in turn, each keeping a row's angles for all its heads.
    const long long fill = (long long)kRopeFill * sms, want = (long long)kRopeSpread * sms / std::max(p.rows, 1);
    p.slices = (int)std::max<long long>(1, std::min<long long>(want, all));
    p.row_ctas = (int)((std::min<long long>(p.rows, std::max<long long>(fill, 1)) * p.slices + kRopeWarps - 1) / kRopeWarps);
    if (cache != kNoCache) p.row_ctas = std::max(p.row_ctas, 1);  // the first looks at the refused segments
    long long ctas = p.row_ctas;
    size_t smem = (size_t)kRopeWarps * 2048;  // angles, exchange
    p.page_warps = 1;
    if (cache == kFp4) {
        // V pages of one (segment, kv head): no more warps than it can have new pages
        const long long units = (long long)p.S * p.Hkv, pages = (p.rows + kPage - 2) / kPage + 1;
        p.page_warps = (int)std::max<long long>(1, std::min(fill / units, pages));
        ctas += (units * p.page_warps + kRopeWarps - 1) / kRopeWarps;
        smem = std::max(smem, (size_t)kRopeWarps * kPage * (p.D + p.D / 16));
    }
    if (ctas == 0) return cudaSuccess;
    const void *fn = cache == kFp4        ? pick_pair<__nv_bfloat16, kFp4>(pair)
                     : cache == kSameType ? (f32 ? pick_pair<float, kSameType>(pair) : pick_pair<__nv_bfloat16, kSameType>(pair))
                                          : (f32 ? pick_pair<float, kNoCache>(pair) : pick_pair<__nv_bfloat16, kNoCache>(pair));
    void *args[] = {&p};
    // Programmatic dependent launch: the kernel waits for the one before it
    // first thing, and only its start overlaps that one's end.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kRopeWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute after;
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &after;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pkv
