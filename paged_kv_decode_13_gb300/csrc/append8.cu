// Launch of the append to an 8-bit cache, and reading it back.
#include <algorithm>

#include "append8.cuh"
#include "rope_launch.h"

namespace pkv {

cudaError_t launch_append8(const RopeParams &r, int sms, cudaStream_t stream) {
    Append8Params a;
    a.r = r;
    const bool plain = !r.q && r.rot_dim == 0 && !r.k_weight;
    const int pair = plain ? kPlainRows : r.rot_dim == 0 || r.interleaved ? kInLane : r.rot_dim % 16 == 0 ? kByShuffle : kByShared;
    // A CTA a page that the rows can have at most, up to kAppend8Most an SM (which then take
    // several); with few, a page's heads are spread over CTAs until an SM has kAppend8Fill.
    const long long pages = r.S + ((long long)r.rows + 14ll * std::min(r.S, r.rows)) / kPage + 1;
    a.page_ctas = (int)std::max<long long>(1, std::min(pages, (long long)sms * kAppend8Most));
    const int items = (r.q ? r.Hq : 0) + 2 * r.Hkv;
    const long long active = std::min<long long>(a.page_ctas, r.S + r.rows / kPage);  // CTAs with a page, about
    a.head_ctas = (int)std::max<long long>(1, std::min<long long>((items + kAppend8Warps - 1) / kAppend8Warps, (long long)sms * kAppend8Fill / std::max(active, 1ll)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.page_ctas * a.head_ctas));
    cfg.blockDim = dim3(kAppend8Warps * 32);
    cfg.dynamicSmemBytes = (size_t)kPage * (r.rot_dim / 2) * 8 + (pair == kByShared ? kAppend8Warps * 1024 : 0);
    cfg.stream = stream;
    cudaLaunchAttribute after;  // waits for the kernel before it first thing; only the start overlaps that one's end
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &after;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    const void *fn = r.D == 64 ? pick_append8_64(pair, r.ring_rows) : r.D == 128 ? pick_append8_128(pair, r.ring_rows) : pick_append8_256(pair, r.ring_rows);
    return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t launch_read8(const void *k, const void *v, void *k_out, void *v_out, long long n, int kv_heads, int head_dim, int sms, cudaStream_t stream) {
    Read8Params p;
    p.pool[0] = reinterpret_cast<const unsigned char *>(k);
    p.pool[1] = reinterpret_cast<const unsigned char *>(v);
    p.out[0] = reinterpret_cast<__nv_bfloat16 *>(k_out);
    p.out[1] = reinterpret_cast<__nv_bfloat16 *>(v_out);
    p.n = n;
    p.Hkv = kv_heads;
    p.D = head_dim;
    const long long ctas = std::min<long long>((2 * n * kv_heads * (head_dim / 8) + 255) / 256, (long long)sms * 16);
    read8_kernel<<<(unsigned)ctas, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
