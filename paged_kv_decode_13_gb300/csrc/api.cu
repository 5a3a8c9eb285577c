// C-ABI entry points of libpkv: argument checks, launch planning and launches.
// Every entry point validates on the host first and returns a negative
// pkv_status before launching anything; nothing here allocates memory,
// synchronises the host or keeps state beyond kernel attributes and occupancy, per device.
#include <cuda_runtime.h>

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include <math.h>

#include "attend4_launch.h"
#include "kernel_table.h"
#include "launch.h"
#include "misc_kernels.cuh"
#include "prompt_launch.h"
#include "rope_launch.h"

using namespace pkv;

namespace {

constexpr int kDefaultSms = 152;       // GB300, used when no device is visible
constexpr int kTargetWaves = 3;        // split count: about this many waves of resident CTAs
constexpr int kMaxCluster = 16;        // largest thread-block cluster (non-portable size)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(int dtype) { return dtype == PKV_BF16 ? 2 : dtype == PKV_F32 ? 4 : 0; }

// A cache held in 4 or 8 bits.
bool is_quantised(const pkv_cache *c) { return c && (c->dtype == PKV_FP4 || c->dtype == PKV_FP8); }
// Bytes of its page block of one kv head.
int block_bytes(const pkv_cache *c) { return c->dtype == PKV_FP4 ? 9 * c->head_dim : 16 * c->head_dim + 16; }

// quantised: whether the call takes such caches.
int check_cache(const pkv_cache *c, bool quantised = false) {
    if (!c) return PKV_EINVAL;
    if (c->dtype != PKV_BF16 && c->dtype != PKV_F32 && !(quantised && is_quantised(c))) return PKV_EUNSUPPORTED;
    // vLLM-Omni paged_decode_supported: head_dim a multiple of 8, at most 256.
    if (c->head_dim <= 0 || c->head_dim % 8 != 0 || c->head_dim > 256) return PKV_EUNSUPPORTED;
    if (is_quantised(c) && c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return PKV_EUNSUPPORTED;
    if (c->num_layers <= 0 || c->kv_heads <= 0 || c->num_blocks <= 0) return PKV_EINVAL;
    if (c->num_blocks > INT32_MAX || c->kv_heads > 65535) return PKV_EINVAL;
    if (c->max_seqs <= 0 || c->max_blocks_per_seq <= 0) return PKV_EINVAL;
    if (!c->k || !c->v || !c->block_table) return PKV_EINVAL;
    if ((reinterpret_cast<uintptr_t>(c->block_table) & 3u) != 0) return PKV_EINVAL;
    if ((reinterpret_cast<uintptr_t>(c->first_valid) & 3u) != 0) return PKV_EINVAL;
    if (c->ring_rows < 0 || c->ring_rows % PKV_BLOCK_SIZE != 0) return PKV_EINVAL;
    if ((long long)c->ring_rows > (long long)c->max_blocks_per_seq * PKV_BLOCK_SIZE) return PKV_EINVAL;
    return PKV_OK;
}

int check_layer(const pkv_cache *c, int layer) {
    if (layer < 0 || layer >= c->num_layers) return PKV_EINVAL;
    if (!c->k[layer] || !c->v[layer] || !aligned16(c->k[layer]) || !aligned16(c->v[layer])) return PKV_EINVAL;
    return PKV_OK;
}

// Launch plan of one attention call.
struct Plan {
    AttnKernel k;
    int G, rows_max, row_tiles, units, ncta;
    bool gm;  // decode kernel merging its splits through a global workspace (no cluster)
};

constexpr int kMaxSplitsGm = 64;  // splits per key range when merging through global memory

constexpr int kKernelRoom = 512;  // (kernel, device) pairs whose state is kept

// The current device, or -1 when none answers.
int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return dev;
}

// SMs of a device (GB300's count when no device answers).
int device_sms(int dev) {
    static std::atomic<int> known[64];
    int n = 0;
    if (dev < 0) return kDefaultSms;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return kDefaultSms;
    }
    if (dev < 64 && n > 0) known[dev].store(n, std::memory_order_relaxed);
    return n > 0 ? n : kDefaultSms;
}

// Workspace layout of the global merge: partial rows, (max, sum), flags,
// counters, each region 256-byte aligned.
struct WsLayout {
    size_t part, stat, flag, count, total;
};
// The counters come first, at a place that depends only on the unit count.
WsLayout ws_layout(long long units, int ncta, int dp) {
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    WsLayout w;
    w.count = 0;
    w.part = al((size_t)units * 4);
    w.stat = al(w.part + (size_t)units * ncta * 8 * dp * 4);
    w.flag = al(w.stat + (size_t)units * ncta * 8 * 8);
    w.total = al(w.flag + (size_t)units * ncta * 4);
    return w;
}

AttnKernel pick(int variant, int dp, int rc) {
    switch (variant * 1000 + dp) {
        case 64: return pick_0_64(rc);
        case 128: return pick_0_128(rc);
        case 256: return pick_0_256(rc);
        case 1064: return pick_1_64(rc);
        case 1128: return pick_1_128(rc);
        case 1256: return pick_1_256(rc);
        case 2064: return pick_2_64(rc);
        case 2128: return pick_2_128(rc);
        case 2256: return pick_2_256(rc);
    }
    return AttnKernel{nullptr, 0, 0, 0, 0, false, false};
}

// Clusters of c CTAs of this kernel that the current device `dev` holds at once
// (c = 1: resident CTAs); kept per kernel, device and size, 0 when none fits or no
// device answers the query (which is not kept).
int active_clusters(const AttnKernel &k, int c, int dev) {
    struct Counts {
        int n[kMaxCluster + 1];  // one more than the count, 0: not asked
    };
    static std::mutex mu;
    static KernelTable<Counts, kKernelRoom> known;
    if (c < 1 || c > kMaxCluster || dev < 0) return 0;
    std::lock_guard<std::mutex> lock(mu);
    Counts *kept = known.find(k.fn, dev);
    if (!kept) kept = known.add(k.fn, dev, Counts{});
    if (kept && kept->n[c]) return kept->n[c] - 1;
    int clusters = 0;
    cudaError_t e;
    if (c == 1) {
        int per_sm = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k.fn, k.threads, k.smem);
        clusters = per_sm * device_sms(dev);
    } else {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)c, 1, 1);
        cfg.blockDim = dim3((unsigned)k.threads);
        cfg.dynamicSmemBytes = k.smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)c;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters, k.fn, &cfg);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    clusters = std::max(clusters, 0);
    if (kept) kept->n[c] = clusters + 1;
    return clusters;
}

// Largest cluster size <= want that the device can schedule for this kernel
// (1 when no device answers the query).
int schedulable_cluster(const AttnKernel &k, int want, int dev) {
    for (int c = want; c > 1; --c)
        if (active_clusters(k, c, dev) > 0) return c;
    return 1;
}

// Automatic split count of a kernel that fits once per SM.  A key range's
// CTAs form one cluster, and clusters only start where a GPC has that many
// free SMs, so a large cluster size can leave part of the units for a second
// or third wave (16-CTA clusters: seven at a time on GB300's 152 SMs).  The
// time of a launch goes about as waves / cluster size, waves = units over the
// clusters held at once; take the size at or below `want` that minimises it,
// and of equal ones the size with fewer waves (each wave repeats the ramp-up
// and the merge).  The waves run in lock step only when there are few units
// (at most half the resident CTAs), each split across many CTAs; with more
// units of uneven length the split balances the long ranges instead, so
// those launches keep `want`.  Kernels that fit twice per SM keep it too:
// there the second slot holds the next layer's CTAs (programmatic launch),
// which the wave count does not see.
int wave_cluster(const AttnKernel &k, long long units, int want, int dev) {
    const int resident = active_clusters(k, 1, dev);
    if (want <= 1 || units <= 0 || resident > device_sms(dev) || 2 * units > resident) return want;
    auto waves = [&](int c) {
        const long long a = active_clusters(k, c, dev);
        return a > 0 ? (units + a - 1) / a : (long long)1 << 40;
    };
    int best = want;
    long long best_w = waves(want);
    for (int c = want - 1; c >= 1; --c) {
        const long long w = waves(c);
        // w / c against best_w / best, exactly
        const long long lhs = w * best, rhs = best_w * c;
        if (lhs < rhs || (lhs == rhs && w < best_w)) {
            best = c;
            best_w = w;
        }
    }
    return best;
}

int make_plan(const pkv_cache *c, int Hq, int S, int max_q_len, long long max_kv, int num_splits,
              unsigned flags, bool want_gm, int dev, Plan *pl) {
    int st = check_cache(c);
    if (st) return st;
    if (Hq <= 0 || Hq % c->kv_heads != 0) return PKV_EINVAL;
    if (S < 0 || S > 65535 || max_q_len <= 0 || max_kv <= 0 || num_splits < 0 || num_splits > kMaxSplitsGm)
        return PKV_EINVAL;
    const int D = c->head_dim;
    const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    const int variant = c->dtype == PKV_F32 ? kSimtF32 : (flags & PKV_FLAG_SIMT) ? kSimtBf16 : kMmaBf16;
    pl->G = Hq / c->kv_heads;
    const long long rows_max = (long long)pl->G * max_q_len;
    if (rows_max > (1 << 20)) return PKV_EINVAL;
    pl->rows_max = (int)rows_max;
    // bf16 groups of at most 8 rows take the decode kernel (rows as the MMA's
    // N side; with PKV_FLAG_SIMT its CUDA-core variant).  Long buckets take
    // the decode configuration with more warps (class 5).
    const long long max_pages0 = (max_kv + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE + 1;
    // Wider bf16 groups with head_dim 128 take the tcgen05 tile (class 6)
    // unless the caller asks for the mma.sync one.
    const bool tc = variant == kMmaBf16 && rows_max > 8 && D == 128 && !(flags & PKV_FLAG_MMA_SYNC);
    const int rc = (variant != kSimtF32 && rows_max <= 8) ? (max_pages0 > 256 ? 5 : 4)
                   : tc ? 6
                   : rows_max <= 16 ? 0 : rows_max <= 32 ? 1 : rows_max <= 64 ? 2 : 3;
    pl->k = pick(variant, dp, rc);
    if (!pl->k.fn) return PKV_EUNSUPPORTED;
    pl->gm = want_gm && (rc == 4 || rc == 5);
    if (!pl->gm && num_splits > kMaxCluster) return PKV_EINVAL;
    pl->row_tiles = (int)((rows_max + pl->k.rows - 1) / pl->k.rows);
    if ((long long)c->kv_heads * pl->row_tiles > 65535) return PKV_EINVAL;
    const long long units = (long long)std::max(S, 1) * c->kv_heads * pl->row_tiles;
    pl->units = (int)units;
    const long long max_pages = (max_kv + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE + 1;
    long long n = num_splits;
    if (pl->gm) {
        // independent CTAs: one per SM across the launch (the next layer's
        // CTAs take the second slot of each SM), at least 4 pages each
        if (n == 0) n = std::min<long long>({(device_sms(dev) + units - 1) / units, std::max<long long>(1, max_pages / 4),
                                             (long long)kMaxSplitsGm});
        pl->ncta = (int)std::max<long long>(1, std::min<long long>(n, max_pages));
        return PKV_OK;
    }
    if (n == 0) {
        // CTAs of this kernel that fit on one SM by shared memory.  The
        // tcgen05 tile aims at one wave: its fixed cost per CTA (first page
        // loads, cluster merge) is worth about 15 groups of 64 keys, and it
        // orders ranges longest first and runs short ones alone instead.
        const long long per_sm = std::max<long long>(1, 232448 / ((long long)pl->k.smem + 1024));
        const long long target = (long long)(pl->k.tc ? 1 : kTargetWaves) * device_sms(dev) * per_sm;
        const long long want = (target + units - 1) / units;
        n = 1;
        while (n < want && n < kMaxCluster) n *= 2;
    }
    if ((rc == 4 || rc == 5) && num_splits == 0) {
        // decode kernel: no more CTAs than keep each of their warps two pages
        long long cap = 1;
        while (cap * 2 <= max_pages / 8 && cap * 2 <= kMaxCluster) cap *= 2;
        n = std::min(n, cap);
    }
    n = std::max<long long>(1, std::min<long long>(n, max_pages));
    pl->ncta = (int)n;
    return PKV_OK;
}

// Opt a kernel into its dynamic shared memory size and cluster sizes, once per
// device (the current one, `dev`).
int prepare_kernel(const AttnKernel &k, int dev) {
    static std::mutex mu;
    static KernelTable<bool, kKernelRoom> done;
    std::lock_guard<std::mutex> lock(mu);
    if (done.find(k.fn, dev)) return PKV_OK;
    // Ask for the largest shared-memory carveout so two CTAs fit on an SM:
    // with programmatic dependent launch the next layer's CTAs can then start
    // streaming their pages beside this layer's.
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem) != cudaSuccess ||
        cudaFuncSetAttribute(k.fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
        cudaFuncSetAttribute(k.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ECUDA;
    }
    done.add(k.fn, dev, true);
    return PKV_OK;
}

int launch_status(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ECUDA;
    }
    return PKV_OK;
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// 4-D view (head_dim, kv_heads, 16, num_blocks) of one pool; a box is 128
// bytes of one row of one kv head across the 16 tokens of a page, loaded with
// 128-byte swizzling.
int encode_pool(CUtensorMap *map, const void *pool, const pkv_cache *c) {
    auto fn = encode_fn();
    if (!fn) return PKV_ECUDA;
    const int eb = elem_bytes(c->dtype);
    const cuuint64_t D = (cuuint64_t)c->head_dim, H = (cuuint64_t)c->kv_heads;
    cuuint64_t dims[4] = {D, H, (cuuint64_t)PKV_BLOCK_SIZE, (cuuint64_t)c->num_blocks};
    cuuint64_t strides[3] = {D * eb, H * D * eb, (cuuint64_t)PKV_BLOCK_SIZE * H * D * eb};
    cuuint32_t box[4] = {(cuuint32_t)(128 / eb), 1, (cuuint32_t)PKV_BLOCK_SIZE, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, c->dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                    4, const_cast<void *>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PKV_OK : PKV_ECUDA;
}

// 5-D view (64, 16, D / 64, kv_heads, num_blocks) of one pool, head_dim
// split into 64-element halves (or quarters) ordered after the 16 tokens: one
// box is a whole page tile of one kv head, laid out in shared memory exactly
// as the 4-D view's D / 64 boxes back to back (128-byte swizzle).  Needs
// head_dim a multiple of 64 (no partial last part).
int encode_pool_pages(CUtensorMap *map, const void *pool, const pkv_cache *c) {
    auto fn = encode_fn();
    if (!fn) return PKV_ECUDA;
    const int eb = elem_bytes(c->dtype);
    const cuuint64_t D = (cuuint64_t)c->head_dim, H = (cuuint64_t)c->kv_heads;
    const cuuint64_t part = 128 / eb;
    cuuint64_t dims[5] = {part, (cuuint64_t)PKV_BLOCK_SIZE, D / part, H, (cuuint64_t)c->num_blocks};
    cuuint64_t strides[4] = {H * D * eb, part * eb, D * eb, (cuuint64_t)PKV_BLOCK_SIZE * H * D * eb};
    cuuint32_t box[5] = {(cuuint32_t)part, (cuuint32_t)PKV_BLOCK_SIZE, (cuuint32_t)(D / part), 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, c->dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                    5, const_cast<void *>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PKV_OK : PKV_ECUDA;
}

// ---- quantised caches

struct Plan4 {
    Attend4Kernel k4;
    int G, row_tiles, ncta;
    long long units, pages;  // ranges, and the pages of the longest
    Attend4Kernel ks;  // the kernel of equal shares
    int shares;        // its CTAs, 0: not for these bounds
};

// Equal shares are taken up to this many percent above what the clusters cost at equal
// lengths: they balance lengths that differ, which the bounds do not tell.
// (16 sequences, 8 kv heads, head_dim 128: of 8192 keys each 42 us in shares
// against 35, of random lengths up to that 32 against 32; up to 16384 65
// against 60 and 37 against 47; one sequence of 131072 keys 42 against 59.)
// Every CTA sums the segment table's pages, so the table has to be short.
constexpr int kSharesEdge = 15;
constexpr int kSharesSegments = 512;
constexpr int kSharesTiles = 16;  // each tile's range is taken as long as its segment's: not for long causal chunks
constexpr int kPieceTile = 50;  // (tiles of 16 and 32 rows; 30 and 80 are slower for uneven lengths at every head_dim)
// Rows a kv head from which the tcgen05 kernel (tiles of 128) is faster than mma.sync tiles
// of 32: as shares of 8 sequences of 4096 keys and 8 heads, 32 rows 43 us
// against 34, 36 rows 43 against 51, 128 rows 51 against 89.
constexpr int kWideFrom = 33;

// Whether the kernel was compiled to the register count its warps hand around
// (setmaxnreg waits for registers the launch must have brought).
bool regs_ok(const void *fn, int want, int dev) {
    static std::mutex mu;
    static KernelTable<int, 64> known;
    if (!want) return true;
    std::lock_guard<std::mutex> lock(mu);
    if (const int *regs = known.find(fn, dev)) return *regs == want;
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, fn) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    known.add(fn, dev, a.numRegs);
    return a.numRegs == want;
}

Attend4Kernel pick4_rows(int dtype, int head_dim, int rows, bool few) {
    if (dtype == PKV_FP8) return head_dim == 64 ? pick8_64(rows, few) : head_dim == 128 ? pick8_128(rows, few) : pick8_256(rows, few);
    return head_dim == 64 ? pick4_64(rows, few) : head_dim == 128 ? pick4_128(rows, few) : pick4_256(rows, few);
}

// Clusters of n CTAs that the current device `dev` holds at once with at most l of the
// kernel's CTAs an SM: held[l][n], l up to the CTAs that fit.  Asked once a
// kernel and device (with more shared memory for the smaller l); a guess where no
// device answers.
struct Fit4 {
    int held[5][kMaxCluster + 1];
};
const Fit4 &fit4(const Attend4Kernel &k, int dev) {
    static std::mutex mu;
    static KernelTable<Fit4, 512> known;  // 22 kernels
    static thread_local Fit4 f;
    std::lock_guard<std::mutex> lock(mu);
    if (const Fit4 *kept = known.find(k.fn, dev)) return *kept;
    bool all = dev >= 0 && cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) == cudaSuccess &&
               cudaFuncSetAttribute(k.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    const bool asks = all;
    for (int l = 1; l <= k.ctas; ++l)
        for (int c = 1; c <= kMaxCluster; ++c) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)c, 1, 1);
            cfg.blockDim = dim3((unsigned)k.threads);
            cfg.dynamicSmemBytes = l == k.ctas ? k.smem : std::max<size_t>(k.smem, 233472 / (l + 1));
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)c;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (!asks || cudaOccupancyMaxActiveClusters(&f.held[l][c], k.fn, &cfg) != cudaSuccess) {
                f.held[l][c] = l * kDefaultSms / c;
                all = false;
            }
        }
    if (!all) cudaGetLastError();
    const Fit4 *kept = all ? known.add(k.fn, dev, f) : nullptr;
    return kept ? *kept : f;
}

// What a launch of `units` clusters of n CTAs over `pages` pages each takes
// besides a constant, in ns.  Measured over 1 to 256 ranges of 256 to 16384
// keys at every head_dim and row class: CTAs that share an SM slow each other
// (k.full; two where four fit by 3 / 8 of that), each adds about 0.6 us to
// the launch, a further wave 5 us, and the merge of a cluster 1 us.  Clusters
// start only where a GPC has room for all their CTAs, so the CTAs an SM gets come
// from the occupancy of clusters (32 ranges of 8192 keys: 8 CTAs each, two an SM at
// most, 14.8 us; 9, three an SM, 19.5; 48 ranges: 11 each 18.7 us, 12, a
// second wave, 27.4; 96: 6 each 27.4, 7 each 40.6).  Large clusters, and kernels of
// one or two CTAs an SM, need some room to spare (16 ranges, 32 rows, 8192 keys:
// 12 CTAs each, 23 clusters fit, 24.3 us; 13, 19 fit, 32.5).
// few: the kernel with eight warps, for ranges that leave it alone on its SM: it is
// through a page sooner, and its merge takes longer (one range of 256 keys
// 5.3 us against 5.9, of 4096 7.4 against 6.9, of 8192 7.5 against 8.7).
constexpr double kNever = 1e30;
double cost4(const Attend4Kernel &k, const Fit4 &f, bool few, long long units, long long pages, int n) {
    const int held = f.held[k.ctas][n];
    if (held <= 0) return kNever;
    const double time = (double)((pages + n - 1) / n) * k.page_ns;
    const long long room = n >= 12 ? units + units / 4 : n >= 8 || (n >= 3 && k.ctas <= 2) ? units + units / 16 : units;
    int l = 1;
    while (l < k.ctas && f.held[l][n] < room) ++l;
    const long long waves = held >= room ? 1 : std::max<long long>(2, (units + units / 8 + held - 1) / held);
    if (few) {
        if (l > 1 || waves > 1) return kNever;
        return n == 1 ? time - 1100 : std::max(time - 100, 1700.0);
    }
    const int slow = l == 1 ? 20 : k.ctas == 4 && l == 2 ? 20 + (k.full - 20) * 3 / 8 : k.full;
    return waves * time * slow / 20 + 600 * (l - 1) + 5000.0 * (waves - 1) - (n == 1 ? 1000 : 0);
}

// CTAs of a range (num_splits, or the cheapest number), their kernel and the cost.
double split4(Attend4Kernel *k4, int dtype, int head_dim, int rows, long long units, long long pages, int num_splits, int dev, int *ncta) {
    double best = kNever;
    const Attend4Kernel cand[2] = {*k4, pick4_rows(dtype, head_dim, rows, true)};
    *ncta = 1;
    for (int few = 0; few < (cand[1].fn == cand[0].fn ? 1 : 2); ++few) {
        const Attend4Kernel &k = cand[few];
        const Fit4 &f = fit4(k, dev);
        // no more CTAs than leave each of its warps four pages
        const int top = (int)std::max<long long>(1, std::min<long long>(kMaxCluster, pages / (4 * k.warps)));
        for (int n = num_splits ? num_splits : 1; n <= (num_splits ? num_splits : top); ++n) {
            const double cost = cost4(k, f, few, units, pages, n);
            if (cost < best) {
                best = cost;
                *k4 = k;
                *ncta = n;
            }
        }
    }
    if (best == kNever && num_splits) *ncta = num_splits;  // (the launch takes the largest that fits)
    return best;
}

// What a piece of a range costs a CTA of equal shares besides its pages (query rows in,
// first pages, partials out), in pages: CTAs are dealt equal sums of both.
// The batch of 32 uneven sequences (8 rows, head_dim 128) takes 77, 63, 58 us with
// 0, 12, 24 pages; uneven 16-row tiles of head_dim 256 (16 sequences up to 4096 keys) took 67 us
// with 12 and 43 with 50, the tcgen05 kernel's drafts of 16 sequences 82, 72, 73 us with 10, 36, 24
// (65 now).
int piece_pages4(const Attend4Kernel &k, int block) {
    return k.rows == 128 ? 36 : k.rows == 8 ? (56 << 10) / (2 * block) : kPieceTile;
}

// The same of equal shares: `units` ranges (by this kernel's row tiles) of `pages`
// pages each, pieces and pages read by all SMs at 1.1 times what full SMs take;
// the second launch and the scan of the segment table cost 10 us (the tcgen05 kernel: 14.5).
double cost4_shares(const Attend4Kernel &k, int block, long long units, long long pages, int dev) {
    return (k.rows == 128 ? 14500 : 10000) +
           (double)units * (pages + piece_pages4(k, block)) * k.page_ns * k.full * 11 / (200.0 * k.ctas * device_sms(dev));
}

struct Ws4Layout {
    size_t head, stat, part, total;
};
Ws4Layout ws4_layout(int shares, int rows, int head_dim) {
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    Ws4Layout w;
    w.head = 0;
    w.stat = al((size_t)2 * shares * 16);
    w.part = al(w.stat + (size_t)2 * shares * rows * 8);
    w.total = al(w.part + (size_t)2 * shares * rows * head_dim * 4);
    return w;
}

int make_plan4(const pkv_cache *c, int Hq, int S, int max_q_len, long long max_kv, int window, int num_splits, int dev, Plan4 *pl) {
    const int st = check_cache(c, true);
    if (st) return st;
    if (Hq <= 0 || Hq % c->kv_heads != 0) return PKV_EINVAL;
    if (S < 0 || S > 65535 || max_q_len <= 0 || max_kv <= 0 || num_splits < 0 || num_splits > kMaxCluster) return PKV_EINVAL;
    pl->G = Hq / c->kv_heads;
    const long long rows = (long long)pl->G * max_q_len;
    if (rows > (1 << 20)) return PKV_EINVAL;
    pl->k4 = pick4_rows(c->dtype, c->head_dim, (int)rows, false);
    pl->row_tiles = (int)((rows + pl->k4.rows - 1) / pl->k4.rows);
    if ((long long)c->kv_heads * pl->row_tiles > 65535) return PKV_EINVAL;
    pl->units = (long long)std::max(S, 1) * c->kv_heads * pl->row_tiles;
    const long long keys = window > 0 ? std::min<long long>(max_kv, (long long)window + max_q_len) : max_kv;
    pl->pages = (keys + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE;
    pl->shares = 0;
    pl->ks = pl->k4;
    const double cost = split4(&pl->k4, c->dtype, c->head_dim, (int)rows, pl->units, pl->pages, num_splits, dev, &pl->ncta);
    if (num_splits == 0 && S > 0 && S <= kSharesSegments) {
        const Attend4Kernel wide = c->dtype == PKV_FP8 ? pick8_wide() : pick4_wide();
        if (c->head_dim == 128 && rows >= kWideFrom && regs_ok(wide.balance, wide.regs, dev)) pl->ks = wide;
        const long long tiles = (rows + pl->ks.rows - 1) / pl->ks.rows;
        const double shares = cost4_shares(pl->ks, block_bytes(c), (long long)S * c->kv_heads * tiles, pl->pages, dev);
        if (tiles <= kSharesTiles && shares < cost * (100 + kSharesEdge) / 100)
            pl->shares = std::min(device_sms(dev) * pl->ks.ctas, kMerge4Slots);
    }
    return PKV_OK;
}

int attend4(const pkv_cache *c, int layer, const void *q, int Hq, int total_rows, const int *seq_info, int S, int max_q_len,
            long long max_kv, int num_splits, float scale, int causal, int window, void *out, float *lse, void *workspace,
            long long workspace_bytes, unsigned *err, unsigned flags, void *stream, bool check_only = false) {
    Plan4 pl;
    const int dev = current_device();
    int st = make_plan4(c, Hq, S, max_q_len, max_kv, window, num_splits, dev, &pl);
    if (st) return st;
    if ((st = check_layer(c, layer))) return st;
    if (total_rows < 0 || window < 0 || (causal != 0 && causal != 1)) return PKV_EINVAL;
    if (!err || !out || !aligned16(out) || (total_rows > 0 && (!q || !aligned16(q)))) return PKV_EINVAL;
    if (S > 0 && (!seq_info || !aligned16(seq_info))) return PKV_EINVAL;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return PKV_EINVAL;
    if (S == 0 && total_rows == 0) return PKV_OK;
    if (workspace && (!aligned16(workspace) || workspace_bytes < 0)) return PKV_EINVAL;
    bool shares = pl.shares > 0 && workspace;
    const Ws4Layout wl = ws4_layout(pl.shares, pl.ks.rows, c->head_dim);
    if (shares && workspace_bytes < (long long)wl.total) {
        // The size query knows no window.  Where it asks for nothing, any workspace will
        // do, though shares would pay for the keys that the window leaves.
        Plan4 whole;
        if (window == 0 || (st = make_plan4(c, Hq, S, max_q_len, max_kv, 0, num_splits, dev, &whole)) || whole.shares) return PKV_EINVAL;
        shares = false;
    }
    if (check_only) return PKV_OK;
    const Attend4Kernel &k4 = shares ? pl.ks : pl.k4;
    const void *fn = shares ? k4.balance : k4.fn;
    const AttnKernel prep{fn, k4.threads, k4.smem, k4.rows, c->head_dim, true, shares && k4.rows == 128};
    if ((st = prepare_kernel(prep, dev))) return st;
    const int ncta = S == 0 || shares ? 1 : schedulable_cluster(prep, pl.ncta, dev);
    Attend4Params p;
    p.k = reinterpret_cast<const unsigned char *>(c->k[layer]);
    p.v = reinterpret_cast<const unsigned char *>(c->v[layer]);
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.block_table = c->block_table;
    p.seq_info = reinterpret_cast<const int4 *>(seq_info);
    p.first_valid = c->first_valid;
    p.out = out;
    p.lse = lse;
    p.err = err;
    p.num_blocks = c->num_blocks;
    p.Hq = Hq;
    p.Hkv = c->kv_heads;
    p.G = pl.G;
    p.total_rows = total_rows;
    p.S = S;
    p.max_seqs = c->max_seqs;
    p.mbps = c->max_blocks_per_seq;
    p.ring_rows = c->ring_rows;
    p.max_q_len = max_q_len;
    p.row_tiles = pl.row_tiles;
    p.min_pages = 4 * k4.warps;  // four a warp
    p.causal = causal;
    p.window = window;
    p.out_bf16 = (flags & PKV_FLAG_OUT_BF16) ? 1 : 0;
    p.early = (flags & PKV_FLAG_PDL) ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.piece_pages = piece_pages4(k4, block_bytes(c));
    p.ws_head = nullptr;
    p.ws_stat = nullptr;
    p.ws_part = nullptr;
    if (shares) {
        char *base = reinterpret_cast<char *>(workspace);
        p.ws_head = reinterpret_cast<int4 *>(base + wl.head);
        p.ws_stat = reinterpret_cast<float2 *>(base + wl.stat);
        p.ws_part = reinterpret_cast<float *>(base + wl.part);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = S == 0 ? dim3(1, 1, 1) : dim3((unsigned)ncta, (unsigned)(c->kv_heads * pl.row_tiles), (unsigned)S);
    if (shares) cfg.gridDim = dim3((unsigned)pl.shares, 1, 1);
    cfg.blockDim = dim3((unsigned)k4.threads);
    cfg.dynamicSmemBytes = k4.smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (ncta > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)ncta;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (!shares || (flags & PKV_FLAG_PDL)) {  // (an early start gains a long launch nothing, and takes room from the merge before it)
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = na ? attr : nullptr;
    cfg.numAttrs = (unsigned)na;
    void *args[] = {&p};
    if ((st = launch_status(cudaLaunchKernelExC(&cfg, fn, args))) || !shares) return st;
    cudaLaunchConfig_t mc = {};
    const int merge_rows = pl.ks.rows == 8 ? 1 : kMerge4Threads / 32;  // a CTA's
    mc.gridDim = dim3((unsigned)pl.shares, (unsigned)((std::min(pl.ks.rows, pl.G * max_q_len) + merge_rows - 1) / merge_rows), 1);
    mc.blockDim = dim3(kMerge4Threads);
    mc.stream = cfg.stream;
    cudaLaunchAttribute after;
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    mc.attrs = &after;
    mc.numAttrs = 1;
    return launch_status(cudaLaunchKernelExC(&mc, pl.ks.merge, args));
}

// ---- norm + rotary + append

// A row argument: 16-byte aligned, rows a multiple of 16 bytes apart and at least `need` elements.
bool rows_ok(const void *ptr, long long stride, long long need, int eb) {
    return ptr && aligned16(ptr) && stride >= need && stride * eb % 16 == 0;
}

// Fields of the row warps, after their checks.  stored: whether v rows come too (append).
int rope_params(const pkv_rope *rope, const pkv_rows *r, int dtype, int head_dim, int kv_heads, bool append, RopeParams *p) {
    const int eb = dtype == PKV_F32 ? 4 : 2;
    if (!r || r->total_rows < 0 || r->q_heads < 0 || r->q_heads > 65535) return PKV_EINVAL;
    const long long nq = (long long)r->q_heads * head_dim, nk = (long long)kv_heads * head_dim;
    const bool q = r->q != nullptr, k = r->k != nullptr;
    if (r->total_rows > 0) {
        if (q != (r->q_heads > 0) || q != (r->q_out != nullptr)) return PKV_EINVAL;
        if (q && (!rows_ok(r->q, r->q_stride, nq, eb) || !rows_ok(r->q_out, r->q_out_stride, nq, eb))) return PKV_EINVAL;
        if (append ? !k || !r->v : k != (r->k_out != nullptr) || r->v || r->v_out || (!q && !k)) return PKV_EINVAL;
        if (k && !rows_ok(r->k, r->k_stride, nk, eb)) return PKV_EINVAL;
        if (r->k_out && !rows_ok(r->k_out, r->k_out_stride, nk, eb)) return PKV_EINVAL;
        if (append && !rows_ok(r->v, r->v_stride, nk, eb)) return PKV_EINVAL;
        if (r->v_out && !rows_ok(r->v_out, r->v_out_stride, nk, eb)) return PKV_EINVAL;
        if (reinterpret_cast<uintptr_t>(r->positions) & 3u) return PKV_EINVAL;
    }
    *p = RopeParams{};
    if (rope) {
        if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 2 || (rope->interleaved != 0 && rope->interleaved != 1))
            return PKV_EINVAL;
        if (rope->rot_dim > 0 && (!rope->turns || (reinterpret_cast<uintptr_t>(rope->turns) & 7u))) return PKV_EINVAL;
        if (!aligned16(rope->q_weight) || !aligned16(rope->k_weight)) return PKV_EINVAL;
        if (!append && rope->rot_dim > 0 && r->total_rows > 0 && !r->positions) return PKV_EINVAL;
        if (rope->num_axes < 0 || rope->num_axes > PKV_ROPE_AXES || (rope->num_axes > 1) != (rope->axis != nullptr)) return PKV_EINVAL;
        p->turns = reinterpret_cast<const unsigned long long *>(rope->turns);
        p->axis = rope->axis;
        p->axes = rope->num_axes > 1 ? rope->num_axes : 1;
        p->rot_dim = rope->rot_dim;
        p->interleaved = rope->interleaved;
        p->mscale = rope->mscale;
        p->eps = rope->eps;
        p->q_weight = rope->q_weight;
        p->k_weight = rope->k_weight;
    }
    p->q = r->q;
    p->k = r->k;
    p->v = r->v;
    p->q_out = r->q_out;
    p->k_out = r->k_out;
    p->v_out = r->v_out;
    p->q_stride = r->q_stride;
    p->k_stride = r->k_stride;
    p->v_stride = r->v_stride;
    p->q_out_stride = r->q_out_stride;
    p->k_out_stride = r->k_out_stride;
    p->v_out_stride = r->v_out_stride;
    p->positions = r->positions;
    p->rows = r->total_rows;
    p->Hq = r->q_heads;
    p->Hkv = kv_heads;
    p->D = head_dim;
    return PKV_OK;
}

int attend_common(const pkv_cache *c, int layer, const void *q, const void *k_new, const void *v_new,
                  int Hq, int total_rows, const int *seq_info, int S, int max_q_len, long long max_kv,
                  int num_splits, float scale, int causal, int window, float *out, float *lse,
                  void *workspace, long long workspace_bytes, unsigned *err, unsigned flags, void *stream,
                  int *counters = nullptr) {
    if (flags & PKV_FLAG_OUT_BF16) return PKV_EUNSUPPORTED;  // 4-bit caches only
    Plan pl;
    const int dev = current_device();
    int st = make_plan(c, Hq, S, max_q_len, max_kv, num_splits, flags, workspace != nullptr, dev, &pl);
    if (st) return st;
    if (workspace && (!aligned16(workspace) || workspace_bytes < 0)) return PKV_EINVAL;
    if ((st = check_layer(c, layer))) return st;
    if (total_rows < 0 || window < 0 || (causal != 0 && causal != 1)) return PKV_EINVAL;
    if (!err || !out || (total_rows > 0 && (!q || !aligned16(q)))) return PKV_EINVAL;
    if (S > 0 && (!seq_info || !aligned16(seq_info))) return PKV_EINVAL;
    if ((reinterpret_cast<uintptr_t>(out) & 3u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return PKV_EINVAL;
    if (k_new && (!v_new || !aligned16(k_new) || !aligned16(v_new))) return PKV_EINVAL;
    if (S == 0 && total_rows == 0) return PKV_OK;
    const bool gm = pl.gm && S > 0 && pl.ncta > 1;
    const WsLayout wl = ws_layout((long long)S * c->kv_heads * pl.row_tiles, pl.ncta, pl.k.dp);
    if (gm && workspace_bytes < (long long)wl.total) return PKV_EINVAL;
    if ((st = prepare_kernel(pl.k, dev))) return st;
    int ncta = S == 0 ? 1 : pl.gm ? pl.ncta : schedulable_cluster(pl.k, pl.ncta, dev);
    if (S > 0 && !pl.gm && num_splits == 0) ncta = wave_cluster(pl.k, pl.units, ncta, dev);

    AttendParams p;
    // bf16 page tiles come in one box when head_dim fills its padded width
    // exactly (128 or 256); otherwise, and for fp32, the 4-D view.
    const bool page_box = c->dtype == PKV_BF16 && c->head_dim == pl.k.dp && c->head_dim > 64 && !pl.k.tc;
    auto encode = [&](CUtensorMap *m, const void *pool) {
        return page_box ? encode_pool_pages(m, pool, c) : encode_pool(m, pool, c);
    };
    p.page_box = page_box ? 1 : 0;
    if (pl.k.tc) {
        // tcgen05 tile: K in 64-column boxes (one K-major tile per 4 pages), V in page boxes
        if ((st = encode_pool(&p.tmap_k, c->k[layer], c)) || (st = encode_pool_pages(&p.tmap_v, c->v[layer], c)))
            return st;
    } else if ((st = encode(&p.tmap_k, c->k[layer])) || (st = encode(&p.tmap_v, c->v[layer]))) {
        return st;
    }
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_pool_w = c->k[layer];
    p.v_pool_w = c->v[layer];
    p.block_table = c->block_table;
    p.seq_info = reinterpret_cast<const int4 *>(seq_info);
    p.first_valid = c->first_valid;
    p.out = out;
    p.lse = lse;
    p.err = err;
    p.num_blocks = c->num_blocks;
    p.Hq = Hq;
    p.Hkv = c->kv_heads;
    p.D = c->head_dim;
    p.G = pl.G;
    p.total_rows = total_rows;
    p.S = S;
    p.max_seqs = c->max_seqs;
    p.mbps = c->max_blocks_per_seq;
    p.ring_rows = c->ring_rows;
    p.max_q_len = max_q_len;
    p.row_tiles = pl.row_tiles;
    p.causal = causal;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.ws_part = nullptr;
    p.ws_stat = nullptr;
    p.ws_flag = nullptr;
    p.ws_count = nullptr;
    if (gm) {
        char *base = reinterpret_cast<char *>(workspace);
        p.ws_part = reinterpret_cast<float *>(base + wl.part);
        p.ws_stat = reinterpret_cast<float2 *>(base + wl.stat);
        p.ws_flag = reinterpret_cast<int *>(base + wl.flag);
        p.ws_count = counters ? counters : reinterpret_cast<int *>(base + wl.count);
    }
    p.k_next = p.v_next = nullptr;
    p.pf_next = 0;
    if ((flags & PKV_FLAG_PREFETCH_NEXT) && layer + 1 < c->num_layers && S > 0 && !check_layer(c, layer + 1)) {
        p.k_next = c->k[layer + 1];
        p.v_next = c->v[layer + 1];
        // L2 budget: ~48 MB; a page is warmed once for all kv heads (K and V).
        const long long page = 2LL * PKV_BLOCK_SIZE * c->kv_heads * c->head_dim * elem_bytes(c->dtype);
        p.pf_next = (int)std::max<long long>(0, std::min<long long>(1 << 20, (48LL << 20) / ((long long)ncta * S * page)));
    }

    cudaLaunchConfig_t cfg = {};
    if (S == 0)
        cfg.gridDim = dim3(1, 1, 1);
    else
        cfg.gridDim = dim3((unsigned)ncta, (unsigned)(c->kv_heads * pl.row_tiles), (unsigned)S);
    cfg.blockDim = dim3((unsigned)pl.k.threads);
    cfg.dynamicSmemBytes = pl.k.smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (ncta > 1 && !gm) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)ncta;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (flags & PKV_FLAG_PDL) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = na ? attr : nullptr;
    cfg.numAttrs = (unsigned)na;
    void *args[] = {&p};
    return launch_status(cudaLaunchKernelExC(&cfg, pl.k.fn, args));
}

int copy_rows(const void *s0, const void *s1, void *d0, void *d1, long long n, int H, int row_bytes,
              long long ss, long long sh, long long ds, long long dh, void *stream) {
    if (n <= 0) return PKV_OK;
    CopyParams p{reinterpret_cast<const char *>(s0), reinterpret_cast<const char *>(s1),
                 reinterpret_cast<char *>(d0), reinterpret_cast<char *>(d1), n, H, row_bytes / 16,
                 ss, sh, ds, dh};
    const long long total = 2 * n * H * (row_bytes / 16);
    const long long blocks = std::min<long long>((total + 255) / 256, (long long)kDefaultSms * 8);
    strided_copy_kernel<<<(unsigned)blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launch_status(cudaSuccess);
}

// Fixed split-merge scratch of pkv_append_attend_noalloc: file-scope device
// memory (zero at module load; every call leaves its counters at zero), so
// that entry point never allocates.
// The arrival counters live in an array of their own, so they are zero at
// every call whatever shape the previous call had.
constexpr long long kStaticScratchBytes = 8ll << 20;
constexpr int kStaticUnits = 4096;
static __device__ __align__(256) unsigned char g_split_scratch[kStaticScratchBytes];
static __device__ __align__(256) int g_split_counters[kStaticUnits];

// Device addresses of g_split_scratch and g_split_counters in the current
// context.  Looked up on every call: the lookup is a host-side query, and an
// address cached from an earlier context (before a cudaDeviceReset, say)
// would be stale.  The first lookup on a device loads the library's module.
bool static_scratch(void **scratch, int **counters) {
    void *a = nullptr, *b = nullptr;
    if (cudaGetSymbolAddress(&a, g_split_scratch) != cudaSuccess ||
        cudaGetSymbolAddress(&b, g_split_counters) != cudaSuccess || !a || !b) {
        cudaGetLastError();
        return false;
    }
    *scratch = a;
    *counters = reinterpret_cast<int *>(b);
    return true;
}

}  // namespace

extern "C" {

int64_t pkv_bucket_for(int64_t length) {
    // vLLM-Omni paged_decode.py: BUCKETS then TAIL_STEP-sized growth.
    static const int64_t buckets[] = {512, 1024, 2048, 4096, 8192};
    for (int64_t b : buckets)
        if (length <= b) return b;
    const int64_t tail = 2048;
    return 8192 + ((length - 8192 + tail - 1) / tail) * tail;
}

const char *pkv_status_str(int s) {
    switch (s) {
        case PKV_OK: return "ok";
        case PKV_EMPTY: return "empty: nothing to copy";
        case PKV_SAME_BUCKET: return "same bucket: no resize needed";
        case PKV_EINVAL: return "invalid argument";
        case PKV_EUNSUPPORTED: return "unsupported dtype or head_dim";
        case PKV_ECUDA: return "CUDA launch or copy failed";
        case PKV_ECAPACITY: return "capacity exceeded";
        case PKV_ESTALE: return "caches describe different shapes";
    }
    return "unknown status";
}

int pkv_append(const pkv_cache *c, int32_t layer, const void *k_new, const void *v_new, int32_t total_rows,
               const int32_t *seq_info, int32_t S, int32_t window, uint32_t *err, void *stream) {
    int st = check_cache(c, true);
    if (st) return st;
    if (is_quantised(c)) {
        const int64_t n = (int64_t)c->kv_heads * c->head_dim;
        pkv_rows r = {};
        r.k = k_new;
        r.v = v_new;
        r.k_stride = r.v_stride = n;
        r.total_rows = total_rows;
        return pkv_norm_rope_append(c, layer, nullptr, &r, seq_info, S, window, err, stream);
    }
    if ((st = check_layer(c, layer))) return st;
    if (S < 0 || total_rows < 0 || window < 0 || !err) return PKV_EINVAL;
    if (S == 0) return PKV_OK;
    if (!seq_info || !aligned16(seq_info)) return PKV_EINVAL;
    if (total_rows > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new))) return PKV_EINVAL;
    AppendParams p;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_pool = c->k[layer];
    p.v_pool = c->v[layer];
    p.block_table = c->block_table;
    p.seq_info = reinterpret_cast<const int4 *>(seq_info);
    p.err = err;
    p.num_blocks = c->num_blocks;
    p.row_bytes = c->kv_heads * c->head_dim * elem_bytes(c->dtype);
    p.total_rows = total_rows;
    p.S = S;
    p.max_seqs = c->max_seqs;
    p.mbps = c->max_blocks_per_seq;
    p.ring_rows = c->ring_rows;
    p.window = window;
    append_kernel<<<(unsigned)S, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launch_status(cudaSuccess);
}

int pkv_rope_turns(const double *inv_freq, int32_t n, uint64_t *turns) {
    if (n < 0 || (n > 0 && (!inv_freq || !turns))) return PKV_EINVAL;
    for (int i = 0; i < n; ++i)
        if (!isfinite(inv_freq[i])) return PKV_EINVAL;
    for (int i = 0; i < n; ++i) {
        // the fraction of a turn a position, in units of 2^-64: whole turns do not matter
        const double t = inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
        const double f = t - floor(t);
        turns[i] = f >= 1.0 ? 0 : (uint64_t)ldexp(f, 32) << 32 | (uint64_t)ldexp(ldexp(f, 32) - floor(ldexp(f, 32)), 32);
    }
    return PKV_OK;
}

int pkv_rope_inv_freq(int32_t rot_dim, double theta, int32_t scaling, double factor, double trained_len, double beta_fast,
                      double beta_slow, double *inv_freq, double *mscale) {
    if (rot_dim <= 0 || rot_dim % 2 || !(theta > 1.0) || !isfinite(theta) || !inv_freq || !mscale) return PKV_EINVAL;
    if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_YARN) return PKV_EINVAL;
    if (scaling != PKV_ROPE_PLAIN && !(factor >= 1.0 && isfinite(factor))) return PKV_EINVAL;
    if (scaling == PKV_ROPE_NTK && rot_dim == 2) return PKV_EINVAL;
    const double two_pi = 6.283185307179586;
    double lo = 0.0, hi = 1.0;
    if (scaling == PKV_ROPE_YARN) {
        if (!(trained_len > 0.0 && isfinite(trained_len)) || !(beta_fast > beta_slow) || !(beta_slow > 0.0) || !isfinite(beta_fast))
            return PKV_EINVAL;
        // the pair index whose wave turns `beta` times in the trained context
        auto pair = [&](double beta) { return rot_dim * log(trained_len / (beta * two_pi)) / (2.0 * log(theta)); };
        lo = fmax(floor(pair(beta_fast)), 0.0);
        hi = fmin(ceil(pair(beta_slow)), rot_dim - 1.0);
        if (!(hi > lo)) hi = lo + 0.001;
    }
    const double base = scaling == PKV_ROPE_NTK ? theta * pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == PKV_ROPE_LINEAR) inv_freq[i] = f / factor;
        else if (scaling == PKV_ROPE_YARN) {
            const double slow = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);  // 1: stretched by the whole factor
            inv_freq[i] = f / factor * slow + f * (1.0 - slow);
        } else {
            inv_freq[i] = f;
        }
    }
    *mscale = scaling == PKV_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return PKV_OK;
}

int pkv_norm_rope(const pkv_rope *rope, int32_t dtype, int32_t head_dim, int32_t kv_heads, const pkv_rows *rows, void *stream) {
    if (dtype != PKV_BF16 && dtype != PKV_F32) return PKV_EUNSUPPORTED;
    if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 256) return PKV_EUNSUPPORTED;
    if (kv_heads < 0 || kv_heads > 65535 || !rope) return PKV_EINVAL;
    RopeParams p;
    const int st = rope_params(rope, rows, dtype, head_dim, kv_heads, false, &p);
    if (st) return st;
    if (p.rows == 0) return PKV_OK;
    return launch_status(launch_rope(p, kNoCache, dtype == PKV_F32, device_sms(current_device()), reinterpret_cast<cudaStream_t>(stream)));
}

int pkv_norm_rope_append(const pkv_cache *c, int32_t layer, const pkv_rope *rope, const pkv_rows *rows, const int32_t *seq_info,
                         int32_t S, int32_t window, uint32_t *err, void *stream) {
    int st = check_cache(c, true);
    if (st) return st;
    if ((st = check_layer(c, layer))) return st;
    if (S < 0 || window < 0 || !err) return PKV_EINVAL;
    if (S > 0 && (!seq_info || !aligned16(seq_info))) return PKV_EINVAL;
    RopeParams p;
    if ((st = rope_params(rope, rows, c->dtype, c->head_dim, c->kv_heads, true, &p))) return st;
    if (S == 0) return PKV_OK;
    p.k_pool = c->k[layer];
    p.v_pool = c->v[layer];
    p.block_table = c->block_table;
    p.seq_info = reinterpret_cast<const int4 *>(seq_info);
    p.err = err;
    p.num_blocks = c->num_blocks;
    p.S = S;
    p.max_seqs = c->max_seqs;
    p.mbps = c->max_blocks_per_seq;
    p.ring_rows = c->ring_rows;
    p.window = window;
    if (c->dtype == PKV_FP8) {
        const int sms = device_sms(current_device());
        if (p.q && p.rows >= kAppend8OwnQ) {
            RopeParams q = p;  // no heads of k and v
            q.k = q.v = nullptr;
            q.k_out = q.v_out = nullptr;
            q.k_pool = q.v_pool = nullptr;
            q.Hkv = 0;
            const cudaError_t e = launch_rope(q, kSameType, false, sms, reinterpret_cast<cudaStream_t>(stream));
            if (e != cudaSuccess) return launch_status(e);
            p.q = nullptr;
            p.q_out = nullptr;
        }
        return launch_status(launch_append8(p, sms, reinterpret_cast<cudaStream_t>(stream)));
    }
    return launch_status(launch_rope(p, c->dtype == PKV_FP4 ? kFp4 : kSameType, c->dtype == PKV_F32, device_sms(current_device()),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int pkv_attend_varlen(const pkv_cache *c, int32_t layer, const void *q, int32_t Hq, int32_t total_rows,
                      const int32_t *seq_info, int32_t S, int32_t max_q_len, int64_t max_kv, int32_t num_splits,
                      float scale, int32_t causal, int32_t window, float *out, float *lse, void *workspace,
                      int64_t workspace_bytes, uint32_t *err, uint32_t flags, void *stream) {
    if (is_quantised(c))
        return attend4(c, layer, q, Hq, total_rows, seq_info, S, max_q_len, max_kv, num_splits, scale, causal, window, out, lse,
                       workspace, workspace_bytes, err, flags, stream);
    return attend_common(c, layer, q, nullptr, nullptr, Hq, total_rows, seq_info, S, max_q_len, max_kv,
                         num_splits, scale, causal, window, out, lse, workspace, workspace_bytes, err, flags,
                         stream);
}

int pkv_attend_prompt(int32_t head_dim, int32_t kv_heads, const pkv_rows *r, const int32_t *seq_info, int32_t S, int32_t max_len,
                      float scale, int32_t causal, int32_t window, void *out, float *lse, uint32_t *err, uint32_t flags, void *stream) {
    if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 256) return PKV_EUNSUPPORTED;
    if (!r || r->total_rows < 0 || kv_heads <= 0 || r->q_heads <= 0 || r->q_heads % kv_heads != 0) return PKV_EINVAL;
    if (r->q_heads / kv_heads > 128) return PKV_EUNSUPPORTED;  // a token's heads fill more than a tile
    if (r->q_out || r->k_out || r->v_out || r->positions || (flags & ~(PKV_FLAG_OUT_BF16 | PKV_FLAG_PDL))) return PKV_EINVAL;
    if (S < 0 || S > 65535 || max_len <= 0 || window < 0 || (causal != 0 && causal != 1) || !(scale > 0.f) || !isfinite(scale * 1.4426950408889634f)) return PKV_EINVAL;
    const long long nq = (long long)r->q_heads * head_dim, nk = (long long)kv_heads * head_dim;
    if (!err || (!out && r->total_rows > 0) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return PKV_EINVAL;
    if (S > 0 && (!seq_info || !aligned16(seq_info))) return PKV_EINVAL;
    if (r->total_rows == 0) return PKV_OK;
    if (!rows_ok(r->q, r->q_stride, nq, 2) || !rows_ok(r->k, r->k_stride, nk, 2) || !rows_ok(r->v, r->v_stride, nk, 2)) return PKV_EINVAL;
    const PromptKernel k = pick_prompt(head_dim);
    PromptParams p;
    p.G = r->q_heads / kv_heads;
    p.tokens = 128 / p.G;
    const int group = k.tiles * p.tokens;  // tokens of a CTA
    // tile groups that segments without a row in common can have: each that has rows has one that they do not fill
    const long long each = ((long long)std::min(max_len, r->total_rows) + group - 1) / group;
    const long long units = std::max(std::min(each * S, (long long)r->total_rows / group + std::min(S, r->total_rows)), 1ll), ctas = units * kv_heads;
    if (ctas > INT32_MAX || each * std::max(S, 1) * kv_heads > INT32_MAX) return PKV_EINVAL;  // (segments that overlap may ask for the second)
    p.units = (int)units;
    auto fn = encode_fn();
    if (!fn) return PKV_ECUDA;
    // (head_dim, heads, rows); a box is 64 columns of the given heads and rows, with 128-byte swizzling
    auto encode = [&](CUtensorMap *map, const void *base, int heads, int64_t stride, int box_heads, int box_rows) {
        cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)r->total_rows};
        cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)stride * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, estr[3] = {1, 1, 1};
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!encode(&p.tmap_q, r->q, r->q_heads, r->q_stride, p.G, p.tokens) || !encode(&p.tmap_k, r->k, kv_heads, r->k_stride, 1, 128) ||
        !encode(&p.tmap_v, r->v, kv_heads, r->v_stride, 1, 128))
        return PKV_ECUDA;
    p.q = reinterpret_cast<const __nv_bfloat16 *>(r->q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(r->k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(r->v);
    p.q_stride = r->q_stride;
    p.k_stride = r->k_stride;
    p.v_stride = r->v_stride;
    p.seq_info = reinterpret_cast<const int4 *>(seq_info);
    p.out = out;
    p.lse = lse;
    p.err = err;
    p.Hq = r->q_heads;
    p.Hkv = kv_heads;
    p.D = head_dim;
    p.total_rows = r->total_rows;
    p.S = S;
    p.max_len = max_len;
    p.causal = causal;
    p.window = window;
    p.out_bf16 = (flags & PKV_FLAG_OUT_BF16) ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    const int dev = current_device();
    if (!regs_ok(k.fn, k.regs, dev)) return PKV_ECUDA;  // (never so as built: its warps would wait for registers)
    int st = prepare_kernel(AttnKernel{k.fn, k.threads, k.smem, 128, head_dim, true, true}, dev);
    if (st) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)k.threads);
    cfg.dynamicSmemBytes = k.smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute after;  // waits for the kernel before it first thing; only the start overlaps that one's end
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &after;
    cfg.numAttrs = 1;
    void *args[] = {&p};
    return launch_status(cudaLaunchKernelExC(&cfg, k.fn, args));
}

int pkv_append_attend(const pkv_cache *c, int32_t layer, const void *q, const void *k_new, const void *v_new,
                      int32_t Hq, int32_t total_rows, const int32_t *seq_info, int32_t S, int32_t max_q_len,
                      int64_t max_kv, int32_t num_splits, float scale, int32_t causal, int32_t window,
                      float *out, float *lse, void *workspace, int64_t workspace_bytes, uint32_t *err,
                      uint32_t flags, void *stream) {
    if (total_rows > 0 && (!k_new || !v_new)) return PKV_EINVAL;
    if (is_quantised(c)) {
        // The attention's arguments are checked first, so that a refused call writes nothing.
        auto attend = [&](bool check_only) {
            return attend4(c, layer, q, Hq, total_rows, seq_info, S, max_q_len, max_kv, num_splits, scale, causal, window, out, lse,
                           workspace, workspace_bytes, err, flags, stream, check_only);
        };
        int st = attend(true);
        if (st) return st;
        if ((st = pkv_append(c, layer, k_new, v_new, total_rows, seq_info, S, window, err, stream))) return st;
        return attend(false);
    }
    return attend_common(c, layer, q, total_rows > 0 ? k_new : nullptr, total_rows > 0 ? v_new : nullptr, Hq,
                         total_rows, seq_info, S, max_q_len, max_kv, num_splits, scale, causal, window, out, lse,
                         workspace, workspace_bytes, err, flags, stream);
}

int pkv_append_attend_noalloc(const pkv_cache *c, int32_t layer, const void *q, const void *k_new,
                              const void *v_new, int32_t Hq, int32_t total_rows, const int32_t *seq_info, int32_t S,
                              int32_t max_q_len, int64_t max_kv, int32_t num_splits, float scale, int32_t causal,
                              int32_t window, float *out, float *lse, uint32_t *err, uint32_t flags, void *stream) {
    if (is_quantised(c))  // needs no scratch
        return pkv_append_attend(c, layer, q, k_new, v_new, Hq, total_rows, seq_info, S, max_q_len, max_kv, num_splits, scale,
                                 causal, window, out, lse, nullptr, 0, err, flags, stream);
    const int64_t need = pkv_attend_workspace_bytes(c, Hq, S, max_q_len, max_kv, num_splits, flags);
    if (need < 0) return (int)need;
    if (need > 0) {
        // One arrival counter per (segment, kv head, row tile) range: the
        // same count the kernel indexes them by.
        Plan pl;
        const int st = make_plan(c, Hq, S, max_q_len, max_kv, num_splits, flags, true, current_device(), &pl);
        if (st) return st;
        if (need > kStaticScratchBytes || (long long)S * c->kv_heads * pl.row_tiles > kStaticUnits)
            return PKV_ECAPACITY;  // rejected before any launch
    }
    void *ws = nullptr;
    int *counters = nullptr;
    if (need > 0 && !static_scratch(&ws, &counters)) return PKV_ECUDA;
    if (total_rows > 0 && (!k_new || !v_new)) return PKV_EINVAL;
    return attend_common(c, layer, q, total_rows > 0 ? k_new : nullptr, total_rows > 0 ? v_new : nullptr, Hq,
                         total_rows, seq_info, S, max_q_len, max_kv, num_splits, scale, causal, window, out, lse, ws,
                         need > 0 ? kStaticScratchBytes : 0, err, flags, stream, counters);
}

int64_t pkv_attend_workspace_bytes(const pkv_cache *c, int32_t Hq, int32_t S, int32_t max_q_len, int64_t max_kv,
                                   int32_t num_splits, uint32_t flags) {
    if (is_quantised(c)) {  // equal shares merge through it, clusters need none
        Plan4 pl4;
        const int st = make_plan4(c, Hq, S, max_q_len, max_kv, 0, num_splits, current_device(), &pl4);
        return st ? st : pl4.shares ? (int64_t)ws4_layout(pl4.shares, pl4.ks.rows, c->head_dim).total : 0;
    }
    Plan pl;
    const int st = make_plan(c, Hq, S, max_q_len, max_kv, num_splits, flags, true, current_device(), &pl);
    if (st) return st;
    if (!pl.gm || S == 0 || pl.ncta <= 1) return 0;
    return (int64_t)ws_layout((long long)S * c->kv_heads * pl.row_tiles, pl.ncta, pl.k.dp).total;
}

int pkv_seq_clone(const pkv_cache *c, int32_t src_col, int32_t dst_col, int64_t n, uint32_t *err, void *stream) {
    int st = check_cache(c);
    if (st) return st;
    if (!err || n < 0 || src_col < 0 || src_col >= c->max_seqs || dst_col < 0 || dst_col >= c->max_seqs)
        return PKV_EINVAL;
    if (!c->ring_rows && n > (long long)c->max_blocks_per_seq * PKV_BLOCK_SIZE) return PKV_ECAPACITY;
    if (n > INT32_MAX - PKV_BLOCK_SIZE) return PKV_EINVAL;
    for (int l = 0; l < c->num_layers; ++l)
        if ((st = check_layer(c, l))) return st;
    if (n == 0 || src_col == dst_col) return PKV_OK;
    const long long lo = (c->ring_rows && n > c->ring_rows) ? n - c->ring_rows : 0;
    const int row_chunks = c->kv_heads * c->head_dim * elem_bytes(c->dtype) / 16;
    for (int l0 = 0; l0 < c->num_layers; l0 += kCloneLayers) {
        CloneParams p = {};
        p.layers = std::min(kCloneLayers, c->num_layers - l0);
        for (int i = 0; i < p.layers; ++i) {
            p.k[i] = reinterpret_cast<char *>(c->k[l0 + i]);
            p.v[i] = reinterpret_cast<char *>(c->v[l0 + i]);
        }
        p.block_table = c->block_table;
        p.err = err;
        p.num_blocks = c->num_blocks;
        p.lo = lo;
        p.n = n;
        p.row_chunks = row_chunks;
        p.mbps = c->max_blocks_per_seq;
        p.ring_rows = c->ring_rows;
        p.src = src_col;
        p.dst = dst_col;
        const long long total = 2LL * p.layers * (n - lo) * row_chunks;
        const long long blocks = std::max<long long>(1, std::min<long long>((total + 255) / 256, (long long)device_sms(current_device()) * 8));
        seq_clone_kernel<<<(unsigned)blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
        if ((st = launch_status(cudaSuccess))) return st;
    }
    return PKV_OK;
}

int pkv_rewind(const pkv_cache *c, int32_t *seq_info, int32_t n, const int32_t *amount, int32_t window,
               uint32_t *err, void *stream) {
    int st = check_cache(c, true);
    if (st) return st;
    if (n < 0 || window < 0 || !err) return PKV_EINVAL;
    if (n == 0) return PKV_OK;
    if (!seq_info || !aligned16(seq_info) || !amount || (reinterpret_cast<uintptr_t>(amount) & 3u)) return PKV_EINVAL;
    rewind_kernel<<<(unsigned)((n + 127) / 128), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<int4 *>(seq_info), amount, n, c->ring_rows, window, err);
    return launch_status(cudaSuccess);
}

int pkv_seqinfo_from_seqused(const int32_t *cu, const int32_t *used, int32_t n, int32_t *out, void *stream) {
    if (n < 0) return PKV_EINVAL;
    if (n == 0) return PKV_OK;
    if (!cu || !used || !out || !aligned16(out)) return PKV_EINVAL;
    seqinfo_from_seqused_kernel<<<(unsigned)((n + 127) / 128), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        cu, used, n, reinterpret_cast<int4 *>(out));
    return launch_status(cudaSuccess);
}

int pkv_advance(int32_t *seq_info, int32_t n, void *stream) {
    if (n < 0) return PKV_EINVAL;
    if (n == 0) return PKV_OK;
    if (!seq_info || !aligned16(seq_info)) return PKV_EINVAL;
    advance_kernel<<<(unsigned)((n + 127) / 128), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<int4 *>(seq_info), n);
    return launch_status(cudaSuccess);
}

int pkv_resize_bucket(const pkv_cache *o, pkv_cache *n, int64_t old_len, void *stream) {
    int st = check_cache(o);
    if (st) return st;
    if ((st = check_cache(n))) return st;
    if (o->num_layers != n->num_layers || o->kv_heads != n->kv_heads || o->head_dim != n->head_dim ||
        o->dtype != n->dtype)
        return PKV_ESTALE;
    if (o->ring_rows || n->ring_rows) return PKV_EINVAL;
    if (old_len < 0) return PKV_EINVAL;
    if (n->bucket == o->bucket) return PKV_SAME_BUCKET;
    if (old_len > o->num_blocks * PKV_BLOCK_SIZE || old_len > n->num_blocks * PKV_BLOCK_SIZE) return PKV_ECAPACITY;
    const int row = o->head_dim * elem_bytes(o->dtype);
    const long long tok = (long long)o->kv_heads * row;
    for (int l = 0; l < o->num_layers; ++l) {
        if (check_layer(o, l) || check_layer(n, l)) return PKV_EINVAL;
    }
    for (int l = 0; l < o->num_layers; ++l) {
        st = copy_rows(o->k[l], o->v[l], n->k[l], n->v[l], old_len, o->kv_heads, row, tok, row, tok, row, stream);
        if (st) return st;
    }
    n->generation = o->generation + 1;
    return PKV_OK;
}

int pkv_load_prefix(const pkv_cache *c, const void *const *keys, const void *const *values, int64_t n,
                    int64_t stride_s, int64_t stride_h, void *stream) {
    int st = check_cache(c);
    if (st) return st;
    if (n == 0 || !keys) return PKV_EMPTY;
    if (n < 0 || !values) return PKV_EINVAL;
    if (n > c->num_blocks * PKV_BLOCK_SIZE) return PKV_ECAPACITY;
    const int eb = elem_bytes(c->dtype);
    const int row = c->head_dim * eb;
    if (stride_s < 0 || stride_h < 0 || (stride_s * eb) % 16 || (stride_h * eb) % 16) return PKV_EINVAL;
    for (int l = 0; l < c->num_layers; ++l) {
        if (check_layer(c, l) || !keys[l] || !values[l] || !aligned16(keys[l]) || !aligned16(values[l]))
            return PKV_EINVAL;
    }
    const long long tok = (long long)c->kv_heads * row;
    for (int l = 0; l < c->num_layers; ++l) {
        st = copy_rows(keys[l], values[l], c->k[l], c->v[l], n, c->kv_heads, row, stride_s * eb, stride_h * eb,
                       tok, row, stream);
        if (st) return st;
    }
    return PKV_OK;
}

int pkv_to_contiguous(const pkv_cache *c, int32_t layer, int64_t n, void *keys_out, void *values_out,
                      void *stream) {
    const bool fp8 = c && c->dtype == PKV_FP8;
    int st = check_cache(c, fp8);
    if (st) return st;
    if ((st = check_layer(c, layer))) return st;
    if (n < 0 || n > c->num_blocks * PKV_BLOCK_SIZE) return PKV_ECAPACITY;
    if (n == 0) return PKV_OK;
    if (!keys_out || !values_out || !aligned16(keys_out) || !aligned16(values_out)) return PKV_EINVAL;
    if (fp8)
        return launch_status(launch_read8(c->k[layer], c->v[layer], keys_out, values_out, n, c->kv_heads, c->head_dim, device_sms(current_device()),
                                          reinterpret_cast<cudaStream_t>(stream)));
    const int row = c->head_dim * elem_bytes(c->dtype);
    const long long tok = (long long)c->kv_heads * row;
    return copy_rows(c->k[layer], c->v[layer], keys_out, values_out, n, c->kv_heads, row, tok, row, row,
                     n * row, stream);
}

}  // extern "C"
