// Host-side view of the norm + rotary + append kernel.
#pragma once

#include "rope.cuh"

namespace pkv {

// Warps an SM holds, and takes rows in turn with.
constexpr int kRopeFill = 20;
// Warps an SM is given before the warps of a row take more than one group of its heads.
constexpr int kRopeSpread = 20;

// Picks the instantiation and the split (fills the fields the split decides).
// cache: RopeCache; f32: the rows' type (bf16 otherwise; 4-bit caches take bf16 rows).
cudaError_t launch_rope(RopeParams &p, int cache, bool f32, int sms, cudaStream_t stream);

// CTAs an SM is given, at most, before pages share one, and before the heads of a page do.
constexpr int kAppend8Most = 16;
constexpr int kAppend8Fill = 6;

// The append to an 8-bit cache (bf16 rows; head_dim 64, 128 or 256, S > 0).
cudaError_t launch_append8(const RopeParams &p, int sms, cudaStream_t stream);
// The first n rows of a layer's 8-bit pools, in page order, as bf16 [kv_heads][n][head_dim].
cudaError_t launch_read8(const void *k, const void *v, void *k_out, void *v_out, long long n, int kv_heads, int head_dim, int sms, cudaStream_t stream);

}  // namespace pkv
