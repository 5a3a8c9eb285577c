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
// Rows from which the queries of such a step go through the row kernel, in a launch of their own.  A page's
// CTA reads every angle again for each head, which is soon slower than the second launch: 32 + 8 heads of 128,
// one launch against two: 512 rows of one prompt 12.9 / 21.2 us, 1024 rows 23.6 / 23.9, 4096 rows 67 / 51;
// a row for each of 256 sequences 20.8 / 20.4, 512 sequences 25.6 / 21.4, 1024 52 / 38, 4096 228 / 151.  (Between 256 and 1024
// sequences of a row each two launches would be faster: the rule asks for the rows alone, where a prompt and a batch meet.)
constexpr int kAppend8OwnQ = 1024;

// The append to an 8-bit cache (bf16 rows; head_dim 64, 128 or 256, S > 0).
cudaError_t launch_append8(const RopeParams &p, int sms, cudaStream_t stream);
// The first n rows of a layer's 8-bit pools, in page order, as bf16 [kv_heads][n][head_dim].
cudaError_t launch_read8(const void *k, const void *v, void *k_out, void *v_out, long long n, int kv_heads, int head_dim, int sms, cudaStream_t stream);

}  // namespace pkv
