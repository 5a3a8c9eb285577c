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

}  // namespace pkv
