// Instantiates the append to an 8-bit cache for one head_dim (-DPKV_INST_D=<64|128|256>).
#include "append8.cuh"

#ifndef PKV_INST_D
#error "PKV_INST_D not set"
#endif

namespace pkv {

template <int D, bool RING>
static const void *pick(int pair) {
    switch (pair) {
        case kPlainRows: return reinterpret_cast<const void *>(&append8_kernel<D, kPlainRows, RING>);
        case kInLane: return reinterpret_cast<const void *>(&append8_kernel<D, kInLane, RING>);
        case kByShuffle: return reinterpret_cast<const void *>(&append8_kernel<D, kByShuffle, RING>);
        default: return reinterpret_cast<const void *>(&append8_kernel<D, kByShared, RING>);
    }
}

#define PICK_APPEND8_2(D) pick_append8_##D
#define PICK_APPEND8(D) PICK_APPEND8_2(D)

const void *PICK_APPEND8(PKV_INST_D)(int pair, bool ring) { return ring ? pick<PKV_INST_D, true>(pair) : pick<PKV_INST_D, false>(pair); }

}  // namespace pkv
