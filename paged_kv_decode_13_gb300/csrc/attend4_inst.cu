// Instantiates the 4-bit attention kernel for one head_dim (-DPKV_INST_D=<64|128|256>).
#include "attend4.cuh"

#ifndef PKV_INST_D
#error "PKV_INST_D not set"
#endif

namespace pkv {

template <class C>
static Attend4Kernel info4() {
    return Attend4Kernel{reinterpret_cast<const void *>(&attend4_kernel<C>), C::kThreads, C::kSmem, C::R, C::KW, C::kCtas};
}

#define PICK4_NAME2(D) pick4_##D
#define PICK4_NAME(D) PICK4_NAME2(D)

Attend4Kernel PICK4_NAME(PKV_INST_D)(int rows) {
#if PKV_INST_D == 64
    if (rows <= 8) return info4<Cfg4<64, 1, 8, 6, 2>>();
    if (rows <= 16) return info4<Cfg4<64, 2, 8, 6, 2>>();
    return info4<Cfg4<64, 4, 8, 6, 2>>();
#elif PKV_INST_D == 128
    if (rows <= 8) return info4<Cfg4<128, 1, 8, 4, 2>>();
    if (rows <= 16) return info4<Cfg4<128, 2, 8, 4, 1>>();
    return info4<Cfg4<128, 4, 8, 4, 1>>();
#else
    if (rows <= 8) return info4<Cfg4<256, 1, 8, 3, 1>>();
    return info4<Cfg4<256, 2, 8, 3, 1>>();
#endif
}

}  // namespace pkv
