// Instantiates the 4-bit attention kernel for one head_dim (-DPKV_INST_D=<64|128|256>).
#include "attend4.cuh"

#ifndef PKV_INST_D
#error "PKV_INST_D not set"
#endif
#if PKV_INST_D == 128
#include "wide4.cuh"
#endif

namespace pkv {

template <class C>
static Attend4Kernel info4(int page_ns, int full) {
    return Attend4Kernel{reinterpret_cast<const void *>(&attend4_kernel<C>), reinterpret_cast<const void *>(&balance4_kernel<C>),
                         reinterpret_cast<const void *>(&merge4_kernel<C::D, C::R, C::R == 8 ? kMerge4Threads : 32>), C::kThreads, C::kSmem, C::R, C::KW, C::kCtas, page_ns, full, 0};
}

#define PICK4_NAME2(D) pick4_##D
#define PICK4_NAME(D) PICK4_NAME2(D)

Attend4Kernel PICK4_NAME(PKV_INST_D)(int rows, bool few) {
#if PKV_INST_D == 64
    if (rows <= 8 && few) return info4<Cfg4<64, 1, 8, 2, 2, 2, false>>(46, 20);
    if (rows <= 8) return info4<Cfg4<64, 1, 4, 4, 2, 4, false>>(78, 34);
    if (rows <= 16) return info4<Cfg4<64, 2, 8, 4, 1, 2, true>>(78, 27);
    return info4<Cfg4<64, 4, 8, 4, 1, 1, true>>(107, 20);
#elif PKV_INST_D == 128
    if (rows <= 8 && few) return info4<Cfg4<128, 1, 8, 2, 2, 2, false>>(67, 20);
    if (rows <= 8) return info4<Cfg4<128, 1, 4, 2, 2, 4, false>>(100, 42);
    if (rows <= 16) return info4<Cfg4<128, 2, 8, 4, 1, 1, true>>(100, 20);
    return info4<Cfg4<128, 4, 4, 4, 1, 2, true>>(228, 27);
#else
    if (rows <= 8 && few) return info4<Cfg4<256, 1, 8, 3, 1, 1, true>>(110, 20);
    if (rows <= 8) return info4<Cfg4<256, 1, 4, 3, 1, 3, true>>(180, 33);
    return info4<Cfg4<256, 2, 8, 3, 1, 1, true>>(153, 20);
#endif
}

#if PKV_INST_D == 128
Attend4Kernel pick4_wide() {
    return Attend4Kernel{nullptr, reinterpret_cast<const void *>(&wide4_kernel), reinterpret_cast<const void *>(&merge4_kernel<128, 128, 32>),
                         Wide4::kThreads, Wide4::kSmem, Wide4::R, 8, 1, 235, 20, Wide4::kRegs};
}
#endif

}  // namespace pkv
