// Instantiates the attention over quantised caches for one head_dim (-DPKV_INST_D=<64|128|256>) and
// format (-DPKV_INST_BITS=<4|8>).
#include "attend4.cuh"

#ifndef PKV_INST_D
#error "PKV_INST_D not set"
#endif
#ifndef PKV_INST_BITS
#error "PKV_INST_BITS not set"
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

#define PICK4_NAME2(B, D) pick##B##_##D
#define PICK4_NAME(B, D) PICK4_NAME2(B, D)

// (page times of the 8-bit kernels: those of 4 bits choose as well at head_dim 64 and 128, over 336 shapes; their own ones
// at 256, 173 and more measured, are up to a quarter better there: 16 uneven sequences up to 8192 keys 69 -> 56 us.)
Attend4Kernel PICK4_NAME(PKV_INST_BITS, PKV_INST_D)(int rows, bool few) {
#if PKV_INST_BITS == 8
#if PKV_INST_D == 64
    if (rows <= 8 && few) return info4<Cfg4<64, 1, 8, 2, 2, 2, false, 8>>(46, 20);
    if (rows <= 8) return info4<Cfg4<64, 1, 4, 3, 2, 3, false, 8>>(78, 34);
    if (rows <= 16) return info4<Cfg4<64, 2, 8, 4, 1, 2, true, 8>>(78, 27);
    return info4<Cfg4<64, 4, 8, 4, 1, 1, true, 8>>(107, 20);
#elif PKV_INST_D == 128
    if (rows <= 8 && few) return info4<Cfg4<128, 1, 8, 2, 2, 1, false, 8>>(67, 20);
    if (rows <= 8) return info4<Cfg4<128, 1, 4, 2, 2, 3, false, 8>>(100, 42);
    if (rows <= 16) return info4<Cfg4<128, 2, 8, 4, 1, 1, true, 8>>(100, 20);
    return info4<Cfg4<128, 4, 4, 4, 1, 2, true, 8>>(228, 27);
#else
    if (rows <= 8 && few) return info4<Cfg4<256, 1, 8, 3, 1, 1, true, 8>>(165, 20);
    if (rows <= 8) return info4<Cfg4<256, 1, 4, 2, 1, 2, true, 8>>(185, 36);
    return info4<Cfg4<256, 2, 8, 2, 1, 1, true, 8>>(162, 20);
#endif
#elif PKV_INST_D == 64
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
#define WIDE4_NAME2(B) pick##B##_wide
#define WIDE4_NAME(B) WIDE4_NAME2(B)
Attend4Kernel WIDE4_NAME(PKV_INST_BITS)() {
    using C = Wide4<PKV_INST_BITS>;
    return Attend4Kernel{nullptr, reinterpret_cast<const void *>(&wide4_kernel<C>), reinterpret_cast<const void *>(&merge4_kernel<128, 128, 32>),
                         C::kThreads, C::kSmem, C::R, 8, 1, 235, 20, C::kRegs};
}
#endif

}  // namespace pkv
