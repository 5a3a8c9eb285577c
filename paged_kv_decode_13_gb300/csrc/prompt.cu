// Instantiations of the prompt attention kernel.
#include "prompt.cuh"

namespace pkv {

template <int DP>
static PromptKernel info_prompt() {
    using C = PromptCfg<DP>;
    return PromptKernel{reinterpret_cast<const void *>(&prompt_kernel<C>), C::kThreads, C::kSmem, C::NT, C::kRegs};
}

PromptKernel pick_prompt(int head_dim) {
    return head_dim <= 64 ? info_prompt<64>() : head_dim <= 128 ? info_prompt<128>() : info_prompt<256>();
}

}  // namespace pkv
