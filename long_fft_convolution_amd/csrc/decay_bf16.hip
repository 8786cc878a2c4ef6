// decay_bf16.hip -- the decay-attention kernels (decay_kernels.hpp) for bf16 storage.
#include "decay_kernels.hpp"

namespace fftconv {
FFTCONV_DECAY_TYPE(bf16, __bf16)
}  // namespace fftconv
