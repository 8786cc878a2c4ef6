// decay_f16.hip -- the decay-attention kernels (decay_kernels.hpp) for f16 storage.
#include "decay_kernels.hpp"

namespace fftconv {
FFTCONV_DECAY_TYPE(f16, _Float16)
}  // namespace fftconv
