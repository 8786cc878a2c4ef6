// decay_f32.hip -- the decay-attention kernels (decay_kernels.hpp) for f32 storage.
#include "decay_kernels.hpp"

namespace fftconv {
FFTCONV_DECAY_TYPE(f32, float)
}  // namespace fftconv
