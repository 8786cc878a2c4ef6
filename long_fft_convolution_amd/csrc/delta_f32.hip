// delta_f32.hip -- the gated delta rule kernels (delta_kernels.hpp) for f32 storage.
#include "delta_kernels.hpp"

namespace fftconv {
FFTCONV_DELTA_TYPE(f32, float)
}  // namespace fftconv
