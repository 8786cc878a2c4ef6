// linear_f32.hip -- the linear-product kernels (linear_kernels.hpp) for f32 storage.
#include "linear_kernels.hpp"

namespace fftconv {
FFTCONV_LINEAR_TYPE(f32, float)
}  // namespace fftconv
