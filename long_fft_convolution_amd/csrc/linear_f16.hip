// linear_f16.hip -- the linear-product kernels (linear_kernels.hpp) for f16 storage.
#include "linear_kernels.hpp"

namespace fftconv {
FFTCONV_LINEAR_TYPE(f16, _Float16)
}  // namespace fftconv
