// delta_f16.hip -- the gated delta rule kernels (delta_kernels.hpp) for f16 storage.
#include "delta_kernels.hpp"

namespace fftconv {
FFTCONV_DELTA_TYPE(f16, _Float16)
}  // namespace fftconv
