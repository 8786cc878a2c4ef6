// delta_bf16.hip -- the gated delta rule kernels (delta_kernels.hpp) for bf16 storage.
#include "delta_kernels.hpp"

namespace fftconv {
FFTCONV_DELTA_TYPE(bf16, __bf16)
}  // namespace fftconv
