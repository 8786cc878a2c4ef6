// linear_bf16.hip -- the linear-product kernels (linear_kernels.hpp) for bf16 storage.
#include "linear_kernels.hpp"

namespace fftconv {
FFTCONV_LINEAR_TYPE(bf16, __bf16)
}  // namespace fftconv
