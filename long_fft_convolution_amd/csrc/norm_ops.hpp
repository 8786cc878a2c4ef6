// norm_ops.hpp -- what the host side of the root-mean-square norm
// (norm_ops.cpp) passes to its kernels (norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fftconv {

// Rows are (M, G) of D values; strides (row, group) in elements.
struct NormFwd {
    const void *x, *res, *weight;    // res, weight: null = none
    void *out, *sum;                 // sum: null = not kept
    float *scales;                   // (M, G), out is in 8 bits; null = out in the storage type
    int64_t xs[2], rs[2], os[2], ss[2];
    uint32_t rows, G;
    int D;
    float eps;
};

struct NormBwd {
    const void *dout, *x, *weight, *dsum;    // weight, dsum: null = none
    void *dx;                                // null = skip
    float *part;                             // (slabs, D) sums of the weight's gradient, null = skip
    float *stats;                            // (rows, 2), rows that no workgroup holds only
    int64_t gs[2], xs[2], us[2], ds[2];
    uint32_t rows, G;
    int D;
    float eps;
};

// How a call's rows are met: `lanes` of a workgroup's 256 threads hold a row, each `loads` pieces of
// `vec` values; loads = 0: the row is read again instead of held.
constexpr int kFwdWave = 2, kBwdWave = 5;      // the most pieces a lane of a wave that holds a row by itself
struct NormPlan {
    int vec, lanes, loads;
    int64_t groups;      // workgroups
    int64_t slabs;       // partial sums of the weight's gradient
};

hipError_t launch_norm_fwd(int dtype, const NormFwd &a, const NormPlan &p, hipStream_t stream);
hipError_t launch_norm_bwd(int dtype, const NormBwd &a, const NormPlan &p, void *dweight, hipStream_t stream);

}  // namespace fftconv
