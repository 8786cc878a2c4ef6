// sequence_device.hpp -- device helpers that the walks over sequences share
// (decay_kernels.hpp, delta_kernels.hpp).
#pragma once
#include "mma.hpp"

namespace fftconv {

// Slot of sequence seq in the state pool, or -1 (no state kept).
__device__ __forceinline__ int64_t state_slot(const int32_t *slots, int64_t n_slots, int64_t seq) {
    if (!slots) return seq;
    const int64_t s = slots[seq];
    return s >= 0 && s < n_slots ? s : -1;
}

constexpr float kLog2e = 1.44269504088896340736f;

// A 64-bit value that is the same in every lane, as a scalar.
__device__ __forceinline__ int64_t scalar(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// NT * 4 neighbouring outputs of a lane at byte offset off (or kSkip).  WHOLE: aligned, and all there
// or none; else `left` of them are, written one by one unless vec and all are there.
template <typename TO, int NT, bool WHOLE>
__device__ __forceinline__ void put_row(__amdgpu_buffer_rsrc_t view, uint32_t off, const f32x4 *o, int vec, int left) {
    struct Row { TO w[NT * 4]; } row;
#pragma unroll
    for (int j = 0; j < NT * 4; ++j) row.w[j] = (TO)o[j >> 2][j & 3];
    const bool whole = WHOLE | ((vec != 0) & (NT * 4 <= left));
    view_store(view, whole ? off : kSkip, row);
    if (!WHOLE) {
#pragma unroll
        for (int j = 0; j < NT * 4; ++j)
            view_store(view, (!whole) & (j < left) & (off != kSkip) ? off + j * (uint32_t)sizeof(TO) : kSkip, row.w[j]);
    }
}

}  // namespace fftconv
