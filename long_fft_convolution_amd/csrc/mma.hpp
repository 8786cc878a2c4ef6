// mma.hpp -- real 16x16x32 tile products on the matrix cores for the three
// storage types, shared by the decay-attention and linear-product kernels.
//
// mma(a, b, c): C (16x16, fp32) += A (16 x 32) B (32 x 16).  Lane l = 16 g + c
// holds, of A, row c at the 8 K slots 8 g + j; of B, column c at the same
// slots; of C, rows 4 g + i of column c.  fp16 / bf16: one
// v_mfma_f32_16x16x32.  fp32: eight v_mfma_f32_16x16x4, the j-th taking slot
// 8 g + j of every lane -- the contraction index may be met in any order as
// long as A and B agree, so the fp32 operands keep the 16-bit operand layout.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fftconv_internal.hpp"

namespace fftconv {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Mma;

// fp16 and bf16: 4 values at column steps of a transposed LDS read
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define FFTCONV_LDS_CAST(type, p) \
    ((__attribute__((address_space(3))) type *)(__attribute__((address_space(3))) void *)(p))

template <> struct Mma<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    typedef _Float16 v4 __attribute__((ext_vector_type(4)));
    static constexpr int kParts = 1;
    static __device__ __forceinline__ f32x4 mma(v8 a, v8 b, f32x4 c, int part = 0) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    // terms of the storage type that hold an fp32 value to fp32 precision (2 x 11 bits, given a scale
    // that keeps the second term out of the subnormals), and to well below one storage rounding
    static constexpr int kExactTerms = 2, kTerms = 2;
    static constexpr bool kNarrow = true;   // the type's range needs that scale
};
template <> struct Mma<__bf16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    typedef __bf16 v4 __attribute__((ext_vector_type(4)));
    static constexpr int kParts = 1;
    static __device__ __forceinline__ f32x4 mma(v8 a, v8 b, f32x4 c, int part = 0) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static constexpr int kExactTerms = 3, kTerms = 2;   // 3 x 8 bits; 2 x 8 bits
    static constexpr bool kNarrow = false;
};
template <> struct Mma<float> {
    typedef float v8 __attribute__((ext_vector_type(8)));
    typedef float v4 __attribute__((ext_vector_type(4)));
    static constexpr int kParts = 8;      // instructions of one product, for callers that interleave several
    static __device__ __forceinline__ f32x4 mma(const v8 &a, const v8 &b, f32x4 c, int part) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a[part], b[part], c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mma(const v8 &a, const v8 &b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static constexpr int kExactTerms = 1, kTerms = 1;
    static constexpr bool kNarrow = false;
};

// Splits eight fp32 values into TERMS operands of the storage type whose sum holds them: the products
// of all terms with another operand add up to the product with the value.
template <typename T, int TERMS> __device__ __forceinline__ void split8(const float (&x)[8], typename Mma<T>::v8 (&out)[TERMS]) {
    if constexpr (sizeof(T) == 2 && TERMS > 1 && !Mma<T>::kNarrow) {
        // bf16 is the upper half of fp32: cutting it off leaves an exact rest, so three terms of 8 bits hold
        // all 24 and each costs one bit operation and one subtraction
        float rest[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
        for (int s = 0; s < TERMS; ++s) {
            if (s == TERMS - 1 && TERMS < 3) {
#pragma unroll
                for (int j = 0; j < 8; ++j) out[s][j] = (T)rest[j];      // the last of two, rounded
                continue;
            }
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)     // upper halves of two values: bytes 2, 3 of each
                u[j] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, rest[2 * j + 1]), __builtin_bit_cast(uint32_t, rest[2 * j]),
                                             0x07060302u);
            __builtin_memcpy(&out[s], u, 16);
            if (s + 1 < TERMS) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rest[j] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest[j]) & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float rest = x[j];
            // one value for every use: left to itself the compiler rounds a product to fp16 once through
            // fp32 and once fused, and the two first terms then differ at ties
            if (TERMS > 1) asm("" : "+v"(rest));
#pragma unroll
            for (int s = 0; s < TERMS; ++s) {
                const T part = (T)rest;
                out[s][j] = part;
                rest -= (float)part;
            }
        }
    }
}

// A raw buffer view at a wave-uniform p whose offsets up to 2^31 - 2 are in range; kSkip is out of
// range, so a load there reads zero and a store there writes nothing.  Lanes that have nothing to do
// take that offset instead of a branch: the accumulators then never live across a region that runs with
// part of the lanes (where moving one to another register would lose the others' values).
constexpr uint32_t kSkip = 0x80000000u;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t wide_view(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, 0x7fffffff, 0x00020000);
}
// one value, and `bytes` bytes, at a byte offset of a view
template <typename T> __device__ __forceinline__ T view_load(__amdgpu_buffer_rsrc_t v, uint32_t off) {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(v, off, 0, 0));
    else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(v, off, 0, 0));
}
template <typename V> __device__ __forceinline__ V view_load_wide(__amdgpu_buffer_rsrc_t v, uint32_t off) {
    if constexpr (sizeof(V) == 8) return __builtin_bit_cast(V, (u32x2)__builtin_amdgcn_raw_buffer_load_b64(v, off, 0, 0));
    else return __builtin_bit_cast(V, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(v, off, 0, 0));
}
template <typename V> __device__ __forceinline__ void view_store(__amdgpu_buffer_rsrc_t v, uint32_t off, const V &x) {
    if constexpr (sizeof(V) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, x), v, off, 0, 0);
    else if constexpr (sizeof(V) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), v, off, 0, 0);
    else if constexpr (sizeof(V) == 8) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), v, off, 0, 0);
    else if constexpr (sizeof(V) == 16) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), v, off, 0, 0);
    else {
        struct Half { unsigned char b[sizeof(V) / 2]; };
        struct Two { Half h[2]; };
        const Two t = __builtin_bit_cast(Two, x);
        view_store(v, off, t.h[0]);
        view_store(v, off + (uint32_t)(sizeof(V) / 2), t.h[1]);     // kSkip + 16 is out of range, too
    }
}

// The 64 lanes' 16 bytes at byte offsets off from the wave-uniform p, straight into LDS at dst + 16 lane
// (dst wave-uniform); zeros for offsets out of range, like wide_view.  Written out because the compiler
// follows only a few of such loads apart and makes every LDS read wait for the rest: here the kernel says
// itself (wait_loads) what has to have arrived.  The instruction has no destination register, and waits
// that the compiler adds for its own loads only grow stricter by loads it does not know.
__device__ __forceinline__ void lds_load16(const void *p, void *dst, uint32_t off) {
    const uint64_t base = reinterpret_cast<uint64_t>(p);
    const u32x4 view = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
    const uint32_t at = (uint32_t)(uintptr_t)FFTCONV_LDS_CAST(void, dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(view) : "memory", "m0");
}
// Waits until at most LEFT of this wave's vector loads and stores, and none of its LDS reads, are on their
// way, then for the other waves of the workgroup.
template <int LEFT> __device__ __forceinline__ void wait_loads_and_barrier() {
    static_assert(LEFT < 64, "six bits");
    // products before the wait are issued before it: they are what it hides behind
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | 0x70 | (LEFT >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Largest of the four lanes 16 g + c of each c, in all of them: two steps that exchange rows of 16.  For values that
// are not negative, whose bits have their order (a NaN counts as the largest).
__device__ __forceinline__ uint32_t rows_max_bits(uint32_t x) {
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = a[0] > a[1] ? a[0] : a[1];
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return b[0] > b[1] ? b[0] : b[1];
}
__device__ __forceinline__ float rows_max(float x) {
    const uint32_t most = rows_max_bits(__builtin_bit_cast(uint32_t, x));
    return __builtin_bit_cast(float, most);
}
// The same of the wave's 64 values: four steps within rows of 16 lanes, then the rows.
__device__ __forceinline__ float wave_max(float x) {
    uint32_t u = __builtin_bit_cast(uint32_t, x);
#define FFTCONV_DPP(CTRL) \
    { const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)u, CTRL, 0xf, 0xf, true); u = u > other ? u : other; }
    FFTCONV_DPP(0xb1);      // lanes 1 0 3 2 of each four
    FFTCONV_DPP(0x4e);      // lanes 2 3 0 1
    FFTCONV_DPP(0x141);     // halves of a row mirrored
    FFTCONV_DPP(0x140);     // rows mirrored
#undef FFTCONV_DPP
    u = rows_max_bits(u);
    return __builtin_bit_cast(float, u);
}
// 32 bits whose lower half has bit c set where any of the lanes 16 g + c votes
__device__ __forceinline__ uint32_t rows_vote(bool yes) {
    const uint64_t lanes = __ballot(yes);
    const uint32_t two = (uint32_t)lanes | (uint32_t)(lanes >> 32);
    return two | two >> 16;
}
// fp16 operands need no scale while their largest value is below kFp16High and not below kFp16Low (one row) or
// kFp16LowAll (several columns, some of which may be smaller): values above 2^-14 are normal numbers, smaller ones
// are off by 2^-25, which is 2^-15 of a largest value of 2^-10.
constexpr float kFp16Low = 0x1p-10f, kFp16LowAll = 0x1p-2f, kFp16High = 0x1p15f;
// Power of two that brings a largest value of `top` to 2^14 .. 2^15 (2^100 at most: what is smaller still needs no
// bits); infinity, NaN and zero as they come.
__device__ __forceinline__ int fp16_shift(float top) {
    const int s = 15 - __builtin_amdgcn_frexp_expf(top);
    return s < 100 ? s : 100;
}

}  // namespace fftconv
