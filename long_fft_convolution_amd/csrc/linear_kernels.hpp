// linear_kernels.hpp -- out = act(x W^T + bias) + residual and its gradients
// on the matrix cores.  Instantiated per storage type by linear_f16.hip,
// linear_bf16.hip and linear_f32.hip.
//
// One tile kernel serves the three products of a linear layer,
//     C[m][n] = sum_k A(m, k) B(n, k):
//     out: A = x, B = W, both contiguous along k;
//     dx:  A = dz, B(n, k) = W[k][n], contiguous along n;
//     dW:  A(m, k) = dz[k][m], B(n, k) = x[k][n], both contiguous along the tile.
// A workgroup computes a BM x BN tile over K steps of 32.  Tiles of both
// operands stream from HBM straight into LDS (buffer loads with an LDS
// destination, 16 bytes a lane, zero past the operand's edge by the buffer
// unit's range check) through a ring of S stages, so S - 1 steps of loads are
// on their way and no register holds them.  Fragments are read from LDS half
// a step ahead of the products that take them: the second half of a wave's
// rows under the products of the first, the next step's columns and first half
// under those of the second.  The destination of an LDS load is linear in the
// lane, so the bank swizzle permutes the source: lane l fetches the 16 bytes
// that belong at its place.
//
// An operand contiguous along k lies in LDS as rows of 32 values, its 16-byte
// slots exchanged so that one slot of 16 neighbouring rows covers all banks;
// one contiguous along the tile as k rows of the tile's width, read with the
// transposing LDS read (16-bit types; 32-byte granules exchanged by k) or value
// by value (fp32; 64-byte granules exchanged by k / 8).  The product is taken as
// B A (rows n, columns m), so a lane holds four neighbouring n of one row.
#pragma once

#include "mma.hpp"
#include "sequence_ops.hpp"

namespace fftconv {

// exp and reciprocal of the hardware (each within an ulp or two of fp32, against results rounded to
// 16 bits, or to 24 after sums of K terms)
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + exp(-x)); 0 and 1 at the far ends
__device__ __forceinline__ float logistic(float x) { return fast_rcp(1.0f + fast_exp(-x)); }
// Phi(z), the normal distribution's integral, from e = exp(-z^2 / 2): erfc by Abramowitz and Stegun,
// Handbook of Mathematical Functions, 7.1.26, |error| <= 1.5e-7.
__device__ __forceinline__ float normal_cdf(float z, float e) {
    const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752440f, fabsf(z), 1.0f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    const float tail = 0.5f * p * e;                // Phi(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
}
// z (1 + tanh u) / 2 = z logistic(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
constexpr float kTanh2 = 2.0f * 0.79788456080286535588f;
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
    case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case ACT_GELU: return z * normal_cdf(z, fast_exp(-0.5f * z * z));
    case ACT_GELU_TANH: return z * logistic(kTanh2 * z * fmaf(0.044715f * z, z, 1.0f));
    case ACT_SILU: return z * logistic(z);
    default: return z;
    }
}
__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
    case ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case ACT_GELU: {
        const float e = fast_exp(-0.5f * z * z);
        return normal_cdf(z, e) + (e == 0.0f ? 0.0f : z * e * 0.39894228040143267794f);
    }
    case ACT_GELU_TANH: {
        const float u = z * z, p = logistic(kTanh2 * z * fmaf(0.044715f, u, 1.0f)), n = p * (1.0f - p);
        return p + (n == 0.0f ? 0.0f : z * n * kTanh2 * fmaf(0.134145f, u, 1.0f));   // n vanishes first
    }
    case ACT_SILU: {
        const float p = logistic(z), n = p * (1.0f - p);
        return p + (n == 0.0f ? 0.0f : z * n);
    }
    default: return 1.0f;
    }
}

template <typename T> struct Quad { T v[4]; };

template <typename T> __device__ __forceinline__ void load_quad(const T *p, int n, int vec, float *f) {
    if (vec && n >= 4) {
        Quad<T> q;
        __builtin_memcpy(&q, __builtin_assume_aligned(p, 4 * sizeof(T)), sizeof q);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)q.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < n ? (float)p[i] : 0.0f;
    }
}
template <typename T> __device__ __forceinline__ void store_quad(T *p, int n, int vec, const float *f) {
    if (vec && n >= 4) {
        Quad<T> q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q.v[i] = (T)f[i];
        __builtin_memcpy(__builtin_assume_aligned(p, 4 * sizeof(T)), &q, sizeof q);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = (T)f[i];
    }
}

// bias, kept pre-activation, activation, residual, store: values n .. n + 3 of row m
template <typename T>
__device__ __forceinline__ void linear_epilogue(const LinearGemm &a, int64_t m, int64_t n, float *f) {
    const int left = a.N - n < 4 ? (int)(a.N - n) : 4;
    float t[4];
    if (a.bias) {
        load_quad(static_cast<const T *>(a.bias) + n, left, a.vec_b, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += t[i];
    }
    if (a.pre) store_quad(static_cast<T *>(a.pre) + m * a.ldp + n, left, a.vec_p, f);
    if (a.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = act_value(f[i], a.act);
    }
    if (a.res) {
        load_quad(static_cast<const T *>(a.res) + m * a.ldr + n, left, a.vec_r, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += t[i];
    }
    store_quad(static_cast<T *>(a.C) + m * a.ldc + n, left, a.vec_c, f);
}

// One operand's tile: R rows (of m or n) by 32 of k.  KC: contiguous along k.
constexpr int kStepK = 32;
template <typename T, int R, int NW, bool KC> struct OperandTile {
    static constexpr int E = 16 / (int)sizeof(T);
    static constexpr int PR = KC ? kStepK / E : R / E;      // 16-byte pieces of an LDS row
    static constexpr int VALUES = R * kStepK;
    static constexpr int N = VALUES / E / (64 * NW);        // loads of a lane
    static_assert(VALUES / E % (64 * NW) == 0, "whole loads");

    // An LDS cycle serves 128 bytes: eight lanes of a 16-byte read, sixteen of a transposing one.
    // Exchange of the slots of a row of k values (4 in 16-bit types, 8 in fp32): one slot of eight
    // neighbouring rows covers 128 bytes.
    static __device__ __forceinline__ int turn(int row) { return PR == 4 ? (row >> 1) & 3 : row & 7; }
    // Exchange of the 32-byte granules of a 16-bit tile's k rows: one granule of four neighbouring rows does.
    static __device__ __forceinline__ int granule(int k) { return R >= 128 ? (k & 3) | ((k >> 1) & 4) : k & 3; }
    // LDS piece p holds source piece (row, slot)
    static __device__ __forceinline__ void source(int i, int &row, int &slot) {
        const int p = i * 64 * NW + (int)threadIdx.x;
        row = p / PR;
        const int s = p % PR;
        if (KC) slot = s ^ turn(row);
        else if (sizeof(T) == 2) slot = (s & ~15) | ((((s >> 1) & 7) ^ granule(row)) << 1) | (s & 1);
        else slot = (s & ~15) | ((((s >> 2) & 3) ^ ((row >> 3) & 3)) << 2) | (s & 3);
    }

    uint32_t off[N];    // byte offset of each load from the tile's origin at k = 0
    // rows: how many of the tile's R rows exist (rounded up to pieces along the tile)
    __device__ __forceinline__ void prepare(int64_t ld, int64_t rows) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int row, slot;
            source(i, row, slot);
            const bool in = KC ? row < rows : slot * E < rows;
            off[i] = in ? (uint32_t)(row * ld * (int64_t)sizeof(T)) + slot * 16 : kSkip;
        }
    }
    // origin: the tile's first row at the step's first k; kleft: k values left in this step
    // (pieces that begin past it read zero)
    __device__ __forceinline__ void issue(const T *origin, T *tile, int kleft) const {
        // the buffer view and the LDS place are scalar operands: the wave index as one
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        auto place = [&](int i) { return tile + (i * NW + wave) * 64 * E; };
        if (kleft >= kStepK) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds_load16(origin, place(i), off[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int row, slot;
            source(i, row, slot);
            const uint32_t o = (KC ? slot * E : row) < kleft ? off[i] : kSkip;
            lds_load16(origin, place(i), o);
        }
    }
    // the same tile without alignment or whole pieces: through registers, value by value at the edges
    __device__ __forceinline__ void fetch(const T *origin, int64_t ld, int64_t rows, int64_t kleft, uint4 *r) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int row, slot;
            source(i, row, slot);
            const int64_t most = KC ? kleft : rows;     // along the contiguous direction
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < (KC ? rows : kleft)) {
                const T *p = origin + row * ld + slot * E;
                if (slot * E + E <= most) {
                    __builtin_memcpy(&v, p, 16);
                } else {
                    T e[E];
#pragma unroll
                    for (int j = 0; j < E; ++j) e[j] = slot * E + j < most ? p[j] : (T)0.0f;
                    __builtin_memcpy(&v, e, 16);
                }
            }
            r[i] = v;
        }
    }
    static __device__ __forceinline__ void put(T *tile, const uint4 *r) {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<uint4 *>(tile + (i * 64 * NW + (int)threadIdx.x) * E) = r[i];
    }
    // operand of rows r0 .. r0 + 15 at k slots 8 g + j
    static __device__ __forceinline__ typename Mma<T>::v8 frag(const T *tile, int r0) {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
        if constexpr (KC) {
            const int row = r0 + c;
            if constexpr (sizeof(T) == 2) {
                return *reinterpret_cast<const typename Mma<T>::v8 *>(tile + row * kStepK + (g ^ turn(row)) * E);
            } else {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + row * kStepK + ((2 * g) ^ turn(row)) * E);
                const f32x4 b = *reinterpret_cast<const f32x4 *>(tile + row * kStepK + ((2 * g + 1) ^ turn(row)) * E);
                return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        } else if constexpr (sizeof(T) == 2) {
            const int k = g * 8 + (c >> 2);                       // and k + 4
            const int col = r0 + (c & 3) * 4;                     // 16 columns: one 32-byte granule
            const int h = granule(k);                             // the same for k + 4
            const T *p = tile + k * R + ((col & ~127) | ((((col >> 4) & 7) ^ h) << 4) | (col & 15));
            typedef typename Mma<T>::v4 v4;
            const v4 a = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p)));
            const v4 b = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p + 4 * R)));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typename Mma<T>::v8 v;
            const int col = r0 + c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = g * 8 + j;
                v[j] = tile[k * R + ((col & ~63) | ((((col >> 4) & 3) ^ (g & 3)) << 4) | (col & 15))];
            }
            return v;
        }
    }
};

// Tile of workgroup id: ids are dealt to the 8 XCDs in turn, so consecutive ids of one XCD take
// neighbouring tiles (bands of 8 tile rows), whose operands its own L2 then holds.
__device__ __forceinline__ void tile_of(int64_t id, int64_t tm, int64_t tn, int64_t &bm, int64_t &bn) {
    const int64_t total = tm * tn, per = total / 8, rest = total % 8;
    const int64_t xcd = id % 8, at = id / 8;
    id = xcd * per + (xcd < rest ? xcd : rest) + at;
    const int64_t band = 8 * tn, b = id / band;
    const int64_t rows = tm - b * 8 < 8 ? tm - b * 8 : 8;
    // scalar values: what they address is the same for the whole wave
    bm = __builtin_amdgcn_readfirstlane((int)(b * 8 + id % band % rows));
    bn = __builtin_amdgcn_readfirstlane((int)(id % band / rows));
}

// TM x TN 16x16 tiles per wave, WM x WN waves, S stages (even).  VEC: operands 16-byte aligned in rows of
// whole pieces.
template <typename T, int LAYOUT, int TM, int TN, int WM, int WN, int S, bool VEC>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_gemm_kernel(const LinearGemm a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass, which cannot take the scalar operands, needs the stub alone
    constexpr int BM = TM * WM * 16, BN = TN * WN * 16, NW = WM * WN, BK = kStepK;
    constexpr bool AK = LAYOUT != LAYOUT_TN, BKC = LAYOUT == LAYOUT_NT;
    using TA = OperandTile<T, BM, NW, AK>;
    using TB = OperandTile<T, BN, NW, BKC>;
    using v8 = typename Mma<T>::v8;
    static_assert(S == 2 || S == 4, "the loop is unrolled over the stages and the two fragment sets");
    __shared__ __attribute__((aligned(128))) T sa0[TA::VALUES], sb0[TB::VALUES], sa1[TA::VALUES], sb1[TB::VALUES];
    __shared__ __attribute__((aligned(128))) T sa2[S > 2 ? TA::VALUES : 8], sb2[S > 2 ? TB::VALUES : 8];
    __shared__ __attribute__((aligned(128))) T sa3[S > 2 ? TA::VALUES : 8], sb3[S > 2 ? TB::VALUES : 8];
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    int64_t bm, bn;
    tile_of(blockIdx.x, tm, tn, bm, bn);
    const int64_t m0 = bm * BM, n0 = bn * BN;
    const int64_t k0 = blockIdx.y * a.kper, k1 = k0 + a.kper < a.K ? k0 + a.kper : a.K;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / WN) * TM * 16, wn = (wave % WN) * TN * 16;
    const T *pa = static_cast<const T *>(a.A) + (AK ? m0 * a.lda + k0 : k0 * a.lda + m0);
    const T *pb = static_cast<const T *>(a.B) + (BKC ? n0 * a.ldb + k0 : k0 * a.ldb + n0);
    const int64_t sa_step = AK ? BK : BK * a.lda, sb_step = BKC ? BK : BK * a.ldb;

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    constexpr int H = TM / 2;       // row tiles of a half
    auto read_b = [&](const T *t, v8 *f) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TN; ++j) f[j] = TB::frag(t, wn + j * 16);
    };
    auto read_a = [&](const T *t, v8 *f, int half) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < H; ++i) f[i] = TA::frag(t, wm + (half * H + i) * 16);
    };
    auto multiply = [&](const v8 *fa, const v8 *fb, int half) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < Mma<T>::kParts; ++p)
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[half * H + i][j] = Mma<T>::mma(fb[j], fa[i], acc[half * H + i][j], p);
    };
    TA ta;
    TB tb;
    if constexpr (VEC) {
        constexpr int kLoads = TA::N + TB::N, kLeft = (S - 2) * kLoads;
        ta.prepare(a.lda, a.M - m0);
        tb.prepare(a.ldb, a.N - n0);
        const int steps = (int)((k1 - k0 + BK - 1) / BK), full = (int)((k1 - k0) / BK);
        int next = 0;              // the next step to bring
        auto bring = [&](T *na, T *nb, bool whole) __attribute__((always_inline)) {
            const int kl = whole || next < full ? BK : (int)(k1 - k0) - next * BK;
            ta.issue(pa, na, kl);
            tb.issue(pb, nb, kl);
            pa += sa_step;
            pb += sb_step;
            ++next;
        };
        // waits until the oldest stage of this wave's loads is there (with `deep`, S - 2 stages behind it may
        // still travel) and its LDS reads are done, then for the other waves
        auto arrive = [&](bool deep) __attribute__((always_inline)) {
            if (deep) wait_loads_and_barrier<kLeft>();
            else wait_loads_and_barrier<0>();
        };
        v8 lo[H], hi[H], b0[TN], b1[TN];
        if (steps > 0) bring(sa0, sb0, false);
        if (steps > 1) bring(sa1, sb1, false);
        if (S > 2 && steps > 2) bring(sa2, sb2, false);
        if (S > 2 && steps > 3) bring(sa3, sb3, false);
        if (steps > 0) {
            arrive(false);
            read_b(sb0, b0);
            read_a(sa0, lo, 0);
        }
        // one step in stage (ca, cb); the fragments of the next come from (na, nb).  At the barrier every
        // wave has all it needs of (ca, cb), which then takes the step S ahead.
        auto step = [&](T *ca, T *cb, const T *na, const T *nb, const v8 *fb, v8 *gb) __attribute__((always_inline)) {
            read_a(ca, hi, 1);
            __builtin_amdgcn_sched_barrier(0);      // reads first: products of the half before hide them
            multiply(lo, fb, 0);
            arrive(true);
            read_b(nb, gb);
            read_a(na, lo, 0);
            bring(ca, cb, true);
            __builtin_amdgcn_sched_barrier(0);
            multiply(hi, fb, 1);
        };
        // the same near the end, where there may be no next step and nothing left to bring
        auto last = [&](int k, T *ca, T *cb, const T *na, const T *nb, const v8 *fb, v8 *gb) __attribute__((always_inline)) {
            read_a(ca, hi, 1);
            multiply(lo, fb, 0);
            if (k + 1 < steps) {
                arrive(k + S - 1 < steps);
                if (k + S < steps) bring(ca, cb, false);
                read_b(nb, gb);
                read_a(na, lo, 0);
            }
            multiply(hi, fb, 1);
        };
        int k = 0;
        for (; k + 2 * S <= full; k += S) {
            step(sa0, sb0, sa1, sb1, b0, b1);
            if constexpr (S == 2) {
                step(sa1, sb1, sa0, sb0, b1, b0);
            } else {
                step(sa1, sb1, sa2, sb2, b1, b0);
                step(sa2, sb2, sa3, sb3, b0, b1);
                step(sa3, sb3, sa0, sb0, b1, b0);
            }
        }
        for (; k < steps; k += S) {
            last(k, sa0, sb0, sa1, sb1, b0, b1);
            if constexpr (S == 2) {
                if (k + 1 < steps) last(k + 1, sa1, sb1, sa0, sb0, b1, b0);
            } else {
                if (k + 1 < steps) last(k + 1, sa1, sb1, sa2, sb2, b1, b0);
                if (k + 2 < steps) last(k + 2, sa2, sb2, sa3, sb3, b0, b1);
                if (k + 3 < steps) last(k + 3, sa3, sb3, sa0, sb0, b1, b0);
            }
        }
    } else {
        uint4 ra[TA::N], rb[TB::N];
        auto fetch = [&](int64_t k) __attribute__((always_inline)) {
            const int kl = k1 - k < BK ? (int)(k1 - k) : BK;
            ta.fetch(pa, a.lda, a.M - m0, kl, ra);
            tb.fetch(pb, a.ldb, a.N - n0, kl, rb);
            pa += sa_step;
            pb += sb_step;
        };
        auto step = [&](int64_t k, T *ca, T *cb) __attribute__((always_inline)) {
            v8 fa[H], fb[TN];
            TA::put(ca, ra);
            TB::put(cb, rb);
            __syncthreads();
            if (k + BK < k1) fetch(k + BK);
            read_b(cb, fb);
            read_a(ca, fa, 0);
            multiply(fa, fb, 0);
            read_a(ca, fa, 1);
            multiply(fa, fb, 1);
        };
        if (k0 < k1) fetch(k0);
        for (int64_t k = k0; k < k1; k += 2 * BK) {
            step(k, sa0, sb0);
            if (k + BK < k1) step(k + BK, sa1, sb1);
        }
    }
    if (a.quads && !a.part) {
        // every row of every tensor in whole, aligned quads: 32-bit places in views of the tile, no branches
        struct Q { T v[4]; };
        const int64_t at = m0 + wm, col = n0 + wn;
        const auto vc = wide_view(static_cast<T *>(a.C) + at * a.ldc + col), vr = wide_view(static_cast<const T *>(a.res) + at * a.ldr + col),
                   vp = wide_view(static_cast<T *>(a.pre) + at * a.ldp + col), vb = wide_view(static_cast<const T *>(a.bias) + col);
        const int rows = a.M - at < TM * 16 ? (int)(a.M - at) : TM * 16, cols = a.N - col < TN * 16 ? (int)(a.N - col) : TN * 16;
        float bias[TN][4];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const Q q = view_load_wide<Q>(vb, a.bias && j * 16 + g * 4 < cols ? (j * 16 + g * 4) * (uint32_t)sizeof(T) : kSkip);
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[j][e] = (float)q.v[e];
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int row = i * 16 + c;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const bool in = row < rows && j * 16 + g * 4 < cols;
                const uint32_t x = (uint32_t)(j * 16 + g * 4) * (uint32_t)sizeof(T);
                float f[4];
                Q q;
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = acc[i][j][e] + bias[j][e];
                if (a.pre) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q.v[e] = (T)f[e];
                    view_store(vp, in ? (uint32_t)(row * (uint32_t)a.ldp) * (uint32_t)sizeof(T) + x : kSkip, q);
                }
                if (a.act != ACT_NONE) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = act_value(f[e], a.act);
                }
                if (a.res) {
                    q = view_load_wide<Q>(vr, in ? (uint32_t)(row * (uint32_t)a.ldr) * (uint32_t)sizeof(T) + x : kSkip);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] += (float)q.v[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) q.v[e] = (T)f[e];
                view_store(vc, in ? (uint32_t)(row * (uint32_t)a.ldc) * (uint32_t)sizeof(T) + x : kSkip, q);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + wm + i * 16 + c;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t n = n0 + wn + j * 16 + g * 4;
            if (n >= a.N) continue;
            float f[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            if (a.part) {
                float *p = a.part + ((int64_t)blockIdx.y * a.M + m) * a.N + n;
                store_quad(p, a.N - n < 4 ? (int)(a.N - n) : 4, a.N % 4 == 0, f);
            } else {
                linear_epilogue<T>(a, m, n, f);
            }
        }
    }
#endif
}

// joins the splits of a product: sum of the partial sums in split order, then the epilogue
template <typename T> __global__ __launch_bounds__(256) void linear_join_kernel(const LinearGemm a) {
    const int64_t quads = (a.N + 3) / 4, total = a.M * quads;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / quads, n = i % quads * 4;
        const int left = a.N - n < 4 ? (int)(a.N - n) : 4;
        float f[4] = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            float t[4];
            load_quad(a.part + ((int64_t)s * a.M + m) * a.N + n, left, a.N % 4 == 0, t);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] += t[j];
        }
        linear_epilogue<T>(a, m, n, f);
    }
}

// Few rows (M <= 16 MT): bound by the bytes of W.  A wave multiplies 16 rows of W, read straight
// from HBM in the operand layout, with the rows of x; the workgroup's waves share K and join in LDS.
template <typename T, int MT, bool VEC>
__global__ __launch_bounds__(256) void linear_rows_kernel(const LinearGemm a) {
    constexpr int U = 4;
    __shared__ f32x4 part[4][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t per = ((a.K + 31) / 32 + 3) / 4 * 32;
    const int64_t k0 = wave * per, k1 = k0 + per < a.K ? k0 + per : a.K;
    const T *pw = static_cast<const T *>(a.B) + (n0 + c) * a.ldb;
    const T *px = static_cast<const T *>(a.A) + c * a.lda;
    const bool wn = n0 + c < a.N;
    typedef typename Mma<T>::v8 v8;
    auto load8 = [&](const T *p, int64_t k, bool in) {
        v8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (T)0.0f;
        if (VEC) {
            if (in && k < k1) __builtin_memcpy(&v, __builtin_assume_aligned(p + k, 16), sizeof v);
        } else if (in && k + 8 <= k1) {
            __builtin_memcpy(&v, p + k, sizeof v);
        } else if (in) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < k1) v[j] = p[k + j];
        }
        return v;
    };
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
    for (int64_t k = k0; k < k1; k += 32 * U) {
        v8 w[U], x[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load8(pw, k + u * 32 + g * 8, wn);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) x[u][i] = load8(px + (int64_t)i * 16 * a.lda, k + u * 32 + g * 8, i * 16 + c < a.M);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = Mma<T>::mma(w[u], x[u][i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MT; i += 4) {
        const f32x4 s = part[0][i][lane] + part[1][i][lane] + part[2][i][lane] + part[3][i][lane];
        const int64_t m = i * 16 + c, n = n0 + g * 4;
        if (m < a.M && n < a.N) {
            float f[4] = {s[0], s[1], s[2], s[3]};
            linear_epilogue<T>(a, m, n, f);
        }
    }
}

// dz and the column sums of slabs of rows.  grid: (columns / (32 V), slabs); thread: V neighbouring
// columns of every eighth row of the slab; the eight rows' sums are joined in LDS.
template <typename T, int V> __global__ __launch_bounds__(256) void linear_dz_kernel(const LinearDz a) {
    constexpr int U = 4;
    __shared__ float part[8][32 * V];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t n = (blockIdx.x * (int64_t)32 + tx) * V;
    const int64_t m0 = blockIdx.y * a.rows, m1 = m0 + a.rows < a.M ? m0 + a.rows : a.M;
    const T *po = static_cast<const T *>(a.dout) + n, *pp = static_cast<const T *>(a.pre) + n;
    T *pz = static_cast<T *>(a.dz) + n;
    struct Row { T v[V]; };
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    const bool in = n < a.N, pad = a.dz && n < a.ldz;      // (V > 1: N is a multiple of V)
    if (in || pad)
        for (int64_t m = m0 + ty; m < m1; m += 8 * U) {
            Row d[U], z[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (in && m + u * 8 < m1) {
                    __builtin_memcpy(&d[u], __builtin_assume_aligned(po + (m + u * 8) * a.ldo, V * sizeof(T)), sizeof(Row));
                    if (a.act != ACT_NONE)
                        __builtin_memcpy(&z[u], __builtin_assume_aligned(pp + (m + u * 8) * a.ldp, V * sizeof(T)), sizeof(Row));
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) d[u].v[j] = z[u].v[j] = (T)0.0f;
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (m + u * 8 >= m1) continue;
                Row w;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float f = (float)d[u].v[j] * (a.act != ACT_NONE ? act_slope((float)z[u].v[j], a.act) : 1.0f);
                    sum[j] += f;
                    w.v[j] = (T)f;
                }
                if (a.dz) __builtin_memcpy(__builtin_assume_aligned(pz + (m + u * 8) * a.ldz, V * sizeof(T)), &w, sizeof(Row));
            }
        }
    if (!a.colsum) return;
#pragma unroll
    for (int j = 0; j < V; ++j) part[ty][tx * V + j] = sum[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
        const int64_t col = blockIdx.x * (int64_t)(32 * V) + i;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += part[r][i];
        if (col < a.N) a.colsum[blockIdx.y * a.N + col] = s;
    }
}
// sums of the slabs' sums: 16 columns x 16 shares of the slabs a workgroup
template <typename T>
__global__ __launch_bounds__(256) void linear_colsum_kernel(const float *colsum, int64_t slabs, int64_t N, T *dbias) {
    __shared__ float part[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t n = blockIdx.x * (int64_t)16 + tx;
    float s = 0.0f;
    if (n < N) {
#pragma unroll 8
        for (int64_t i = ty; i < slabs; i += 16) s += colsum[i * N + n];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && n < N) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) t += part[r][tx];
        dbias[n] = (T)t;
    }
}

// ---- host side of one storage type ----------------------------------------
template <typename T, int LAYOUT>
static hipError_t gemm_layout(const LinearGemm &a, int tile, bool vec, hipStream_t stream) {
    auto blocks = [&](int bm, int bn) {
        return dim3((unsigned)(((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn)), (unsigned)a.splits);
    };
    constexpr int S = sizeof(T) == 2 ? 4 : 2;      // stages of the 128 tile: 64 KB
    if (!vec) {
        linear_gemm_kernel<T, LAYOUT, 4, 4, 2, 2, 2, false><<<blocks(128, 128), 256, 0, stream>>>(a);
    } else if (tile == 256) {
        if constexpr (sizeof(T) == 2)
            linear_gemm_kernel<T, LAYOUT, 8, 4, 2, 4, 4, true><<<blocks(256, 256), 512, 0, stream>>>(a);
    } else if (tile == 128) {
        linear_gemm_kernel<T, LAYOUT, 4, 4, 2, 2, S, true><<<blocks(128, 128), 256, 0, stream>>>(a);
    } else {
        linear_gemm_kernel<T, LAYOUT, 2, 2, 2, 2, S, true><<<blocks(64, 64), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t gemm_typed(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t stream) {
    hipError_t e = layout == LAYOUT_NT   ? gemm_layout<T, LAYOUT_NT>(a, tile, vec, stream)
                   : layout == LAYOUT_NN ? gemm_layout<T, LAYOUT_NN>(a, tile, vec, stream)
                                         : gemm_layout<T, LAYOUT_TN>(a, tile, vec, stream);
    if (e != hipSuccess || !a.part) return e;
    const int64_t n = (a.M * ((a.N + 3) / 4) + 255) / 256;
    linear_join_kernel<T><<<(unsigned)(n < 4096 ? n : 4096), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T> static hipError_t rows_typed(const LinearGemm &a, bool vec, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.N + 15) / 16);
#define FFTCONV_ROWS(MT)                                                                       \
    do {                                                                                       \
        if (vec) linear_rows_kernel<T, MT, true><<<grid, 256, 0, stream>>>(a);                 \
        else linear_rows_kernel<T, MT, false><<<grid, 256, 0, stream>>>(a);                    \
    } while (0)
    if (a.M <= 16) FFTCONV_ROWS(1);
    else if (a.M <= 32) FFTCONV_ROWS(2);
    else FFTCONV_ROWS(4);
#undef FFTCONV_ROWS
    return hipGetLastError();
}

template <typename T>
static hipError_t dz_typed(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t cols = a.dz ? a.ldz : a.N;
    if (a.vec) linear_dz_kernel<T, V><<<dim3((unsigned)((cols + 32 * V - 1) / (32 * V)), (unsigned)slabs), 256, 0, stream>>>(a);
    else linear_dz_kernel<T, 1><<<dim3((unsigned)((cols + 31) / 32), (unsigned)slabs), 256, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.colsum) return e;
    linear_colsum_kernel<T><<<(unsigned)((a.N + 15) / 16), 256, 0, stream>>>(a.colsum, slabs, a.N, static_cast<T *>(dbias));
    return hipGetLastError();
}

#define FFTCONV_LINEAR_TYPE(NAME, T)                                                                            \
    hipError_t launch_linear_gemm_##NAME(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t s) {   \
        return gemm_typed<T>(a, layout, tile, vec, s);                                                           \
    }                                                                                                            \
    hipError_t launch_linear_rows_##NAME(const LinearGemm &a, bool vec, hipStream_t s) {                         \
        return rows_typed<T>(a, vec, s);                                                                         \
    }                                                                                                            \
    hipError_t launch_linear_dz_##NAME(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t s) {           \
        return dz_typed<T>(a, slabs, dbias, s);                                                                  \
    }

}  // namespace fftconv
