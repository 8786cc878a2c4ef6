// linear_kernels.hpp -- out = act(x W^T + bias) + residual and its gradients
// on the matrix cores.  Instantiated per storage type by linear_f16.hip,
// linear_bf16.hip and linear_f32.hip.
//
// One tile kernel serves the three products of a linear layer,
//     C[m][n] = sum_k A(m, k) B(n, k):
//     out: A = x, B = W, both contiguous along k;
//     dx:  A = dz, B(n, k) = W[k][n], contiguous along n;
//     dW:  A(m, k) = dz[k][m], B(n, k) = x[k][n], both contiguous along the tile.
// A workgroup computes a tile over K stages of 128 bytes (64 or 32 values).
// Tiles of both operands stream from HBM straight into LDS (buffer loads with
// an LDS destination, 16 bytes a lane, whole 128-byte lines, zero past the
// operand's edge by the buffer unit's range check), so no register holds them.
// The destination of such a load is linear in the lane, so the bank swizzle
// permutes the source: lane l fetches the 16 bytes that belong at its place.
//
// LDS holds two stages, but each operand's tile is two halves (A0, A1, B0, B1)
// and a wave reads each of them into registers once, ahead of its products:
//     A0 B0 while B1 of this stage is read, A0 B1 while A1 is,
//     A1 B0, A1 B1 while A0 and B0 of the next stage are read,
// with a barrier before each line.  A half's place is thus free for the stage
// after next long before its products are done, and its loads have a stage and
// a half (three of those lines) to arrive; LDS reads pass under products.
// At 256 x 256 x 64 a line is 32 matrix instructions a wave (1024 cycles of a
// SIMD's two waves) against 12 LDS reads (768 cycles of the CU's LDS).
//
// Measured in bf16: 8192^3 820 us, 1340 TF/s; 16384 x 2560 -> 10240 715 us, 1200 TF/s, 770 us with bias
// and GELU, 920 to 980 with a residual as well, 905 to 930 with the pre-activation kept (the epilogue's
// 0.3 to 0.7 GB and its arithmetic do not pass under products: a tile ends with them).  The library's
// products in the same runs: 690 and 583 us.  Two stages of 128 bytes against four of 64: 785 against
// 857 us, the shorter ones leaving half the loads a line apart.
//
// An operand contiguous along k lies in LDS as rows of 128 bytes, its eight
// 16-byte slots exchanged by the row; one contiguous along the tile as k rows of
// the tile's width, read with the transposing LDS read (16-bit types; 32-byte
// granules exchanged by k) or value by value (fp32; 64-byte granules exchanged by
// k / 8).  The product is taken as B A (rows n, columns m), so a lane holds four
// neighbouring n of one row.
#pragma once

#include "mma.hpp"
#include "sequence_ops.hpp"

namespace fftconv {

// Activations.  FULL: for results in fp32, relative errors of 2^-20 (the tanh form: and 2^-22 for each unit of the
// logistic function's argument, which is rounded); else for results rounded to 16 bits, 2^-15 before that
// rounding.  Slopes: of the size of their two summands.  exp and reciprocal are the hardware's, an ulp or two.
//
// exp(-(a + rest)) to fp32, a >= 0 and rest a correction to it: a log2 e, rounded, is off by 2^-24 of itself, which
// is an absolute error of the exponent, so what the rounding left out is carried along.
constexpr float kLog2eHi = 1.44269504f, kLog2eLo = 1.92596303e-8f;
__device__ __forceinline__ float exp_minus(float a, float rest) {
    constexpr float kLn2 = 0.69314718f;
    a = a > 200.0f ? 200.0f : a;       // exp(-200) is 0; a NaN stays
    const float t = -a * kLog2eHi, left = fmaf(-a, kLog2eHi, -t) - fmaf(a, kLog2eLo, rest * kLog2eHi);
    return __builtin_amdgcn_exp2f(t) * fmaf(left, kLn2, 1.0f);
}
// p = 1 / (1 + exp(-x)) and p (1 - p); 0 and 1 at the far ends
template <bool FULL> __device__ __forceinline__ float logistic(float x, float &n) {
    if (FULL) {
        const float e = exp_minus(fabsf(x), 0.0f), r = __builtin_amdgcn_rcpf(1.0f + e);
        n = e * r * r;
        return x >= 0.0f ? r : e * r;
    }
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2eHi));
    n = p * (1.0f - p);
    return p;
}
// Phi(z), the normal distribution's integral, and e = exp(-z^2 / 2).  Phi(-|z|) / e = t P(t) with t = 1 / (1 + c |z|):
// polynomials fitted here to the least relative error over |z| <= 14 (behind it e is 0), 3e-8 and 5e-6; with the
// roundings of their evaluation 3e-7 and 5e-6.
template <bool FULL> __device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float m = fabsf(z);
    if (FULL) {
        const float b = m > 20.0f ? 20.0f : m, s = b * b;
        e = exp_minus(0.5f * s, 0.5f * fmaf(b, b, -s));
    } else {
        e = __builtin_amdgcn_exp2f(z * (z * (-0.5f * kLog2eHi)));
    }
    const float t = __builtin_amdgcn_rcpf(fmaf(FULL ? 0.35f : 0.31f, m, 1.0f));
    float p;
    if (FULL) {
        p = fmaf(t, -2.914590947e-02f, 1.439716071e-01f);
        p = fmaf(t, p, -2.557140887e-01f);
        p = fmaf(t, p, 1.591739953e-01f);
        p = fmaf(t, p, -2.310973220e-02f);
        p = fmaf(t, p, 1.055079624e-01f);
        p = fmaf(t, p, 1.198328733e-01f);
        p = fmaf(t, p, 1.398618668e-01f);
        p = fmaf(t, p, 1.396214068e-01f);
    } else {
        p = fmaf(t, -7.392912358e-02f, 1.804502904e-01f);
        p = fmaf(t, p, 1.574476436e-02f);
        p = fmaf(t, p, 1.334297657e-01f);
        p = fmaf(t, p, 1.204412803e-01f);
        p = fmaf(t, p, 1.238607019e-01f);
    }
    const float tail = t * p * e;                // Phi(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
}
// z (1 + tanh u) / 2 = z logistic(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
constexpr float kTanh2 = 2.0f * 0.79788456080286535588f;
template <bool FULL> __device__ __forceinline__ float act_value(float z, int act) {
    float unused;
    switch (act) {
    case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case ACT_GELU: return z * normal_cdf<FULL>(z, unused);
    case ACT_GELU_TANH: return z * logistic<FULL>(kTanh2 * z * fmaf(0.044715f * z, z, 1.0f), unused);
    case ACT_SILU: return z * logistic<FULL>(z, unused);
    default: return z;
    }
}
template <bool FULL> __device__ __forceinline__ float act_slope(float z, int act) {
    float n;
    switch (act) {
    case ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case ACT_GELU: {
        const float p = normal_cdf<FULL>(z, n);
        return p + (n == 0.0f ? 0.0f : z * n * 0.39894228040143267794f);
    }
    case ACT_GELU_TANH: {
        const float u = z * z, p = logistic<FULL>(kTanh2 * z * fmaf(0.044715f * z, z, 1.0f), n);
        return p + (n == 0.0f ? 0.0f : z * n * kTanh2 * fmaf(0.134145f, u, 1.0f));   // n vanishes first
    }
    case ACT_SILU: {
        const float p = logistic<FULL>(z, n);
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
        for (int i = 0; i < 4; ++i) f[i] = act_value<sizeof(T) == 4>(f[i], a.act);
    }
    if (a.res) {
        load_quad(static_cast<const T *>(a.res) + m * a.ldr + n, left, a.vec_r, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += t[i];
    }
    store_quad(static_cast<T *>(a.C) + m * a.ldc + n, left, a.vec_c, f);
}

// Half an operand's tile: R rows (of m or n) by BK of k.  KC: contiguous along k.
template <typename T, int R, int NW, bool KC> struct OperandTile {
    static constexpr int E = 16 / (int)sizeof(T);
    static constexpr int BK = 128 / (int)sizeof(T);
    static constexpr int PR = KC ? BK / E : R / E;          // 16-byte pieces of an LDS row
    static constexpr int VALUES = R * BK;
    static constexpr int N = VALUES / E / (64 * NW);        // loads of a lane
    static_assert(VALUES / E % (64 * NW) == 0, "whole loads");

    // An LDS cycle serves 128 bytes: eight lanes of a 16-byte read (one slot of eight neighbouring rows),
    // sixteen of a transposing one (one 32-byte granule of four neighbouring k rows), 32 of a 4-byte one.
    static __device__ __forceinline__ int granule(int k) { return R >= 64 ? k & 3 : (k >> 1) & 1; }
    static __device__ __forceinline__ int granule32(int k) { return (k >> 3) & (R >= 64 ? 3 : 1); }
    // LDS piece p holds source piece (row, slot)
    static __device__ __forceinline__ void source(int i, int &row, int &slot) {
        const int p = i * 64 * NW + (int)threadIdx.x;
        row = p / PR;
        const int s = p % PR;
        if (KC) slot = s ^ (row & 7);
        else if (sizeof(T) == 2) slot = (((s >> 1) ^ granule(row)) << 1) | (s & 1);
        else slot = (((s >> 2) ^ granule32(row)) << 2) | (s & 3);
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
        if (kleft >= BK) {
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
    // operand of rows r0 .. r0 + 15 at k slots kk * 32 + 8 g + j
    static __device__ __forceinline__ typename Mma<T>::v8 frag(const T *tile, int r0, int kk) {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
        if constexpr (KC) {
            const int row = r0 + c;
            if constexpr (sizeof(T) == 2) {
                return *reinterpret_cast<const typename Mma<T>::v8 *>(tile + row * BK + ((kk * 4 + g) ^ (row & 7)) * E);
            } else {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + row * BK + ((2 * g) ^ (row & 7)) * E);
                const f32x4 b = *reinterpret_cast<const f32x4 *>(tile + row * BK + ((2 * g + 1) ^ (row & 7)) * E);
                return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        } else if constexpr (sizeof(T) == 2) {
            const int k = kk * 32 + g * 8 + (c >> 2);             // and k + 4
            const int col = r0 + (c & 3) * 4;                     // 16 columns: one 32-byte granule
            const T *p = tile + k * R + ((((col >> 4) ^ granule(k)) << 4) | (col & 15));   // the same exchange for k + 4
            typedef typename Mma<T>::v4 v4;
            const v4 a = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p)));
            const v4 b = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p + 4 * R)));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typename Mma<T>::v8 v;
            const int col = r0 + c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = kk * 32 + g * 8 + j;
                v[j] = tile[k * R + ((((col >> 4) ^ granule32(k)) << 4) | (col & 15))];
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

// TM x TN 16x16 tiles per wave in each quadrant (A half x B half), WM x WN waves.  VEC: operands 16-byte
// aligned in rows of whole pieces.
template <typename T, int LAYOUT, int TM, int TN, int WM, int WN, bool VEC>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_gemm_kernel(const LinearGemm a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass, which cannot take the scalar operands, needs the stub alone
    constexpr int HM = TM * WM * 16, HN = TN * WN * 16, NW = WM * WN;     // rows and columns of a half
    constexpr bool AK = LAYOUT != LAYOUT_TN, BKC = LAYOUT == LAYOUT_NT;
    using TA = OperandTile<T, HM, NW, AK>;
    using TB = OperandTile<T, HN, NW, BKC>;
    using v8 = typename Mma<T>::v8;
    constexpr int BK = TA::BK, KK = BK / 32;
    __shared__ __attribute__((aligned(128))) T sa[VEC ? 2 : 1][2][TA::VALUES];    // [stage][half]
    __shared__ __attribute__((aligned(128))) T sb[VEC ? 2 : 1][2][TB::VALUES];
    const int64_t tm = (a.M + 2 * HM - 1) / (2 * HM), tn = (a.N + 2 * HN - 1) / (2 * HN);
    const bool whole = blockIdx.x < a.full;
    const int64_t piece = blockIdx.x - a.full;         // of the split tiles
    int64_t bm, bn;
    tile_of(whole ? blockIdx.x : a.full + piece / a.splits, tm, tn, bm, bn);
    const int64_t m0 = bm * 2 * HM, n0 = bn * 2 * HN;
    const int64_t k0 = whole ? 0 : piece % a.splits * a.kper, k1 = !whole && k0 + a.kper < a.K ? k0 + a.kper : a.K;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / WN) * TM * 16, wn = (wave % WN) * TN * 16;      // the wave's part of a half
    // first rows of the halves at the first k; steps of a stage
    const T *pa = static_cast<const T *>(a.A) + (AK ? m0 * a.lda + k0 : k0 * a.lda + m0);
    const T *pb = static_cast<const T *>(a.B) + (BKC ? n0 * a.ldb + k0 : k0 * a.ldb + n0);
    const int64_t a_half = AK ? HM * a.lda : HM, b_half = BKC ? HN * a.ldb : HN;
    const int64_t a_step = AK ? BK : BK * a.lda, b_step = BKC ? BK : BK * a.ldb;

    f32x4 acc[2][2][TM][TN];
#pragma unroll
    for (int i = 0; i < 4 * TM * TN; ++i) (&acc[0][0][0][0])[i] = f32x4{0, 0, 0, 0};
    auto read_a = [&](const T *t, v8 (&f)[KK][TM]) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int i = 0; i < TM; ++i) f[kk][i] = TA::frag(t, wm + i * 16, kk);
    };
    auto read_b = [&](const T *t, v8 (&f)[KK][TN]) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int j = 0; j < TN; ++j) f[kk][j] = TB::frag(t, wn + j * 16, kk);
    };
    auto multiply = [&](const v8 (&fa)[KK][TM], const v8 (&fb)[KK][TN], f32x4 (&o)[TM][TN]) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int p = 0; p < Mma<T>::kParts; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) o[i][j] = Mma<T>::mma(fb[kk][j], fa[kk][i], o[i][j], p);
    };
    v8 a0[KK][TM], a1[KK][TM], b0[KK][TN], b1[KK][TN];
    const int stages = (int)((k1 - k0 + BK - 1) / BK);
    TA ta[2];
    TB tb[2];
    if constexpr (VEC) {
        constexpr int L = TA::N + TB::N;      // loads of one half of each operand
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ta[h].prepare(a.lda, a.M - m0 - h * HM);
            tb[h].prepare(a.ldb, a.N - n0 - h * HN);
        }
        auto bring = [&](int s, int h, bool whole) __attribute__((always_inline)) {
            const int64_t left = k1 - k0 - (int64_t)s * BK;
            const int kl = whole || left >= BK ? BK : (int)left;
            ta[h].issue(pa + s * a_step + h * a_half, sa[s & 1][h], kl);
            tb[h].issue(pb + s * b_step + h * b_half, sb[s & 1][h], kl);
        };
        // one stage; more1, more2, more3: that many stages follow
        auto stage = [&](int s, bool more1, bool more2, bool more3) __attribute__((always_inline)) {
            const int at = s & 1;
            if (more1) wait_loads_and_barrier<2 * L>();     // A1, B1 of this stage have arrived
            else wait_loads_and_barrier<0>();
            read_b(sb[at][1], b1);
            if (more2) bring(s + 2, 0, more3);
            __builtin_amdgcn_sched_barrier(0);              // reads first: the products hide them
            multiply(a0, b0, acc[0][0]);
            __builtin_amdgcn_sched_barrier(0);
            read_a(sa[at][1], a1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(a0, b1, acc[0][1]);
            if (more2) wait_loads_and_barrier<2 * L>();     // A0, B0 of the next
            else if (more1) wait_loads_and_barrier<L>();
            if (more2) bring(s + 2, 1, more3);
            __builtin_amdgcn_sched_barrier(0);
            multiply(a1, b0, acc[1][0]);
            __builtin_amdgcn_sched_barrier(0);
            if (more1) read_a(sa[at ^ 1][0], a0);
            if (more1) read_b(sb[at ^ 1][0], b0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(a1, b1, acc[1][1]);
        };
        if (stages > 0) {
            bring(0, 0, false);
            bring(0, 1, false);
            if (stages > 1) {
                bring(1, 0, false);
                bring(1, 1, false);
                wait_loads_and_barrier<3 * L>();
            } else {
                wait_loads_and_barrier<L>();
            }
            read_a(sa[0][0], a0);
            read_b(sb[0][0], b0);
            int s = 0;
            for (; s + 3 < stages; ++s) stage(s, true, true, true);
            if (s + 2 < stages) stage(s++, true, true, false);
            if (s + 1 < stages) stage(s++, true, false, false);
            stage(s, false, false, false);
        }
    } else {
        uint4 ra[2][TA::N], rb[2][TB::N];
        auto fetch = [&](int s) __attribute__((always_inline)) {
            const int64_t left = k1 - k0 - (int64_t)s * BK;
            const int kl = left < BK ? (int)left : BK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ta[h].fetch(pa + s * a_step + h * a_half, a.lda, a.M - m0 - h * HM, kl, ra[h]);
                tb[h].fetch(pb + s * b_step + h * b_half, a.ldb, a.N - n0 - h * HN, kl, rb[h]);
            }
        };
        if (stages > 0) fetch(0);
        for (int s = 0; s < stages; ++s) {
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                TA::put(sa[0][h], ra[h]);
                TB::put(sb[0][h], rb[h]);
            }
            __syncthreads();
            if (s + 1 < stages) fetch(s + 1);
            read_a(sa[0][0], a0);
            read_b(sb[0][0], b0);
            multiply(a0, b0, acc[0][0]);
            read_b(sb[0][1], b1);
            multiply(a0, b1, acc[0][1]);
            read_a(sa[0][1], a1);
            multiply(a1, b1, acc[1][1]);
            multiply(a1, b0, acc[1][0]);
        }
    }
    if (!whole) {
        float *part = a.part + piece * (4 * HM * HN);
#pragma unroll
        for (int i = 0; i < 4 * TM * TN; ++i) {
            const int ha = i / (2 * TM * TN), hb = i / (TM * TN) % 2, r = i / TN % TM, j = i % TN;
            *reinterpret_cast<f32x4 *>(part + (ha * HM + wm + r * 16 + c) * (2 * HN) + hb * HN + wn + j * 16 + g * 4) = acc[ha][hb][r][j];
        }
        return;
    }
    if (a.quads) {
        // every row of every tensor in whole, aligned quads: 32-bit places in views of the tile, no branches
        struct Q { T v[4]; };
        const auto vc = wide_view(static_cast<T *>(a.C) + m0 * a.ldc + n0), vr = wide_view(static_cast<const T *>(a.res) + m0 * a.ldr + n0),
                   vp = wide_view(static_cast<T *>(a.pre) + m0 * a.ldp + n0), vb = wide_view(static_cast<const T *>(a.bias) + n0);
        const int rows = a.M - m0 < 2 * HM ? (int)(a.M - m0) : 2 * HM, cols = a.N - n0 < 2 * HN ? (int)(a.N - n0) : 2 * HN;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int col = hb * HN + wn + j * 16 + g * 4;
                const uint32_t x = (uint32_t)col * (uint32_t)sizeof(T);
                const Q qb = view_load_wide<Q>(vb, (a.bias != nullptr) & (col < cols) ? x : kSkip);
                float bias[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) bias[e] = (float)qb.v[e];
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const int row = ha * HM + wm + i * 16 + c;
                        const bool in = (row < rows) & (col < cols);
                        float f[4];
                        Q q;
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = acc[ha][hb][i][j][e] + bias[e];
                        if (a.pre) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) q.v[e] = (T)f[e];
                            view_store(vp, in ? (uint32_t)(row * (uint32_t)a.ldp) * (uint32_t)sizeof(T) + x : kSkip, q);
                        }
                        if (a.act != ACT_NONE) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e] = act_value<sizeof(T) == 4>(f[e], a.act);
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
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + ha * HM + wm + i * 16 + c;
            if (m >= a.M) continue;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int64_t n = n0 + hb * HN + wn + j * 16 + g * 4;
                    if (n >= a.N) continue;
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = acc[ha][hb][i][j][e];
                    linear_epilogue<T>(a, m, n, f);
                }
        }
#endif
}

// Joins the split tiles: sum of a tile's parts in their order (so results repeat bit by bit), then the
// epilogue.  grid: (tile rows / rows a workgroup takes, split tiles).  Bound by the parts: 64 tiles of 256 x 256
// in four (67 MB, from the last level cache): 15 us.
template <typename T, int TILE> __global__ __launch_bounds__(256) void linear_join_kernel(const LinearGemm a) {
    constexpr int kQuads = TILE / 4, kRows = 256 / kQuads;
    const int64_t tm = (a.M + TILE - 1) / TILE, tn = (a.N + TILE - 1) / TILE;
    int64_t bm, bn;
    tile_of(a.full + blockIdx.y, tm, tn, bm, bn);
    const int row = blockIdx.x * kRows + threadIdx.x / kQuads, col = threadIdx.x % kQuads * 4;
    const int64_t m = bm * TILE + row, n = bn * TILE + col;
    if (m >= a.M || n >= a.N) return;
    const float *p = a.part + (int64_t)blockIdx.y * a.splits * (TILE * TILE) + row * TILE + col;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) sum += *reinterpret_cast<const f32x4 *>(p + (int64_t)s * (TILE * TILE));
    float f[4] = {sum[0], sum[1], sum[2], sum[3]};
    linear_epilogue<T>(a, m, n, f);
}

// One to four rows: bound by the bytes of W (2560 -> 10240 in bf16, 52 MB: 11.0 us, 4.8 TB/s); more rows take the
// tile kernel.  A wave streams four rows of W, 16 bytes a lane, 1 KB of a row at a time, multiplies them
// with the rows of x in fp32 and joins its lanes at the end.
template <typename T, int M, bool VEC>
__global__ __launch_bounds__(256) void linear_vector_kernel(const LinearGemm a) {
    constexpr int E = 16 / (int)sizeof(T), R = 4, U = M == 1 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * R;
    if (n0 >= a.N) return;
    // VEC: value j of a lane's piece u is k0 + (u * 64 + lane) * E + j; else k0 + (u * E + j) * 64 + lane, value
    // by value.  Loads past K take an offset out of range instead of a branch, so all of a batch are on
    // their way together.
    struct Piece { T v[E]; };
    auto load = [&](const T *row, int64_t k0, int u) {
        const auto view = wide_view(row + k0);
        Piece q;
        if constexpr (VEC) {
            const int at = (u * 64 + lane) * E;
            q = view_load_wide<Piece>(view, k0 + at < a.K ? (uint32_t)at * (uint32_t)sizeof(T) : kSkip);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int at = (u * E + j) * 64 + lane;
                q.v[j] = view_load<T>(view, k0 + at < a.K ? (uint32_t)at * (uint32_t)sizeof(T) : kSkip);
            }
        }
        return q;
    };
    const T *pw[R], *px[M];
#pragma unroll
    for (int r = 0; r < R; ++r) pw[r] = static_cast<const T *>(a.B) + (n0 + r < a.N ? n0 + r : n0) * a.ldb;
#pragma unroll
    for (int m = 0; m < M; ++m) px[m] = static_cast<const T *>(a.A) + (m < a.M ? m : 0) * a.lda;
    float sum[R][M];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) sum[r][m] = 0.0f;
    for (int64_t k0 = 0; k0 < a.K; k0 += 64 * E * U) {
        Piece w[U][R], x[U][M];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) w[u][r] = load(pw[r], k0, u);
#pragma unroll
            for (int m = 0; m < M; ++m) x[u][m] = load(px[m], k0, u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int r = 0; r < R; ++r) sum[r][m] = fmaf((float)w[u][r].v[j], (float)x[u][m].v[j], sum[r][m]);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f[r] = sum[r][m];
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) f[r] += __shfl_xor(f[r], s);
        }
        if (lane == 0 && m < a.M) linear_epilogue<T>(a, m, n0, f);
    }
}

// dz and the column sums of slabs of rows.  grid: (columns / (32 V), slabs); thread: V neighbouring
// columns of every eighth row of the slab; the eight rows' sums are joined in LDS.  dz is rounded to the
// storage type, which the products that follow take; its sums are not.  Bound by memory: 8192 x 10240 in
// bf16 (503 MB): 120 us, 4.2 TB/s.  Kept apart from the products: fused into both their loads it would be
// computed, with its activation's slope, once per tile of the other side, 10 to 40 times.
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
                    const float f = (float)d[u].v[j] * (a.act != ACT_NONE ? act_slope<sizeof(T) == 4>((float)z[u].v[j], a.act) : 1.0f);
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
// Sums of the slabs' sums: 16 columns x 16 shares of the slabs a workgroup, joined in a fixed order.  A launch:
// 2.6 to 5 us.
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
    const unsigned grid = (unsigned)(a.full + (a.tiles - a.full) * a.splits);
    if (!vec) {
        linear_gemm_kernel<T, LAYOUT, 2, 2, 2, 2, false><<<grid, 256, 0, stream>>>(a);
    } else if (tile == 256) {
        if constexpr (sizeof(T) == 2) linear_gemm_kernel<T, LAYOUT, 4, 2, 2, 4, true><<<grid, 512, 0, stream>>>(a);
    } else if (tile == 128) {
        linear_gemm_kernel<T, LAYOUT, 2, 2, 2, 2, true><<<grid, 256, 0, stream>>>(a);
    } else {
        linear_gemm_kernel<T, LAYOUT, 1, 1, 2, 2, true><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t gemm_typed(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t stream) {
    hipError_t e = layout == LAYOUT_NT   ? gemm_layout<T, LAYOUT_NT>(a, tile, vec, stream)
                   : layout == LAYOUT_NN ? gemm_layout<T, LAYOUT_NN>(a, tile, vec, stream)
                                         : gemm_layout<T, LAYOUT_TN>(a, tile, vec, stream);
    const unsigned split = (unsigned)(a.tiles - a.full);
    if (e != hipSuccess || split == 0) return e;
    const dim3 grid((unsigned)(tile * tile / 1024), split);
    if (tile == 256) linear_join_kernel<T, 256><<<grid, 256, 0, stream>>>(a);
    else if (tile == 128) linear_join_kernel<T, 128><<<grid, 256, 0, stream>>>(a);
    else linear_join_kernel<T, 64><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, bool VEC> static hipError_t vector_typed(const LinearGemm &a, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.N + 15) / 16);
    if (a.M == 1) linear_vector_kernel<T, 1, VEC><<<grid, 256, 0, stream>>>(a);
    else if (a.M == 2) linear_vector_kernel<T, 2, VEC><<<grid, 256, 0, stream>>>(a);
    else linear_vector_kernel<T, 4, VEC><<<grid, 256, 0, stream>>>(a);
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
    hipError_t launch_linear_vector_##NAME(const LinearGemm &a, bool vec, hipStream_t s) {                       \
        return vec ? vector_typed<T, true>(a, s) : vector_typed<T, false>(a, s);                                 \
    }                                                                                                            \
    hipError_t launch_linear_dz_##NAME(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t s) {           \
        return dz_typed<T>(a, slabs, dbias, s);                                                                  \
    }

}  // namespace fftconv
