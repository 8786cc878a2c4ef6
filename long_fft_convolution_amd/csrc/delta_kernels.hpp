// delta_kernels.hpp -- the gated delta rule: prompts, gradients and single
// tokens.  Instantiated per storage type by delta_f16.hip, delta_bf16.hip and
// delta_f32.hip.
//
// Mathematics.  Per sequence and head, with a_t = exp(log_decay_t) and an
// fp32 state S (Dk x Dv),
//
//     w_t = v_t - a_t S_{t-1}^T k_t,  u_t = beta_t w_t,  S_t = a_t S_{t-1} + k_t u_t^T,  out_t = scale S_t^T q_t.
//
// Over a chunk of C = 64 tokens that starts from S, with G_i the sum of the
// logarithms up to token i of the chunk, C_ij = exp(G_i - G_j) k_i . k_j for
// j < i and P_ij = scale exp(G_i - G_j) q_i . k_j for j <= i,
//
//     r_i = v_i - exp(G_i) S^T k_i,   (I + C diag(beta)) w = r,   u = beta w,
//     out_i = scale exp(G_i) S^T q_i + sum_j P_ij u_j,
//     S <- exp(G_last) S + sum_j k_j (exp(G_last - G_j) u_j)^T.
//
// The inverse of I + C diag(beta) and P need no state: a first kernel computes
// them for all chunks at once (delta_prepare_kernel).  What is left is serial
// over the chunks and independent over the state's columns: one workgroup of
// four or eight waves walks one (sequence or segment, head, 64 or 128 columns),
// each wave with its 16 columns of S in its accumulators for the whole walk.  r, w and
// u never leave the registers: the accumulators of a product over tokens are
// the next product's operand when its contraction index is met in the order
// token(slot 8 g + j) = 32 s + 16 (j / 4) + 4 g + j % 4, which is the order the
// inverse and P are stored in.  Only k, q, v come through LDS.
//
// A call with few (sequence, head) pairs cuts sequences into segments.  A
// segment is an affine map of the state before it, so a first walk finds its
// own sum (from a zero state) and its map (from the unit matrix, without
// values: Dk more columns), a small kernel chains them into the state before
// each segment, and the walk with outputs starts from there.
//
// Rounding.  The state is an fp32 result over the whole sequence, so nothing
// on its way may lose: all operands are exact sums of bf16 terms (an fp32
// value: three, fp16: two, bf16: itself) and the products of terms i + j < 3
// are taken, which drops 2^-24 of a product.  bf16 terms have fp32's range, so
// nothing is scaled, fp16 included, and bf16 products are the fastest there
// are.  Outputs in 16 bits see the state, u and P in two terms each (2^-15 of a
// value, beside the result's own rounding of 2^-8 or 2^-11).  The sums G are
// 64 bits: behind a token that clears the state (a logarithm below -104, exp
// = 0) the differences of the tokens that follow keep all their bits.
#pragma once

#include "delta_ops.hpp"
#include "sequence_device.hpp"

namespace fftconv {

constexpr int kC = kDeltaChunk, kLdsBytes = 160 * 1024;
typedef Mma<__bf16>::v8 bf8;

// ---- sequences, chunks, segments -------------------------------------------
struct Tokens {
    int64_t seq, start, len;     // sequence, its first token, its length
    int64_t unit;                // chunk or segment of it
    int64_t row0, batch;         // tensors start at (batch, row0)
};
__device__ __forceinline__ void sequence_bounds(const DeltaArgs &a, int64_t b, int64_t &start, int64_t &len) {
    if (!a.cu) {
        start = 0, len = a.N;
        return;
    }
    // bounds come from device memory: clamped to the tokens there are
    int64_t s = a.cu[b], e = a.cu[b + 1];
    s = s < 0 ? 0 : (s > a.N ? a.N : s);
    e = e < s ? s : (e > a.N ? a.N : e);
    start = s, len = e - s;
}
// Place of sequence b's first unit of `length` tokens.  Packed sequences: no two meet, since
// start / length + ceil(len / length) <= (start + len) / length + 1; an empty one has a place of its own too.
__device__ __forceinline__ int64_t first_place(const DeltaArgs &a, int64_t b, int64_t length) {
    if (!a.cu) return b * (a.N > 0 ? (a.N + length - 1) / length : 1);
    int64_t start, len;
    sequence_bounds(a, b, start, len);
    return start / length + b;
}
// The sequence and unit at a place; false when there is none.  An empty sequence has unit 0.
__device__ __forceinline__ bool unit_at(const DeltaArgs &a, int64_t place, int64_t length, Tokens &t) {
    int64_t lo = 0, hi = a.B - 1;
    if (!a.cu) {
        const int64_t per = a.N > 0 ? (a.N + length - 1) / length : 1;
        lo = place / per;
        if (lo >= a.B) return false;
    } else {
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (first_place(a, mid, length) <= place) lo = mid;
            else hi = mid - 1;
        }
    }
    t.seq = lo;
    sequence_bounds(a, lo, t.start, t.len);
    t.unit = place - first_place(a, lo, length);
    t.row0 = a.cu ? t.start : 0;
    t.batch = a.cu ? 0 : t.seq;
    return t.unit >= 0 && (t.unit == 0 || t.unit * length < t.len);
}
__device__ __forceinline__ void make_scalar(Tokens &t) {
    t.seq = scalar(t.seq), t.start = scalar(t.start), t.len = scalar(t.len), t.unit = scalar(t.unit);
    t.row0 = scalar(t.row0), t.batch = scalar(t.batch);
}

// ---- operands ---------------------------------------------------------------
// bf16 terms of a storage value (exact), and of what the outputs see: the state, u and the masked products
template <typename T> struct Terms;
template <> struct Terms<__bf16> { static constexpr int kIn = 1, kOut = delta_terms(2); };
template <> struct Terms<_Float16> { static constexpr int kIn = 2, kOut = delta_terms(2); };
template <> struct Terms<float> { static constexpr int kIn = 3, kOut = delta_terms(4); };

// Eight fp32 values as N bf16 terms.  bf16 is the upper half of fp32: cutting it off leaves an exact rest, so three
// terms of 8 bits hold all 24; the last of two is rounded.  (The rests as dot products of a pair with (-1, 0) and (0, -1)
// are fewer instructions, but those wait for the matrix unit and it for them: 33 cycles for a product and two of them,
// 19 for a product and two ordinary ones.)
template <int N> __device__ __forceinline__ void split_terms(const float (&x)[8], bf8 (&out)[N]) {
    if constexpr (N == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[0][j] = (__bf16)x[j];
    } else {
        split8<__bf16, N>(x, out);
    }
}
template <typename T> struct Raw8 { T v[8]; };
template <typename T> __device__ __forceinline__ void in_terms(const Raw8<T> &x, bf8 (&out)[Terms<T>::kIn]) {
    if constexpr (sizeof(T) == 2 && Terms<T>::kIn == 1) {
        out[0] = __builtin_bit_cast(bf8, x);
    } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)x.v[j];
        split_terms(f, out);
    }
}
// two accumulators of rows 16 (2 s) and 16 (2 s + 1) as the operand over their 32 rows
template <int N> __device__ __forceinline__ void rows_terms(const f32x4 &a, const f32x4 &b, bf8 (&out)[N]) {
    float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    split_terms(f, out);
}
// acc += sum of the products of terms i + j < MOST
template <int MOST, int NA, int NB> __device__ __forceinline__ f32x4 mma_terms(const bf8 (&a)[NA], const bf8 (&b)[NB], f32x4 acc) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < MOST) acc = Mma<__bf16>::mma(a[i], b[j], acc);
    return acc;
}

// exp of a 64-bit difference to fp32 precision: the part that fp32 does not hold as a factor 1 + lo
__device__ __forceinline__ float exp_of(double d) {
    const float hi = (float)d, lo = (float)(d - (double)hi);
    const float e = expf(hi);
    return __builtin_fmaf(e, lo, e);
}

// 8 values of a row at byte offset `at` (or kSkip), of which `left` exist
template <typename T, bool VEC> __device__ __forceinline__ Raw8<T> load_row8(__amdgpu_buffer_rsrc_t view, uint32_t at, int left) {
    Raw8<T> r;
    if constexpr (VEC) {
        const uint32_t o = left > 0 ? at : kSkip;
        if constexpr (sizeof(T) == 2) {
            r = __builtin_bit_cast(Raw8<T>, view_load_wide<u32x4>(view, o));
        } else {
            const u32x4 a = view_load_wide<u32x4>(view, o), b = view_load_wide<u32x4>(view, left > 4 && o != kSkip ? o + 16 : kSkip);
            __builtin_memcpy(&r, &a, 16);
            __builtin_memcpy(reinterpret_cast<char *>(&r) + 16, &b, 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = view_load<T>(view, ((j < left) & (at != kSkip)) ? at + j * (uint32_t)sizeof(T) : kSkip);
    }
    return r;
}

// A token whose logarithm is below this clears the state before it: its decay is 0 in fp32.
constexpr float kClears = -104.0f;
// The caller's state of a sequence and head or null, and whether the sequence's first token (its row in log_decay) clears
// it: products with 0 would keep a NaN or infinity of it.
__device__ __forceinline__ const float *first_state(const DeltaArgs &a, int64_t seq, int64_t token, int64_t len, int h, bool &cleared) {
    cleared = a.state0 && len > 0 && a.log_decay[token * a.H + h] < kClears;
    if (!a.state0) return nullptr;
    const int64_t slot = state_slot(a.slots, a.n_slots, seq);
    return slot >= 0 ? a.state0 + (slot * a.H + h) * (int64_t)a.Dk * a.Dv : nullptr;
}

// Ends a wave's LDS writes before its reads of them by other lanes.
__device__ __forceinline__ void wave_sync() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// ---- the part without state ---------------------------------------------------
constexpr int kLd = kC + 4;      // row stride of a 64 x 64 matrix in LDS: 16-byte rows, columns on all banks

// M (strictly lower, 64 x 64 in LDS) <- (I + M)^-1, lower blocks of 16; the blocks above the diagonal are left.
// Diagonal blocks by forward substitution, a column a lane; the others, row of blocks by row, as
// -T_ii sum_k M_ik T_kj on the fp32 matrix cores.  Rows from n on are those of the unit matrix.
__device__ __forceinline__ void invert_unit_lower(float *M, int n) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    {
        const float *block = M + g * 16 * kLd + g * 16;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4 m = *reinterpret_cast<const f32x4 *>(block + i * kLd + j4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j4 + j < i) s -= m[j] * t[j4 + j];
            }
            t[i] = s;
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 16; ++i) M[(g * 16 + i) * kLd + g * 16 + c] = t[i];
        wave_sync();
    }
    auto row4 = [&](int i, int k) { return *reinterpret_cast<const f32x4 *>(M + (16 * i + c) * kLd + 16 * k + 4 * g); };
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        if (16 * i >= n) return;
        f32x4 x[3];
#pragma unroll
        for (int j = 0; j < i; ++j) {
            x[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = j; k < i; ++k) {
                const f32x4 m = row4(i, k);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    x[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[s], M[(16 * k + 4 * g + s) * kLd + 16 * j + c], x[j], 0, 0, 0);
            }
        }
        const f32x4 d = row4(i, i);
        wave_sync();
#pragma unroll
        for (int j = 0; j < i; ++j) {
            f32x4 t = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < 4; ++s) t = __builtin_amdgcn_mfma_f32_16x16x4f32(d[s], x[j][s], t, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) M[(16 * i + 4 * g + r) * kLd + 16 * j + c] = -t[r];
        }
        wave_sync();
    }
}

// One wave a (chunk, head): record of the chunk.  grid: chunks * H / 4.  Bound by latency (products, the inverse's 16
// serial steps, LDS round trips; eight waves a CU overlap them) and, for long calls, by the records written.  20 heads of
// 128, bf16: 4 x 4096 tokens 91 us, 131072 tokens 605 us (2.7 GB, 4.4 TB/s).  A chunk that ends early has fewer blocks to
// invert (17 tokens: 14.3 us, 16.6 with all of them).
// BACK: the backward call's record (4 x 4096 tokens: 145 to 155 us).
template <typename T, int DXP, bool VEC, bool BACK> __global__ __launch_bounds__(256) void delta_prepare_kernel(const DeltaArgs a) {
    constexpr int KX = DXP / 32, NP = Terms<T>::kOut;
    __shared__ __attribute__((aligned(16))) float matrix[4][kC * kLd];
    __shared__ double sums[4][kC];
    __shared__ float betas[4][kC];
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t item = blockIdx.x * (int64_t)4 + wave;
    if (item >= a.chunks * a.H) return;
    const int64_t place = item / a.H;
    const int h = (int)(item % a.H);
    Tokens t;
    if (!unit_at(a, place, kC, t)) return;
    make_scalar(t);
    const int64_t t0 = t.unit * kC;
    const int n = t.len - t0 < kC ? (int)(t.len - t0) : kC;
    if (n <= 0) return;
    float *M = matrix[wave];
    double *G = sums[wave];
    float *beta = betas[wave];

    // a token a lane: sums of the logarithms, weights
    const int64_t gate = (t.batch * a.N + t.row0 + t0 + lane) * a.H + h;
    float own = lane < n ? a.log_decay[gate] : 0.0f;
    own = own < -128.0f ? -128.0f : own;       // exp of either is 0 in fp32, and the sums stay finite
    const float b = lane < n ? a.beta[gate] : 0.0f;
    double sum = own;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const double up = __shfl_up(sum, s);
        if (lane >= s) sum += up;
    }
    const double last = __shfl(sum, 63);
    G[lane] = sum;
    beta[lane] = b;
    char *rec = a.rec + item * a.rec_bytes;
    {
        float *vec = reinterpret_cast<float *>(rec + kDeltaInverse * 1024);
        const float first = exp_of(sum);
        vec[lane] = first;
        vec[64 + lane] = exp_of(last - sum);
        vec[128 + lane] = b;
        vec[192 + lane] = a.scale * first;
    }
    wave_sync();

    // products of keys (rows i, columns j <= i) and of keys with queries (rows j, columns i)
    f32x4 kk[10], qk[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) kk[i] = qk[i] = f32x4{0, 0, 0, 0};
    {
        const T *k0 = static_cast<const T *>(a.k) + t.batch * a.kb + (t.row0 + t0) * a.kt + (h / a.group) * a.kh;
        const T *q0 = static_cast<const T *>(a.q) + t.batch * a.qb + (t.row0 + t0) * a.qt + (h / a.group) * a.qh;
        const auto kv = wide_view(k0), qv = wide_view(q0);
#pragma unroll 1
        for (int s = 0; s < KX; ++s) {
            const int col = s * 32 + g * 8, left = a.Dk - col;
            bf8 kf[4][Terms<T>::kIn], qf[4][Terms<T>::kIn];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * r + c;
                in_terms(load_row8<T, VEC>(kv, row < n ? (uint32_t)((row * a.kt + col) * (int64_t)sizeof(T)) : kSkip, row < n ? left : 0), kf[r]);
                in_terms(load_row8<T, VEC>(qv, row < n ? (uint32_t)((row * a.qt + col) * (int64_t)sizeof(T)) : kSkip, row < n ? left : 0), qf[r]);
            }
#pragma unroll
            for (int i = 0, at = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j, ++at) {
                    kk[at] = mma_terms<3>(kf[i], kf[j], kk[at]);
                    // BACK: rows i, columns j
                    qk[at] = BACK ? mma_terms<3>(qf[i], kf[j], qk[at]) : mma_terms<3>(kf[j], qf[i], qk[at]);
                }
        }
    }
    // decayed products of keys into LDS, weighted by beta of their column (I + C diag(beta)) or of their row
    auto put = [&](bool by_row) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0, at = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j, ++at)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 4 * g + r, col = 16 * j + c;
                    M[row * kLd + col] = col < row ? kk[at][r] * exp_of(G[row] - G[col]) * beta[by_row ? row : col] : 0.0f;
                }
        wave_sync();
        invert_unit_lower(M, n);
    };
    put(false);
    bf8 *out = reinterpret_cast<bf8 *>(rec);
    bf8 *outp = reinterpret_cast<bf8 *>(rec + (kDeltaInverse + kDeltaVectors) * 1024);
#pragma unroll
    for (int i = 0, e = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s <= i / 2; ++s, ++e) {
            float p[8];
            f32x4 m[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int j = 2 * s + half;      // block of columns
                m[half] = j <= i ? *reinterpret_cast<const f32x4 *>(M + (16 * i + c) * kLd + 16 * j + 4 * g) : f32x4{0, 0, 0, 0};
                if constexpr (!BACK) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * i + c, col = 16 * j + 4 * g + r;
                        const f32x4 x = qk[j <= i ? i * (i + 1) / 2 + j : 0];
                        p[half * 4 + r] = ((j <= i) & (col <= row)) ? x[r] * a.scale * exp_of(G[row] - G[col <= row ? col : row]) : 0.0f;
                    }
                }
            }
            bf8 mt[3];
            rows_terms<3>(m[0], m[1], mt);
#pragma unroll
            for (int u = 0; u < 3; ++u) out[(e * 3 + u) * 64 + lane] = mt[u];
            if constexpr (!BACK) {
                bf8 terms[NP];
                rows_terms<NP>(f32x4{p[0], p[1], p[2], p[3]}, f32x4{p[4], p[5], p[6], p[7]}, terms);
#pragma unroll
                for (int u = 0; u < NP; ++u) outp[(e * NP + u) * 64 + lane] = terms[u];
            }
        }
    if constexpr (BACK) {
        // (I + diag(beta) C)^-1 and P by columns: lane (g, c) holds column 16 j + c at the rows of the operand's slots
        wave_sync();
        put(true);
        f32x4 *outt = reinterpret_cast<f32x4 *>(outp + kDeltaInverse * 64);
#pragma unroll
        for (int j = 0, e = 0; j < 4; ++j)
#pragma unroll
            for (int s = j / 2; s < 2; ++s, ++e) {
                f32x4 m[2], p[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = 2 * s + half;
                    m[half] = p[half] = f32x4{0, 0, 0, 0};
                    if (i >= j) {
                        const f32x4 x = qk[i * (i + 1) / 2 + j];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = 16 * i + 4 * g + r, col = 16 * j + c;
                            m[half][r] = col <= row ? M[row * kLd + col] : 0.0f;
                            p[half][r] = col <= row ? x[r] * a.scale * exp_of(G[row] - G[col <= row ? col : row]) : 0.0f;
                        }
                    }
                    outt[(e * 2 + half) * 64 + lane] = p[half];
                }
                bf8 mt[3];
                rows_terms<3>(m[0], m[1], mt);
#pragma unroll
                for (int u = 0; u < 3; ++u) outp[(e * 3 + u) * 64 + lane] = mt[u];
            }
    }
}

// ---- tiles in LDS ------------------------------------------------------------
// 64 rows of DP values in 16-byte slots, slot s of row r lying at s ^ f(r): eight neighbouring rows of a slot, and
// four rows of four neighbouring slots, then lie on different banks.
template <typename T, int DP, int WAVES> struct RowTile {
    static constexpr int E = 16 / (int)sizeof(T), PR = DP / E, N = kC * PR / (WAVES * 64), BYTES = kC * DP * (int)sizeof(T);
    static_assert(kC * PR % (WAVES * 64) == 0 && PR % 8 == 0, "whole loads");
    static __device__ __forceinline__ int f(int row) { return (row & 1) << 2 | (row & 2) | ((row >> 2) & 1); }
};
// Brings a tensor's rows into a tile: VEC by LDS-destination loads (what lies outside the chunk or the columns reads
// zero by the buffer unit's range check), else value by value.
template <typename T, int DP, int WAVES, bool VEC> struct RowSource {
    using Tile = RowTile<T, DP, WAVES>;
    const T *p;            // the sequence's first row
    int64_t stride;
    int cols, col0;
    __device__ __forceinline__ void init(const void *base, int64_t off, int64_t st, int cols_, int col0_) {
        p = static_cast<const T *>(base) + off;
        stride = st, cols = cols_, col0 = col0_;
    }
    // n of the rows from token t on; the rest of the tile becomes zero
    __device__ __forceinline__ void bring(int64_t t, int n, T *tile) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const T *first = p + t * stride;
#pragma unroll
        for (int i = 0; i < Tile::N; ++i) {
            const int idx = i * WAVES * 64 + threadIdx.x, row = idx / Tile::PR, slot = idx % Tile::PR ^ Tile::f(row);
            const int col = col0 + slot * Tile::E;
            const uint32_t at = (uint32_t)((row * stride + col) * (int64_t)sizeof(T));
            if constexpr (VEC) {
                lds_load16(first, tile + (i * WAVES * 64 + wave * 64) * Tile::E, ((row < n) & (col < cols)) ? at : kSkip);
            } else {
                const auto view = wide_view(first);
                T e[Tile::E];
#pragma unroll
                for (int j = 0; j < Tile::E; ++j)
                    e[j] = view_load<T>(view, ((row < n) & (col + j < cols)) ? at + j * (uint32_t)sizeof(T) : kSkip);
                __builtin_memcpy(tile + idx * Tile::E, e, 16);
            }
        }
    }
};
// `pieces` KB of a record as they are
template <int WAVES, bool VEC> __device__ __forceinline__ void bring_record(const char *rec, int pieces, char *dst) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    for (int i = wave; i < pieces; i += WAVES) {
        if constexpr (VEC) lds_load16(rec, dst + i * 1024, (uint32_t)(i * 1024 + lane * 16));
        else *reinterpret_cast<f32x4 *>(dst + i * 1024 + lane * 16) = *reinterpret_cast<const f32x4 *>(rec + i * 1024 + lane * 16);
    }
}

// Where a wave's operands lie in a tile, as byte offsets of this lane: what the swizzle makes of the lane is in a few
// bases, the rest of an address is a constant of the instruction.
template <typename T, int DP, int WAVES> struct TileReader {
    using Tile = RowTile<T, DP, WAVES>;
    static constexpr int RB = DP * (int)sizeof(T);
    uint32_t row[2], col[sizeof(T) == 2 ? 2 : 8];
    __device__ __forceinline__ void init() {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            row[p] = c * RB + ((sizeof(T) == 2 ? 4 * p + g : 2 * g + p) ^ Tile::f(c)) * 16;
            if constexpr (sizeof(T) == 2) {
                const int r = 4 * g + (c >> 2);
                col[p] = r * RB + ((4 * p + (c & 3)) ^ Tile::f(r)) * 16;
            }
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    col[2 * j + r] = (4 * g + j) * RB + (((c >> 2) * 2 + r) ^ Tile::f(4 * g + j)) * 16 + (c & 3) * 4;
        }
    }
    // columns 32 kk + 8 g .. + 7 of row 16 r + c
    __device__ __forceinline__ Raw8<T> row8(const char *tile, int r, int kk) const {
        Raw8<T> v;
        if constexpr (sizeof(T) == 2) {
            v = *reinterpret_cast<const Raw8<T> *>(__builtin_assume_aligned(tile + row[kk & 1] + (kk >> 1) * 128 + r * 16 * RB, 16));
        } else {
#pragma unroll
            for (int p = 0; p < 2; ++p)
                __builtin_memcpy(reinterpret_cast<char *>(&v) + 16 * p, __builtin_assume_aligned(tile + row[p] + kk * 128 + r * 16 * RB, 16), 16);
        }
        return v;
    }
    // column 32 kk + 8 (c / 4) + 4 r + c % 4 of the rows of an operand over tokens 32 s .. 32 s + 31.  16 bits:
    // transposing reads, in which 16 lanes read four rows of four 4-column groups and lane c receives column c % 4 of
    // group c / 4.
    __device__ __forceinline__ Raw8<T> col8(const char *tile, int s, int kk, int r) const {
        Raw8<T> v;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int rows = (32 * s + 16 * half) * RB;
            if constexpr (sizeof(T) == 2) {
                const char *p = tile + col[kk & 1] + (kk >> 1) * 128 + r * 8 + rows;
                const s16x4 x = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, const_cast<char *>(p))));
                __builtin_memcpy(v.v + 4 * half, &x, 8);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v.v[4 * half + j] = *reinterpret_cast<const T *>(tile + col[2 * j + r] + kk * 128 + rows);
            }
        }
        return v;
    }
};
// The same of a wave's own 16 columns: rows 16 r + 4 g .. + 3 of column 16 wave + c.
template <typename T, int DP, int WAVES> struct ColumnReader {
    using Tile = RowTile<T, DP, WAVES>;
    static constexpr int RB = DP * (int)sizeof(T);
    uint32_t col[sizeof(T) == 2 ? 1 : 4];
    __device__ __forceinline__ void init(int wave) {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
        if constexpr (sizeof(T) == 2) {
            const int r = 4 * g + (c >> 2);
            col[0] = r * RB + ((2 * wave + ((c & 3) >> 1)) ^ Tile::f(r)) * 16 + (c & 1) * 8;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) col[j] = (4 * g + j) * RB + ((4 * wave + (c >> 2)) ^ Tile::f(4 * g + j)) * 16 + (c & 3) * 4;
        }
    }
    __device__ __forceinline__ void col4(const char *tile, int r, T *out) const {
        if constexpr (sizeof(T) == 2) {
            const char *p = tile + col[0] + r * 16 * RB;
            const s16x4 x = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, const_cast<char *>(p))));
            __builtin_memcpy(out, &x, 8);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = *reinterpret_cast<const T *>(tile + col[j] + r * 16 * RB);
        }
    }
};

// ---- the state in a wave's accumulators ------------------------------------------
// Place of an element in a matrix kept for the gradients, which read it 32 columns at a time: blocks of 32 columns of all
// `rows`.
__device__ __forceinline__ uint32_t kept_at(int row, int col, int rows) { return (uint32_t)((col >> 5) * rows * 32 + row * 32 + (col & 31)); }

// v[kk][r]: rows kk * 32 + g * 8 + r * 4 + i of the column of lane (g, c): as an operand over rows, the lane holds the
// slots 8 g + j of its column.
template <int KX> struct State {
    f32x4 v[KX][2];
    template <typename F> __device__ __forceinline__ void each(F &&f) {
#pragma unroll
        for (int kk = 0; kk < KX; ++kk)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[kk][r][i] = f(kk * 32 + (int)((threadIdx.x & 63) >> 4) * 8 + r * 4 + i, v[kk][r][i]);
    }
    // of a row-major matrix of rows x cols (null: zeros)
    __device__ __forceinline__ void load(const float *p, int rows, int cols, int col) {
        const auto view = wide_view(p);
        each([&](int row, float) __attribute__((always_inline)) {
            return view_load<float>(view, ((p != nullptr) & (row < rows) & (col < cols)) ? (uint32_t)(row * cols + col) * 4u : kSkip);
        });
    }
    // Ends the loads before a loop: waits for them inside it would come with every round, and loads retire in order, so
    // that each would wait for the next chunk's.
    __device__ __forceinline__ void settle() {
        each([&](int, float x) __attribute__((always_inline)) {
            asm volatile("" : "+v"(x));
            return x;
        });
    }
    __device__ __forceinline__ void store(float *p, int rows, int cols, int col) {
        const auto view = wide_view(p);
        each([&](int row, float x) __attribute__((always_inline)) {
            view_store(view, ((row < rows) & (col < cols)) ? (uint32_t)(row * cols + col) * 4u : kSkip, x);
            return x;
        });
    }
    // into a matrix of padded rows, whose padding it fills with what padding gives: zeros
    __device__ __forceinline__ void keep(float *p, int ld, int col) {
        const auto view = wide_view(p);
        each([&](int row, float x) __attribute__((always_inline)) {
            view_store(view, (uint32_t)(row * ld + col) * 4u, x);
            return x;
        });
    }
    // into a matrix kept for the gradients
    __device__ __forceinline__ void keep_blocks(float *p, int col) {
        const auto view = wide_view(p);
        each([&](int row, float x) __attribute__((always_inline)) {
            view_store(view, kept_at(row, col, KX * 32) * 4u, x);
            return x;
        });
    }
    __device__ __forceinline__ void terms(int kk, bf8 (&out)[3]) const { rows_terms<3>(v[kk][0], v[kk][1], out); }
};
// accumulators over tokens (rows 16 r + 4 g + i) into a matrix kept for the gradients
__device__ __forceinline__ void keep_rows(float *p, const f32x4 (&x)[4], int col) {
    const auto view = wide_view(p);
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) view_store(view, kept_at(16 * r + 4 * g + i, col, kC) * 4u, x[r][i]);
}

// Work item of workgroup id: ids go to the 8 XCDs in turn, so runs of `run` items are dealt to one XCD, whose L2
// then holds what they have in common.
__device__ __forceinline__ uint32_t dealt(uint32_t id, uint32_t run) {
    const uint32_t round = id / (8 * run), in = id % (8 * run);
    return (round * 8 + in % 8) * run + in / 8;
}
inline __host__ __device__ int delta_run(int tiles, int group) {
    const int n = tiles * group;
    return n < 16 ? n : 16;
}

// MODE kDeltaSums: a segment's own sum and map, of those that another follows; kDeltaOut: outputs; kDeltaKeep: for
// the backward call, the state before each chunk and w.
enum DeltaMode : int { kDeltaSums = 0, kDeltaOut = 1, kDeltaKeep = 2 };

// Waves a SIMD that the compiler leaves registers for: the sums' walks, which cut sequences into twice as many pieces as
// walk at once, share a CU (131072 tokens x 20 heads of 128: 1380 us, 1555 with one of two stages).
constexpr int walk_waves(int dxp, int waves, int mode, int bytes) { return mode == kDeltaSums && bytes == 2 && dxp <= 128 ? waves / 2 : 1; }

// Eight waves a workgroup, two a SIMD (one splits fp32 values while the other multiplies), for 128 columns; four for 64.
// Bound by the serial chunk: its products, splits and LDS reads each take two to three microseconds of it, in turns.
// 20 heads of 128, bf16: 4 x 4096 tokens 245 us (64 columns, 3.8 us a chunk), one sequence of 6001 among shorter ones 443
// us (128 columns, 4.7 us a chunk), 131072 tokens in 12 segments: sums and maps 1380 us, outputs 990 us.  fp16, fp32:
// 452 and 718 us at 4 x 4096.  32 columns a wave took 1032 us for those outputs, and 2213 us for the sums.
template <typename T, int DXP, int WAVES, int MODE, bool VEC> struct WalkShape {
    static constexpr bool OUT = MODE == kDeltaOut;
    static constexpr int DZT = WAVES * 16;
    using TX = RowTile<T, DXP, WAVES>;
    using TZ = RowTile<T, DZT, WAVES>;
    static constexpr int kQ = TX::BYTES, kV = (OUT ? 2 : 1) * TX::BYTES, kRec = kV + TZ::BYTES;
    // where LDS has no room (fp32 rows wider than 128) the record, or its masked products, are read from memory
    static constexpr int kAll = OUT ? delta_pieces(Terms<T>::kOut) : 20, kFew = kDeltaInverse + kDeltaVectors + 1;
    static constexpr int kPieces = kRec + kAll * 1024 <= kLdsBytes ? kAll : kRec + kFew * 1024 <= kLdsBytes ? kFew : 0;
    static constexpr bool kRecord = kPieces > 0, kProducts = kPieces >= kAll;
    static constexpr int kBytes = kRec + kPieces * 1024;
    // (sums: two workgroups a CU, one of which loads while the other multiplies)
    static constexpr bool kShared = walk_waves(DXP, WAVES, MODE, sizeof(T)) > 1;
    static constexpr int kStages = VEC && 2 * kBytes <= kLdsBytes && !kShared ? 2 : 1;
    static_assert(kBytes <= kLdsBytes, "LDS");
};

// Threads that the walks are compiled for: with 512 the accumulators stay among the 256 registers that all instructions
// reach; four waves of rows up to 128 fit those, too, and moves to and from the other half would cost a tenth of them.
constexpr int walk_bound(int dxp, int waves, int bytes) { return dxp <= 128 && bytes == 2 ? 512 : waves * 64; }

#ifdef __HIP_DEVICE_COMPILE__   // the host pass cannot take the loads' scalar operands and needs the kernels' stubs alone
// w: the work item, of `tiles` column tiles (the first `ztiles` of values) x heads x places
template <typename T, int DXP, int WAVES, int MODE, bool VEC>
__device__ __forceinline__ void delta_walk(const DeltaArgs &a, char *lds, uint32_t w, int ztiles, int tiles) {
    using W = WalkShape<T, DXP, WAVES, MODE, VEC>;
    constexpr bool OUT = W::OUT;
    constexpr int KX = DXP / 32, DZT = W::DZT, NIN = Terms<T>::kIn, NOUT = Terms<T>::kOut;
    const int tile = w % tiles;
    w /= tiles;
    const int h = w % a.H;
    const int64_t place = w / a.H;
    if (place >= a.segs) return;
    Tokens tk;
    if (!unit_at(a, place, a.seg_chunks * kC, tk)) return;
    make_scalar(tk);
    const int64_t chunks = (tk.len + kC - 1) / kC, first = tk.unit * a.seg_chunks;
    const int64_t end = first + a.seg_chunks < chunks ? first + a.seg_chunks : chunks;
    const bool last = end >= chunks;
    if (MODE == kDeltaSums && last) return;
    const bool map = MODE == kDeltaSums && tile >= ztiles;           // this workgroup's columns are the map's
    const int cols = map ? a.Dk : a.Dv, col0 = (map ? tile - ztiles : tile) * DZT;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), zw = wave * 16;
    const int column = col0 + zw + c;                                   // of this lane's part of the state

    RowSource<T, DXP, WAVES, VEC> src_k, src_q;
    RowSource<T, DZT, WAVES, VEC> src_v;
    const int hk = h / a.group;
    src_k.init(a.k, tk.batch * a.kb + tk.row0 * a.kt + hk * a.kh, a.kt, a.Dk, 0);
    if (OUT) src_q.init(a.q, tk.batch * a.qb + tk.row0 * a.qt + hk * a.qh, a.qt, a.Dk, 0);
    src_v.init(a.v, tk.batch * a.vb + tk.row0 * a.vt + h * a.vh, a.vt, map ? 0 : a.Dv, col0);
    const char *rec0 = a.rec + (first_place(a, tk.seq, kC) * a.H + h) * a.rec_bytes;
    const int64_t rec_step = a.H * a.rec_bytes;
    // part 0, 1, 2 of a chunk, -1 for all: the next chunk's loads are spread over this one's products, since a wave that
    // issues many at once waits for the address unit
    auto bring = [&](int64_t ch, char *stage, int part) __attribute__((always_inline)) {
        const int64_t t = ch * kC;
        const int n = tk.len - t < kC ? (int)(tk.len - t) : kC;
        if (part <= 0) src_k.bring(t, n, reinterpret_cast<T *>(stage));
        if (OUT && (part < 0 || part == 1)) src_q.bring(t, n, reinterpret_cast<T *>(stage + W::kQ));
        if (part < 0 || part == 1) src_v.bring(t, n, reinterpret_cast<T *>(stage + W::kV));
        if (W::kRecord && (part < 0 || part == 2)) bring_record<WAVES, VEC>(rec0 + ch * rec_step, W::kPieces, stage + W::kRec);
    };
    if (W::kStages == 2 && first < end) bring(first, lds, -1);

    TileReader<T, DXP, WAVES> in_k;
    ColumnReader<T, DZT, WAVES> in_v;
    in_k.init();
    in_v.init(wave);
    State<KX> S;
    const int64_t nst = (int64_t)a.Dk * a.Dv;
    {
        // Of a sequence of several segments the chain has written the first one's state, too: state1 may be state0's own
        // memory, and nothing orders the last segment's workgroup behind the first one's.
        const bool joined = MODE != kDeltaSums && a.seg_state && chunks > a.seg_chunks;
        bool cleared = false;
        if (joined) S.load(a.seg_state + (place * a.H + h) * (int64_t)DXP * a.sum_ld, DXP, a.sum_ld, column);
        else S.load(MODE == kDeltaSums ? nullptr : first_state(a, tk.seq, tk.batch * a.N + tk.row0, tk.len, h, cleared), a.Dk, cols, column);
        S.settle();
        if (cleared) S.each([](int, float) { return 0.0f; });
        if (map) S.each([&](int row, float) __attribute__((always_inline)) { return row == column ? 1.0f : 0.0f; });
    }
    const int out_cols = a.Dv - (col0 + zw + g * 4);       // of this lane's first column of the output on
    T *out0 = OUT ? static_cast<T *>(a.out) + tk.batch * a.ob + tk.row0 * a.ot + h * a.oh : nullptr;

    for (int64_t ch = first; ch < end; ++ch) {
        char *stage = lds;
        if constexpr (W::kStages == 2) {
            stage += ((ch - first) & 1) * W::kBytes;
            // This chunk's loads were issued in the last one; four stores followed them (16-bit outputs).  The wait on LDS
            // reads keeps every wave's reads of the other stage before the loads into it.
            if (OUT && sizeof(T) == 2 && ch > first) wait_loads_and_barrier<4>();
            else if (MODE == kDeltaKeep && ch > first) wait_loads_and_barrier<16>();     // (those of w)
            else wait_loads_and_barrier<0>();
        } else {
            __syncthreads();
            bring(ch, stage, -1);
            wait_loads_and_barrier<0>();
        }
        auto ahead = [&](int part) __attribute__((always_inline)) {
            if (W::kStages == 2 && ch + 1 < end) bring(ch + 1, lds + ((ch + 1 - first) & 1) * W::kBytes, part);
        };
        ahead(0);
        const char *far = rec0 + ch * rec_step, *rec = W::kRecord ? stage + W::kRec : far;
        const bf8 *inv = reinterpret_cast<const bf8 *>(rec) + lane;
        const float *vec = reinterpret_cast<const float *>(rec + kDeltaInverse * 1024);
        const f32x4 *vec4 = reinterpret_cast<const f32x4 *>(vec) + g;      // the rows 16 r + 4 g ..: [4 r]
        const bf8 *prod = reinterpret_cast<const bf8 *>((W::kProducts ? rec : far) + (kDeltaInverse + kDeltaVectors) * 1024) + lane;
        const int64_t kept = (rec0 - a.rec) / a.rec_bytes + ch * a.H;      // (chunk, head)
        if (MODE == kDeltaKeep) S.keep_blocks(a.states + kept * a.dkp * a.dvp, column);
        // k S
        f32x4 x[4], o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = o[r] = f32x4{0, 0, 0, 0};
        bf8 few[OUT ? KX : 1][NOUT];
#pragma unroll
        for (int kk = 0; kk < KX; ++kk) {
            bf8 st[3];
            S.terms(kk, st);
            if (OUT)
#pragma unroll
                for (int j = 0; j < NOUT; ++j) few[kk][j] = st[j];
            bf8 kf[4][NIN];
#pragma unroll
            for (int r = 0; r < 4; ++r) in_terms(in_k.row8(stage, r, kk), kf[r]);
#pragma unroll
            for (int i = 0; i < NIN; ++i)
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (i + j < 3)
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = Mma<__bf16>::mma(kf[r][i], st[j], x[r]);
        }
        ahead(1);
        // r = v - exp(G) k S as operands over tokens
        bf8 rs[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 res[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                T v[4];
                in_v.col4(stage + W::kV, 2 * s + half, v);
                const f32x4 f = vec4[8 * s + 4 * half];
#pragma unroll
                for (int i = 0; i < 4; ++i) res[half][i] = (float)v[i] - f[i] * x[2 * s + half][i];
            }
            rows_terms<3>(res[0], res[1], rs[s]);
        }
        // the state's part of the outputs, which needs nothing of the above
        if (OUT) {
#pragma unroll
            for (int kk = 0; kk < KX; ++kk) {
                bf8 qf[4][NIN];
#pragma unroll
                for (int r = 0; r < 4; ++r) in_terms(in_k.row8(stage + W::kQ, r, kk), qf[r]);
#pragma unroll
                for (int i = 0; i < NIN; ++i)
#pragma unroll
                    for (int j = 0; j < NOUT; ++j)
                        if (i + j < NOUT)
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[r] = Mma<__bf16>::mma(few[kk][j], qf[r][i], o[r]);
            }
        }
        ahead(2);
        // w = inverse r, u = beta w; terms outermost, so that an accumulator's next product comes four instructions later
        f32x4 u[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) u[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int j = 0; i + j < 3; ++j)
#pragma unroll
                    for (int r = 2 * s; r < 4; ++r) u[r] = Mma<__bf16>::mma(inv[((r + 1) * (r + 1) / 4 + s) * 192 + i * 64], rs[s][j], u[r]);
        if (MODE == kDeltaKeep) keep_rows(a.wrong + kept * kC * a.dvp, u, column);
#pragma unroll
        for (int r = 0; r < 4; ++r) u[r] *= vec4[32 + 4 * r];
        // S <- exp(G_last) S + k^T (exp(G_last - G) u)
        bf8 es[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s) rows_terms<3>(u[2 * s] * vec4[16 + 8 * s], u[2 * s + 1] * vec4[16 + 8 * s + 4], es[s]);
        const float keep = vec[63];
#pragma unroll
        for (int kk = 0; kk < KX; ++kk) {
#pragma unroll
            for (int r = 0; r < 2; ++r) S.v[kk][r] *= keep;
            bf8 kf[2][2][NIN];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r) in_terms(in_k.col8(stage, s, kk, r), kf[s][r]);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < NIN; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (i + j < 3)
#pragma unroll
                            for (int r = 0; r < 2; ++r) S.v[kk][r] = Mma<__bf16>::mma(kf[s][r][i], es[s][j], S.v[kk][r]);
        }
        if (OUT) {
            const int64_t t0 = ch * kC;
            const int n = tk.len - t0 < kC ? (int)(tk.len - t0) : kC;
            bf8 us[2][NOUT];
#pragma unroll
            for (int s = 0; s < 2; ++s) rows_terms<NOUT>(u[2 * s], u[2 * s + 1], us[s]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] *= vec[192 + 16 * r + c];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < NOUT; ++i)
#pragma unroll
                    for (int j = 0; i + j < NOUT; ++j)
#pragma unroll
                        for (int r = 2 * s; r < 4; ++r)
                            o[r] = Mma<__bf16>::mma(us[s][j], prod[(((r + 1) * (r + 1) / 4 + s) * NOUT + i) * 64], o[r]);
            const auto view = wide_view(out0 + t0 * a.ot);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * r + c;
                const uint32_t at = ((row < n) & (out_cols > 0)) ? (uint32_t)((row * a.ot + col0 + zw + g * 4) * (int64_t)sizeof(T)) : kSkip;
                put_row<T, 1, VEC && sizeof(T) == 2>(view, at, &o[r], VEC, out_cols);
            }
        }
    }

    if (MODE == kDeltaSums) {
        const int ld = map ? a.map_ld : a.sum_ld;
        S.keep((map ? a.seg_map : a.seg_sum) + (place * a.H + h) * (int64_t)DXP * ld, ld, column);
    } else if (OUT && a.state1 && last) {
        const int64_t slot = state_slot(a.slots, a.n_slots, tk.seq);
        if (slot >= 0) S.store(a.state1 + (slot * a.H + h) * nst, a.Dk, a.Dv, column);
    }
}
#endif

template <typename T, int DXP, int WAVES, int MODE, bool VEC>
__global__ __launch_bounds__(walk_bound(DXP, WAVES, sizeof(T)), walk_waves(DXP, WAVES, MODE, sizeof(T))) void delta_walk_kernel(const DeltaArgs a, int ztiles, int tiles) {
#ifdef __HIP_DEVICE_COMPILE__
    using W = WalkShape<T, DXP, WAVES, MODE, VEC>;
    __shared__ __attribute__((aligned(1024))) char lds[W::kStages * W::kBytes];
    delta_walk<T, DXP, WAVES, MODE, VEC>(a, lds, dealt(blockIdx.x, delta_run(tiles, a.group)), ztiles, tiles);
#endif
}

// ---- gradients ------------------------------------------------------------------
// With G the gradient of the state behind a chunk, dO the outputs' and S the state before it,
//
//     x_j = exp(G_last - G_j) G^T k_j + sum_{i >= j} P_ij dO_i,    (I + C^T diag(beta)) y = x  (y: the gradient of u),
//     dv = beta y,    dbeta_j = y_j . w_j,
//     G <- exp(G_last) G + sum_i scale exp(G_i) q_i dO_i^T - sum_j exp(G_j) k_j dv_j^T,
//
// a walk from the sequence's end that needs no state and is as serial as the forward one: both run side by side in
// one launch.  What is left is parallel over the chunks (delta_gradients_kernel): with dP_ij = scale exp(G_i - G_j)
// dO_i . u_j (j <= i) and dC_ij = -exp(G_i - G_j) dv_i . u_j (j < i),
//
//     dq_i = scale exp(G_i) S dO_i + sum_j dP_ij k_j,
//     dk_j = sum_i dP_ij q_i + exp(G_last - G_j) G u_j - exp(G_j) S dv_j + sum_i dC_ij k_i + sum_i dC_ji k_i.
//
// Scaling a state by a factor and its values' gradients by the inverse changes nothing, which gives the logarithms'
// gradient without another product: that of G_i is q_i . dq_i - v_i . dv_i, and of a chunk's last sum <G, S behind> on
// top, so dlog_decay_t sums those of the chunk's tokens from t on.
template <typename T, int DXP, int WAVES, bool VEC> struct BackShape {
    static constexpr int DZT = WAVES * 16;
    using TX = RowTile<T, DXP, WAVES>;
    using TZ = RowTile<T, DZT, WAVES>;
    static constexpr int kQ = TX::BYTES, kG = 2 * TX::BYTES, kRec = kG + TZ::BYTES;
    static constexpr int kAll = 32, kFew = kDeltaInverse + kDeltaVectors + 1;
    static constexpr int kPieces = kRec + kAll * 1024 <= kLdsBytes ? kAll : kRec + kFew * 1024 <= kLdsBytes ? kFew : 0;
    static constexpr bool kRecord = kPieces > 0, kProducts = kPieces >= kAll;
    static constexpr int kBytes = kRec + kPieces * 1024;
    static constexpr int kStages = VEC && 2 * kBytes <= kLdsBytes ? 2 : 1;
    static_assert(kDeltaInverse + kAll <= kDeltaBackPieces && kBytes <= kLdsBytes, "LDS");
};

#ifdef __HIP_DEVICE_COMPILE__
template <typename T, int DXP, int WAVES, bool VEC>
__device__ __forceinline__ void delta_walk_back(const DeltaArgs &a, char *lds, uint32_t w, int tiles) {
    using W = BackShape<T, DXP, WAVES, VEC>;
    constexpr int KX = DXP / 32, DZT = W::DZT, NIN = Terms<T>::kIn;
    const int tile = w % tiles;
    w /= tiles;
    const int h = w % a.H;
    const int64_t place = w / a.H;
    if (place >= a.segs) return;
    Tokens tk;
    if (!unit_at(a, place, a.seg_chunks * kC, tk)) return;
    make_scalar(tk);
    const int64_t chunks = (tk.len + kC - 1) / kC;
    const int col0 = tile * DZT;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), zw = wave * 16;
    const int column = col0 + zw + c;

    RowSource<T, DXP, WAVES, VEC> src_k, src_q;
    RowSource<T, DZT, WAVES, VEC> src_g;
    const int hk = h / a.group;
    src_k.init(a.k, tk.batch * a.kb + tk.row0 * a.kt + hk * a.kh, a.kt, a.Dk, 0);
    src_q.init(a.q, tk.batch * a.qb + tk.row0 * a.qt + hk * a.qh, a.qt, a.Dk, 0);
    src_g.init(a.dout, tk.batch * a.gb + tk.row0 * a.gt + h * a.gh, a.gt, a.Dv, col0);
    const int64_t item0 = first_place(a, tk.seq, kC) * a.H + h;
    // vectors, then the operands
    const char *rec0 = a.rec + item0 * a.rec_bytes + kDeltaInverse * 1024;
    const int64_t rec_step = a.H * a.rec_bytes;
    auto bring = [&](int64_t ch, char *stage, int part) __attribute__((always_inline)) {      // (parts as in the forward walk)
        const int64_t t = ch * kC;
        const int n = tk.len - t < kC ? (int)(tk.len - t) : kC;
        if (part <= 0) src_k.bring(t, n, reinterpret_cast<T *>(stage));
        if (part < 0 || part == 1) src_g.bring(t, n, reinterpret_cast<T *>(stage + W::kG));
        if (part < 0 || part == 1) src_q.bring(t, n, reinterpret_cast<T *>(stage + W::kQ));
        if (W::kRecord && (part < 0 || part == 2)) bring_record<WAVES, VEC>(rec0 + ch * rec_step, W::kPieces, stage + W::kRec);
    };
    if (W::kStages == 2 && chunks > 0) bring(chunks - 1, lds, -1);

    TileReader<T, DXP, WAVES> in_k;
    ColumnReader<T, DZT, WAVES> in_g;
    in_k.init();
    in_g.init(wave);
    State<KX> G;
    const int64_t nst = (int64_t)a.Dk * a.Dv;
    G.load(a.dstate1 ? a.dstate1 + (tk.seq * a.H + h) * nst : nullptr, a.Dk, a.Dv, column);
    G.settle();

    for (int64_t back = 0; back < chunks; ++back) {
        const int64_t ch = chunks - 1 - back;
        char *stage = lds;
        if constexpr (W::kStages == 2) {
            stage += (back & 1) * W::kBytes;
            if (back > 0) wait_loads_and_barrier<16>();      // (sixteen stores of y followed the last of those loads)
            else wait_loads_and_barrier<0>();
        } else {
            __syncthreads();
            bring(ch, stage, -1);
            wait_loads_and_barrier<0>();
        }
        auto ahead = [&](int part) __attribute__((always_inline)) {
            if (W::kStages == 2 && ch > 0) bring(ch - 1, lds + ((back + 1) & 1) * W::kBytes, part);
        };
        const char *far = rec0 + ch * rec_step, *rec = W::kRecord ? stage + W::kRec : far;
        const float *vec = reinterpret_cast<const float *>(rec);
        const f32x4 *vec4 = reinterpret_cast<const f32x4 *>(vec) + g;
        const bf8 *inv = reinterpret_cast<const bf8 *>(rec + kDeltaVectors * 1024) + lane;
        const f32x4 *prod = reinterpret_cast<const f32x4 *>((W::kProducts ? rec : far) + (kDeltaVectors + kDeltaInverse) * 1024) + lane;
        const int64_t item = item0 + ch * a.H;
        ahead(0);
        G.keep_blocks(a.grads + item * a.dkp * a.dvp, column);

        // the outputs' gradients as operands over tokens, as they are and by scale exp(G)
        bf8 gf[2][NIN], gs[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Raw8<T> raw;
            in_g.col4(stage + W::kG, 2 * s, raw.v);
            in_g.col4(stage + W::kG, 2 * s + 1, raw.v + 4);
            in_terms(raw, gf[s]);
            f32x4 lo = vec4[48 + 8 * s], hi = vec4[48 + 8 * s + 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) lo[i] *= (float)raw.v[i], hi[i] *= (float)raw.v[4 + i];
            rows_terms<3>(lo, hi, gs[s]);
        }
        // G^T k, and sum_i P_ij dO_i
        f32x4 x[4], p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = p[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KX; ++kk) {
            bf8 st[3], kf[4][NIN];
            G.terms(kk, st);
#pragma unroll
            for (int r = 0; r < 4; ++r) in_terms(in_k.row8(stage, r, kk), kf[r]);
#pragma unroll
            for (int i = 0; i < NIN; ++i)
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (i + j < 3)
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = Mma<__bf16>::mma(kf[r][i], st[j], x[r]);
        }
        ahead(1);
#pragma unroll
        for (int r = 0, e = 0; r < 4; ++r)
#pragma unroll
            for (int s = r / 2; s < 2; ++s, ++e) {
                bf8 pf[3];
                rows_terms<3>(prod[e * 128], prod[e * 128 + 64], pf);
                p[r] = mma_terms<3>(pf, gf[s], p[r]);
            }
        ahead(2);
        // y
        bf8 xs[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 sum[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) sum[half] = x[2 * s + half] * vec4[16 + 8 * s + 4 * half] + p[2 * s + half];
            rows_terms<3>(sum[0], sum[1], xs[s]);
        }
        f32x4 y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 1; s >= 0; --s)
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int j = 0; i + j < 3; ++j)
#pragma unroll
                    for (int r = 0; r < 2 * s + 2; ++r) {
                        const int e = (r < 2 ? 2 * r + s : 3 + r - 1 + s - 1);      // operands (r, s >= r / 2) in order
                        y[r] = Mma<__bf16>::mma(inv[e * 192 + i * 64], xs[s][j], y[r]);
                    }
        keep_rows(a.dright + item * kC * a.dvp, y, column);
        // G <- exp(G_last) G + q^T (scale exp(G) dO) - k^T (exp(G) beta y)
        const float keep = vec[63];
        bf8 ys[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 f[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) f[half] = -vec4[8 * s + 4 * half] * vec4[32 + 8 * s + 4 * half];
            rows_terms<3>(y[2 * s] * f[0], y[2 * s + 1] * f[1], ys[s]);
        }
#pragma unroll
        for (int kk = 0; kk < KX; ++kk) {
#pragma unroll
            for (int r = 0; r < 2; ++r) G.v[kk][r] *= keep;
            bf8 kf[2][2][NIN], qf[2][2][NIN];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    in_terms(in_k.col8(stage + W::kQ, s, kk, r), qf[s][r]);
                    in_terms(in_k.col8(stage, s, kk, r), kf[s][r]);
                }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < NIN; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (i + j < 3)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                G.v[kk][r] = Mma<__bf16>::mma(qf[s][r][i], gs[s][j], G.v[kk][r]);
                                G.v[kk][r] = Mma<__bf16>::mma(kf[s][r][i], ys[s][j], G.v[kk][r]);
                            }
        }
    }
    if (a.dstate0) G.store(a.dstate0 + (tk.seq * a.H + h) * nst, a.Dk, a.Dv, column);
}
#endif

// Both walks of the backward call: even items forwards, odd ones from the end.  Bound as the forward walks, the reverse one
// with twice their products: 4 x 4096 tokens x 20 heads of 128, bf16 540 us (8.5 us a chunk), fp32 1640.
template <typename T, int DXP, int WAVES, bool VEC>
__global__ __launch_bounds__(walk_bound(DXP, WAVES, sizeof(T))) void delta_back_walks_kernel(const DeltaArgs a, int tiles) {
#ifdef __HIP_DEVICE_COMPILE__
    using F = WalkShape<T, DXP, WAVES, kDeltaKeep, VEC>;
    using R = BackShape<T, DXP, WAVES, VEC>;
    constexpr int kF = F::kStages * F::kBytes, kR = R::kStages * R::kBytes;
    __shared__ __attribute__((aligned(1024))) char lds[kF > kR ? kF : kR];
    const uint32_t w = dealt(blockIdx.x, delta_run(2 * tiles, a.group));
    if (w & 1) delta_walk_back<T, DXP, WAVES, VEC>(a, lds, w / 2, tiles);
    else delta_walk<T, DXP, WAVES, kDeltaKeep, VEC>(a, lds, w / 2, tiles, tiles);
#endif
}

// One workgroup a (chunk, head); see above.  A wave has 16 tokens as columns of all products: it forms their columns of
// dP and dC, which stay in its registers as operands over tokens, and their rows of dq and dk.  Operands over the
// values' columns (u, dv, dO, S, G: rows of 32 neighbouring values) are split once, each by one wave, and met by all
// through LDS, 32 columns at a time; k and q, met by columns, follow in the same place.
//
// Bound by waits: half of the time at barriers and for LDS, the rest the matrix units and the splitting.  4 x 4096 tokens x
// 20 heads of 128, bf16: 550 us (612 with S and G loaded into registers), fp32 875.
template <typename T, int DXP> struct GradientShape {
    static constexpr int DP = 64, DT = DP / 16;      // columns of q and k at once, their tiles
    static constexpr int NIN = Terms<T>::kIn;
    static constexpr int kU = 0, kY = 4 * 3, kG = 8 * 3, kS = kG + 4 * NIN, kD = kS + DT * 3, kPieces = kD + DT * 3;
    static constexpr int kTiles = 2 * RowTile<T, DP, 4>::BYTES;
    static constexpr int kRaw = kPieces * 1024 > kTiles ? kPieces * 1024 : kTiles;      // S and G as they come
    static constexpr int kBytes = kRaw + 2 * DP * 128;
};
template <typename T, int DXP, bool VEC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void delta_gradients_kernel(const DeltaArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
    using Sh = GradientShape<T, DXP>;
    constexpr int DP = Sh::DP, DT = Sh::DT, NIN = Sh::NIN;
    using TX = RowTile<T, DP, 4>;
    __shared__ __attribute__((aligned(1024))) char lds[Sh::kBytes];
    __shared__ double sums[kC];
    __shared__ float weights[kC], own[kC], rest[4];
    const int64_t item = blockIdx.x;
    const int64_t place = item / a.H;
    const int h = (int)(item % a.H), hk = h / a.group;
    Tokens t;
    if (!unit_at(a, place, kC, t)) return;
    make_scalar(t);
    const int64_t t0 = t.unit * kC;
    const int n = t.len - t0 < kC ? (int)(t.len - t0) : kC;
    if (n <= 0) return;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t gate0 = (t.batch * a.N + t.row0 + t0) * a.H + h;
    if (wave == 0) {
        float d = lane < n ? a.log_decay[gate0 + (int64_t)lane * a.H] : 0.0f;
        d = d < -128.0f ? -128.0f : d;
        double sum = d;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const double up = __shfl_up(sum, s);
            if (lane >= s) sum += up;
        }
        sums[lane] = sum;
        weights[lane] = lane < n ? a.beta[gate0 + (int64_t)lane * a.H] : 0.0f;
    }
    __syncthreads();

    const float *S = a.states + item * a.dkp * a.dvp, *G = a.grads + item * a.dkp * a.dvp;
    const int mine = 16 * wave + c;                 // this lane's token, as a column
    const int width = mine < n ? a.Dv : 0;          // of its rows that exist
    const float *W = a.wrong + item * kC * a.dvp + mine * 32 + g * 8, *Y = a.dright + item * kC * a.dvp + mine * 32 + g * 8;
    const auto gv = wide_view(static_cast<const T *>(a.dout) + t.batch * a.gb + (t.row0 + t0) * a.gt + h * a.gh);
    const auto vv = wide_view(static_cast<const T *>(a.v) + t.batch * a.vb + (t.row0 + t0) * a.vt + h * a.vh);
    T *dv0 = a.dv ? static_cast<T *>(a.dv) + t.batch * a.dvb + (t.row0 + t0 + mine) * a.dvt + h * a.dvh : nullptr;
    const float beta = weights[mine];
    bf8 *frag = reinterpret_cast<bf8 *>(lds) + lane;
    auto put = [&](int piece, const auto &terms) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(terms) / sizeof(bf8)); ++i) frag[(piece + i) * 64] = terms[i];
    };
    auto get = [&](int piece, auto &terms) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(terms) / sizeof(bf8)); ++i) terms[i] = frag[(piece + i) * 64];
    };

    // slot i: dP and dC of the wave's tokens with those of tile i up to its own (slots 0 .. wave, rows earlier), then
    // with those of tile i - 1 from its own on (rows later)
    f32x4 dp[5], dc[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) dp[i] = dc[i] = f32x4{0, 0, 0, 0};
    float dot_v = 0.0f, dot_w = 0.0f, dot_q = 0.0f, dot_k = 0.0f, inner = 0.0f;
    const double gm = sums[mine];
    const float first = exp_of(gm), last = exp_of(sums[63] - gm);

#pragma unroll 1
    for (int col0 = 0; col0 < DXP && col0 < a.Dk; col0 += DP) {
        f32x4 qa[DT], ka[DT], va[DT];      // S dO, G u, S dv: rows of the states x tokens
#pragma unroll
        for (int d = 0; d < DT; ++d) qa[d] = ka[d] = va[d] = f32x4{0, 0, 0, 0};
        // A block's values, on their way while the block before is multiplied: rows of the tokens into registers, those of
        // the states into LDS, 16-byte slot i of a row at i ^ swizzle (neighbouring lanes' rows on different banks).
        f32x4 wl, wh, yl, yh;
        Raw8<T> go, v;
        auto swizzle = [](int row) { return (row & 3) | ((row >> 3) & 1) << 2; };
        auto fetch = [&](int z0) __attribute__((always_inline)) {
            const int z = z0 + g * 8, left = width - z;
#pragma unroll
            for (int i = 0; i < 2 * DP * 8 / 256; ++i) {
                const int at = i * 256 + threadIdx.x, row = at / 8 % DP, slot = at % 8 ^ swizzle(row);
                lds_load16((i < DP * 8 / 256 ? S : G) + z0 * (int64_t)a.dkp + col0 * 32, lds + Sh::kRaw + (i * 256 + wave * 64) * 16,
                           (uint32_t)(row * 128 + slot * 16));
            }
            const f32x4 *wp = reinterpret_cast<const f32x4 *>(W + z0 * kC), *yp = reinterpret_cast<const f32x4 *>(Y + z0 * kC);
            wl = wp[0], wh = wp[1], yl = yp[0], yh = yp[1];
            go = load_row8<T, VEC>(gv, left > 0 ? (uint32_t)((mine * a.gt + z) * (int64_t)sizeof(T)) : kSkip, left);
            if (col0 == 0) v = load_row8<T, VEC>(vv, left > 0 ? (uint32_t)((mine * a.vt + z) * (int64_t)sizeof(T)) : kSkip, left);
        };
        fetch(0);
#pragma unroll 1
        for (int z0 = 0; z0 < a.dvp; z0 += 32) {
            const int z = z0 + g * 8;
            wait_loads_and_barrier<0>();        // (and the block before has been read)
            bf8 gx[NIN], ux[3], yx[3];
            {
                const int left = width - z;
                if (col0 == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dot_w += wl[j] * yl[j] + wh[j] * yh[j];
                        dot_v += (float)v.v[j] * (yl[j] * beta) + (float)v.v[4 + j] * (yh[j] * beta);
                    }
                    if (dv0 && left > 0) {
                        Raw8<T> o;
#pragma unroll
                        for (int j = 0; j < 4; ++j) o.v[j] = (T)(yl[j] * beta), o.v[4 + j] = (T)(yh[j] * beta);
                        if (VEC && left >= 8) {
                            __builtin_memcpy(__builtin_assume_aligned(dv0 + z, 16), &o, sizeof o);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (j < left) dv0[z + j] = o.v[j];
                        }
                    }
                }
                in_terms(go, gx);
                rows_terms<3>(wl * beta, wh * beta, ux);
                rows_terms<3>(yl * beta, yh * beta, yx);
                if (col0 == 0) {
                    put(Sh::kG + wave * NIN, gx);
                    put(Sh::kU + wave * 3, ux);
                    put(Sh::kY + wave * 3, yx);
                }
#pragma unroll
                for (int d = 0; d < DT / 4; ++d) {
                    // (rows of a pair of tiles in the order of the state's own: a lane's results of both are neighbours)
                    const int tile = wave * (DT / 4) + d, row = (tile >> 1) * 32 + (c >> 2) * 8 + (tile & 1) * 4 + (c & 3);
                    const char *raw = lds + Sh::kRaw + row * 128;
                    const int lo = (2 * g ^ swizzle(row)) * 16, hi = ((2 * g + 1) ^ swizzle(row)) * 16;
                    const f32x4 sl = *reinterpret_cast<const f32x4 *>(raw + lo), sh = *reinterpret_cast<const f32x4 *>(raw + hi);
                    const f32x4 gl = *reinterpret_cast<const f32x4 *>(raw + DP * 128 + lo), gh = *reinterpret_cast<const f32x4 *>(raw + DP * 128 + hi);
                    bf8 x[3];
#pragma unroll
                    for (int j = 0; j < 4; ++j) inner += sl[j] * gl[j] + sh[j] * gh[j];
                    rows_terms<3>(sl, sh, x);
                    put(Sh::kS + (wave * (DT / 4) + d) * 3, x);
                    rows_terms<3>(gl, gh, x);
                    put(Sh::kD + (wave * (DT / 4) + d) * 3, x);
                }
            }
            __syncthreads();
            if (z0 + 32 < a.dvp) fetch(z0 + 32);
            if (col0 == 0) {
#pragma unroll
                for (int i = 0; i < 5; ++i) {
                    if (i <= wave && i < 4) {
                        bf8 u[3];
                        get(Sh::kU + i * 3, u);
                        dp[i] = mma_terms<3>(u, gx, dp[i]);
                        dc[i] = mma_terms<3>(u, yx, dc[i]);
                    } else if (i > wave) {
                        bf8 o[NIN], y[3];
                        get(Sh::kG + (i - 1) * NIN, o);
                        get(Sh::kY + (i - 1) * 3, y);
                        dp[i] = mma_terms<3>(o, ux, dp[i]);
                        dc[i] = mma_terms<3>(y, ux, dc[i]);
                    }
                }
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                bf8 x[3];
                get(Sh::kS + d * 3, x);
#pragma unroll
                for (int i = 0; i < 3; ++i)      // (two accumulators in turn)
#pragma unroll
                    for (int j = 0; i + j < 3; ++j) {
                        if (j < NIN) qa[d] = Mma<__bf16>::mma(x[i], gx[j < NIN ? j : 0], qa[d]);
                        va[d] = Mma<__bf16>::mma(x[i], yx[j], va[d]);
                    }
                get(Sh::kD + d * 3, x);
                ka[d] = mma_terms<3>(x, ux, ka[d]);
            }
        }
        __syncthreads();
        // k and q in the place of the operands
        T *tile_k = reinterpret_cast<T *>(lds), *tile_q = reinterpret_cast<T *>(lds + TX::BYTES);
        {
            RowSource<T, DP, 4, VEC> src;
            src.init(a.k, t.batch * a.kb + t.row0 * a.kt + hk * a.kh, a.kt, a.Dk, col0);
            src.bring(t0, n, tile_k);
            src.init(a.q, t.batch * a.qb + t.row0 * a.qt + hk * a.qh, a.qt, a.Dk, col0);
            src.bring(t0, n, tile_q);
        }
        wait_loads_and_barrier<0>();
        // out: lane (g, c) has 8 neighbouring columns of its token
        auto out = [&](void *base, int64_t sb, int64_t st, int64_t sh, const f32x4 (&v)[2], int col) __attribute__((always_inline)) {
            const int left = a.Dk - col;
            if (!base || mine >= n || left <= 0) return;
            if (a.parts) {
                float *p = static_cast<float *>(base) + ((t.batch * a.N + t.row0 + t0 + mine) * a.H + h) * (int64_t)a.Dk + col;
                if (VEC) {          // (rows of whole 16-byte pieces)
                    *reinterpret_cast<f32x4 *>(p) = v[0];
                    if (left > 4) *reinterpret_cast<f32x4 *>(p + 4) = v[1];
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (r < left) p[r] = v[r >> 2][r & 3];
                }
                return;
            }
            T *p = static_cast<T *>(base) + t.batch * sb + (t.row0 + t0 + mine) * st + hk * sh + col;
            Raw8<T> o;
#pragma unroll
            for (int r = 0; r < 8; ++r) o.v[r] = (T)v[r >> 2][r & 3];
            if (VEC && (sizeof(T) == 2 || left > 4)) {
                __builtin_memcpy(__builtin_assume_aligned(p, 16), &o, sizeof o);
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < left) p[r] = o.v[r];
            }
        };
        TileReader<T, DP, 4> in;
        in.init();
        const char *ck = lds, *cq = lds + TX::BYTES;
        // masked and decayed, once: what is not above (below) the diagonal of earlier (later) rows
        if (col0 == 0) {
#pragma unroll
            for (int i = 0; i < 5; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool low = i <= wave;
                    const int row = 16 * (low ? i : i - 1) + 4 * g + r;
                    const float f = exp_of(row <= mine ? gm - sums[row & 63] : sums[row & 63] - gm);
                    dp[i][r] = (low ? row <= mine : row >= mine) ? dp[i][r] * (f * a.scale) : 0.0f;
                    dc[i][r] = (low ? row < mine : row > mine) ? -dc[i][r] * f : 0.0f;
                }
        }
        const f32x4 zero{0, 0, 0, 0};
        // as operands over tokens: dP for dq, then those for dk
        {
            bf8 m[2][3];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                rows_terms<3>(2 * s <= wave ? dp[2 * s] : zero, 2 * s + 1 <= wave ? dp[2 * s + 1] : zero, m[s]);
            }
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                f32x4 dq[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    dq[r] = qa[2 * kk + r] * (a.scale * first);
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        if (s == 0 || wave >= 2) {
                            bf8 x[NIN];
                            in_terms(in.col8(ck, s, kk, r), x);
                            dq[r] = mma_terms<3>(x, m[s], dq[r]);
                        }
                }
                const Raw8<T> q = in.row8(cq + wave * 16 * TileReader<T, DP, 4>::RB, 0, kk);
#pragma unroll
                for (int r = 0; r < 8; ++r) dot_q += (float)q.v[r] * dq[r >> 2][r & 3];
                out(a.dq, a.dqb, a.dqt, a.dqh, dq, col0 + kk * 32 + 8 * g);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        {
            bf8 m[2][3], b[2][3];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f32x4 x[2], y[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int tile = 2 * s + half;
                    x[half] = tile >= wave ? dp[tile + 1] : zero;
                    y[half] = (tile <= wave ? dc[tile] : zero) + (tile >= wave ? dc[tile + 1] : zero);
                }
                rows_terms<3>(x[0], x[1], m[s]);
                rows_terms<3>(y[0], y[1], b[s]);
            }
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                f32x4 dk[2];
                const Raw8<T> k = in.row8(ck + wave * 16 * TileReader<T, DP, 4>::RB, 0, kk);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    dk[r] = ka[2 * kk + r] * last;
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot_k += (float)k.v[4 * r + i] * dk[r][i];      // <G, what the chunk adds to the state>
                    dk[r] -= va[2 * kk + r] * first;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        bf8 x[NIN];
                        in_terms(in.col8(ck, s, kk, r), x);
                        dk[r] = mma_terms<3>(x, b[s], dk[r]);
                        if (s == 1 || wave < 2) {
                            in_terms(in.col8(cq, s, kk, r), x);
                            dk[r] = mma_terms<3>(x, m[s], dk[r]);
                        }
                    }
                }
                out(a.dk, a.dkb, a.dkt, a.dkh, dk, col0 + kk * 32 + 8 * g);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // a token's own dot products: four lanes have parts of each
    float each = dot_q - dot_v;
    dot_w += __shfl_xor(dot_w, 16), each += __shfl_xor(each, 16);
    dot_w += __shfl_xor(dot_w, 32), each += __shfl_xor(each, 32);
    if (a.dbeta && g == 0 && mine < n) a.dbeta[gate0 + (int64_t)mine * a.H] = dot_w;
    if (!a.dlog_decay) return;
    if (g == 0) own[mine] = each;
    float behind = dot_k + exp_of(sums[63]) * inner;      // <G, S behind>
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) behind += __shfl_xor(behind, s);
    if (lane == 0) rest[wave] = behind;
    __syncthreads();
    if (wave == 0) {
        double sum = own[lane];
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const double down = __shfl_down(sum, s);
            if (lane + s < 64) sum += down;
        }
        sum += (double)((rest[0] + rest[1]) + (rest[2] + rest[3]));
        // (the terms cancel to roundings where a token clears the state: there it is 0)
        const int64_t gate = gate0 + (int64_t)lane * a.H;
        if (lane < n) a.dlog_decay[gate] = a.log_decay[gate] < kClears ? 0.0f : (float)sum;
    }
#endif
}

// State before each segment from the segments' own sums and maps: S <- map S + sum, the first one's as the caller gave it.
// One workgroup a (sequence, head, 16 columns), grid (B, H, tiles); a wave has a quarter of the rows of the map, of which
// those of the next segment are on their way while this one's are in use, and the state goes round through LDS.  Bound by
// latency: the segments are serial (12 segments of 20 heads of 128: 42 us).
template <int DXP> static __global__ __launch_bounds__(256, 1) void delta_chain_kernel(const DeltaArgs a) {
    constexpr int KX = DXP / 32, R = DXP / 64, LD = DXP + 4;
    __shared__ __attribute__((aligned(16))) float state[2][16 * LD];
    const int h = blockIdx.y, col0 = blockIdx.z * 16;
    const int64_t seq = blockIdx.x;
    int64_t start, len;
    sequence_bounds(a, seq, start, len);
    const int64_t length = a.seg_chunks * kC, count = (len + length - 1) / length;
    if (count < 2) return;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, wave = threadIdx.x >> 6, row0 = wave * R * 16;
    const int64_t first = first_place(a, seq, length) * a.H + h, sums = (int64_t)DXP * a.sum_ld, maps = (int64_t)DXP * a.map_ld;
    {
        bool cleared;
        const float *p = first_state(a, seq, a.cu ? start : seq * a.N, len, h, cleared);
        const auto view = wide_view(p);
        float *out = a.seg_state + first * sums;
        for (int i = threadIdx.x; i < DXP * 16; i += 256) {
            const int row = i / 16, col = i % 16;
            const bool there = (p != nullptr) & (row < a.Dk) & (col0 + col < a.Dv);
            float x = view_load<float>(view, there ? (uint32_t)(row * a.Dv + col0 + col) * 4u : kSkip);
            if (cleared) x = 0.0f;
            state[0][col * LD + row] = x;
            out[row * (int64_t)a.sum_ld + col0 + col] = x;
        }
    }
    f32x4 map[R][KX][2], sum[R];
    auto fetch = [&](int64_t i, f32x4 (&m)[R][KX][2], f32x4 (&s)[R]) __attribute__((always_inline)) {
        const float *mp = a.seg_map + (first + i * a.H) * maps, *sp = a.seg_sum + (first + i * a.H) * sums;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    m[r][kk][half] = *reinterpret_cast<const f32x4 *>(mp + (row0 + 16 * r + c) * (int64_t)a.map_ld + kk * 32 + g * 8 + half * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[r][j] = sp[(row0 + 16 * r + 4 * g + j) * (int64_t)a.sum_ld + col0 + c];
        }
    };
    if (DXP <= 128) fetch(0, map, sum);
    __syncthreads();
    for (int64_t i = 0; i + 1 < count; ++i) {
        f32x4 next[R][KX][2], own[R];
        if (DXP > 128) fetch(i, map, sum);      // (registers hold one)
        else if (i + 2 < count) fetch(i + 1, next, own);
        const float *from = state[i & 1];
        float *to = state[(i & 1) ^ 1];
#pragma unroll
        for (int kk = 0; kk < KX; ++kk) {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(from + c * LD + kk * 32 + g * 8);
            bf8 st[3];
            rows_terms<3>(p[0], p[1], st);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                bf8 mf[3];
                rows_terms<3>(map[r][kk][0], map[r][kk][1], mf);
                sum[r] = mma_terms<3>(mf, st, sum[r]);
            }
        }
        float *out = a.seg_state + (first + (i + 1) * a.H) * sums;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            *reinterpret_cast<f32x4 *>(to + c * LD + row0 + 16 * r + 4 * g) = sum[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) out[(row0 + 16 * r + 4 * g + j) * (int64_t)a.sum_ld + col0 + c] = sum[r][j];
        }
        if (DXP <= 128) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sum[r] = own[r];
#pragma unroll
                for (int kk = 0; kk < KX; ++kk) map[r][kk][0] = next[r][kk][0], map[r][kk][1] = next[r][kk][1];
            }
        }
        __syncthreads();
    }
}

// The single-token form.  One workgroup a (sequence, head, LANES * VEC columns), LANES lanes along a row of the state,
// 256 / LANES groups of rows; the rows stay in registers between the products with k and q (which are taken of the
// state before the token: out = scale (a S^T q + (q . k) u)) and the update.  Bound by the state, which is read and
// written once: 256 sequences x 20 heads of 128 140 us, 4.8 TB/s.  For few sequences, workgroups of a fourth of the
// columns are no faster (20 heads: 5.0 and 5.1 us; 340 heads: 12.9 and 12.5).
template <typename T, int VEC, int LANES, int ROWS>
__global__ __launch_bounds__(256) void delta_step_kernel(const DeltaStep a) {
    constexpr int RG = 256 / LANES, W = LANES * VEC;
    static_assert(ROWS * RG <= 256 && W <= 256, "a row and a column a thread");
    __shared__ float sq[256], sk[256];
    __shared__ float part[2][RG][W];
    __shared__ float both[4];
    __shared__ float u[W];
    const int tid = threadIdx.x, lc = tid % LANES, rg = tid / LANES;
    const int64_t b = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / a.group;
    const int dv0 = (blockIdx.y * LANES + lc) * VEC;
    const T *q = static_cast<const T *>(a.q) + b * a.qb + hk * a.qh;
    const T *k = static_cast<const T *>(a.k) + b * a.kb + hk * a.kh;
    const T *v = static_cast<const T *>(a.v) + b * a.vb + h * a.vh;
    const int64_t slot = state_slot(a.slots, a.n_slots, b);
    typedef float vec __attribute__((ext_vector_type(VEC)));
    const bool live = dv0 < a.Dv && slot >= 0;   // VEC divides Dv
    float *s = live ? a.state + (slot * a.H + h) * (int64_t)a.Dk * a.Dv + dv0 : nullptr;
    vec e[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = i * RG + rg;
        e[i] = (vec)0.0f;
        if (live && r < a.Dk) e[i] = *reinterpret_cast<const vec *>(s + (int64_t)r * a.Dv);
    }
    const float log = a.log_decay[b * a.H + h], d = expf(log), beta = a.beta[b * a.H + h];
    if (log < kClears)      // (0 times what is no number would keep it)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) e[i] = (vec)0.0f;
    {
        const float qi = tid < a.Dk ? (float)q[tid] : 0.0f, ki = tid < a.Dk ? (float)k[tid] : 0.0f;
        sq[tid] = qi;
        sk[tid] = ki;
        float x = qi * ki;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) x += __shfl_xor(x, i);
        if ((tid & 63) == 0) both[tid >> 6] = x;
    }
    __syncthreads();
    vec ak = (vec)0.0f, aq = (vec)0.0f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = i * RG + rg;
        ak += e[i] * sk[r];
        aq += e[i] * sq[r];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[0][rg][lc * VEC + i] = ak[i], part[1][rg][lc * VEC + i] = aq[i];
    __syncthreads();
    if (tid < W) {
        const int dv = blockIdx.y * W + tid;
        float k0 = 0.0f, q0 = 0.0f;
        for (int r = 0; r < RG; ++r) k0 += part[0][r][tid], q0 += part[1][r][tid];
        const float vv = dv < a.Dv ? (float)v[dv] : 0.0f;
        const float w = beta * (vv - d * k0);
        u[tid] = w;
        const float qk = (both[0] + both[1]) + (both[2] + both[3]);
        if (dv < a.Dv) static_cast<T *>(a.out)[b * a.ob + h * a.oh + dv] = (T)(slot >= 0 ? a.scale * (d * q0 + qk * w) : 0.0f);
    }
    __syncthreads();
    if (!live) return;
    vec mine;
#pragma unroll
    for (int i = 0; i < VEC; ++i) mine[i] = u[lc * VEC + i];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = i * RG + rg;
        if (r < a.Dk) *reinterpret_cast<vec *>(s + (int64_t)r * a.Dv) = d * e[i] + sk[r] * mine;
    }
}

// ---- host side of one storage type ----------------------------------------
template <typename T, bool VEC, bool BACK> static hipError_t delta_prepare_launch(const DeltaArgs &a, hipStream_t s) {
    const unsigned grid = (unsigned)((a.chunks * a.H + 3) / 4);
    if (grid == 0) return hipSuccess;
    if (a.Dk <= 64) delta_prepare_kernel<T, 64, VEC, BACK><<<grid, 256, 0, s>>>(a);
    else if (a.Dk <= 128) delta_prepare_kernel<T, 128, VEC, BACK><<<grid, 256, 0, s>>>(a);
    else delta_prepare_kernel<T, 256, VEC, BACK><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T> static hipError_t delta_prepare_typed(const DeltaArgs &a, hipStream_t s) {
    if (a.states) return a.vec ? delta_prepare_launch<T, true, true>(a, s) : delta_prepare_launch<T, false, true>(a, s);
    return a.vec ? delta_prepare_launch<T, true, false>(a, s) : delta_prepare_launch<T, false, false>(a, s);
}
template <typename T, int DXP, int WAVES, bool VEC> static hipError_t delta_back_launch(const DeltaArgs &a, hipStream_t s) {
    const int tiles = a.dvp / (WAVES * 16);
    const int64_t items = 2 * a.segs * a.H * tiles, round = 8 * (int64_t)delta_run(2 * tiles, a.group);
    delta_back_walks_kernel<T, DXP, WAVES, VEC><<<(unsigned)((items + round - 1) / round * round), WAVES * 64, 0, s>>>(a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks == 0) return e;
    delta_gradients_kernel<T, DXP, VEC><<<(unsigned)(a.chunks * a.H), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, bool VEC> static hipError_t delta_back(const DeltaArgs &a, hipStream_t s) {
    if (a.Dk > 128) return delta_back_launch<T, 256, 4, VEC>(a, s);
    if (a.Dk > 64) return a.wide ? delta_back_launch<T, 128, 8, VEC>(a, s) : delta_back_launch<T, 128, 4, VEC>(a, s);
    return a.wide ? delta_back_launch<T, 64, 8, VEC>(a, s) : delta_back_launch<T, 64, 4, VEC>(a, s);
}
template <typename T> static hipError_t delta_bwd_typed(const DeltaArgs &a, hipStream_t s) {
    return a.vec ? delta_back<T, true>(a, s) : delta_back<T, false>(a, s);
}
template <typename T, int DXP, int WAVES, int MODE, bool VEC> static hipError_t delta_walk_launch(const DeltaArgs &a, hipStream_t s) {
    constexpr int DZT = WAVES * 16;
    // (the chain reads all DXP columns of a map, zeros behind Dk among them)
    const int ztiles = (a.Dv + DZT - 1) / DZT, tiles = ztiles + (MODE == kDeltaSums ? (DXP + DZT - 1) / DZT : 0);
    const int64_t items = a.segs * a.H * tiles, round = 8 * (int64_t)delta_run(tiles, a.group);
    delta_walk_kernel<T, DXP, WAVES, MODE, VEC><<<(unsigned)((items + round - 1) / round * round), WAVES * 64, 0, s>>>(a, ztiles, tiles);
    return hipGetLastError();
}
template <typename T, int MODE, bool VEC> static hipError_t delta_walks(const DeltaArgs &a, hipStream_t s) {
    // (rows wider than 128 leave registers and LDS for 64 columns only)
    if (a.Dk > 128) return delta_walk_launch<T, 256, 4, MODE, VEC>(a, s);
    if (a.Dk > 64) return a.wide ? delta_walk_launch<T, 128, 8, MODE, VEC>(a, s) : delta_walk_launch<T, 128, 4, MODE, VEC>(a, s);
    return a.wide ? delta_walk_launch<T, 64, 8, MODE, VEC>(a, s) : delta_walk_launch<T, 64, 4, MODE, VEC>(a, s);
}
template <typename T> static hipError_t delta_fwd_typed(const DeltaArgs &a, hipStream_t s) {
    if (a.seg_state) {
        const hipError_t e = a.vec ? delta_walks<T, kDeltaSums, true>(a, s) : delta_walks<T, kDeltaSums, false>(a, s);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)a.B, (unsigned)a.H, (unsigned)((a.Dv + 15) / 16));
        if (a.Dk <= 64) delta_chain_kernel<64><<<grid, 256, 0, s>>>(a);
        else if (a.Dk <= 128) delta_chain_kernel<128><<<grid, 256, 0, s>>>(a);
        else delta_chain_kernel<256><<<grid, 256, 0, s>>>(a);
        const hipError_t e2 = hipGetLastError();
        if (e2 != hipSuccess) return e2;
    }
    return a.vec ? delta_walks<T, kDeltaOut, true>(a, s) : delta_walks<T, kDeltaOut, false>(a, s);
}
template <typename T, int VEC, int LANES> static hipError_t delta_step_rows(const DeltaStep &a, hipStream_t s) {
    constexpr int RG = 256 / LANES;
    const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.Dv + LANES * VEC - 1) / (LANES * VEC)));
    if (a.Dk <= 64) delta_step_kernel<T, VEC, LANES, 64 / RG><<<grid, 256, 0, s>>>(a);
    else if (a.Dk <= 128) delta_step_kernel<T, VEC, LANES, 128 / RG><<<grid, 256, 0, s>>>(a);
    else delta_step_kernel<T, VEC, LANES, 256 / RG><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T> static hipError_t delta_step_typed(const DeltaStep &a, bool vec, hipStream_t s) {
    if (!vec) return delta_step_rows<T, 1, 32>(a, s);
    return delta_step_rows<T, 4, 32>(a, s);
}

#define FFTCONV_DELTA_TYPE(NAME, T)                                                                                  \
    hipError_t launch_delta_prepare_##NAME(const DeltaArgs &a, hipStream_t s) { return delta_prepare_typed<T>(a, s); } \
    hipError_t launch_delta_fwd_##NAME(const DeltaArgs &a, hipStream_t s) { return delta_fwd_typed<T>(a, s); }         \
    hipError_t launch_delta_bwd_##NAME(const DeltaArgs &a, hipStream_t s) { return delta_bwd_typed<T>(a, s); }         \
    hipError_t launch_delta_step_##NAME(const DeltaStep &a, bool vec, hipStream_t s) { return delta_step_typed<T>(a, vec, s); }

}  // namespace fftconv
