// decay_kernels.hpp -- linear attention with a decay for each head: the walk
// over a sequence that serves the prompt form and all three gradients, and
// the recurrent form for single tokens.  Instantiated per storage type by
// decay_f16.hip, decay_bf16.hip and decay_f32.hip.
//
// Mathematics.  With d = exp(log_decay) <= 1 per head, over the tokens t of a
// sequence and an fp32 state E (DX x DZ),
//
//     out_t = i_scale d^off x_t^T E_{t} + p_scale sum_{j <= t} d^(t-j) (x_t . y_j) z_j   (from a chunk's E)
//     E_{t+1} = d E_t + u_scale d^(1-off) y_t z_t^T
//
// The prompt form is x, y, z = q, k, v with off = 1 (the state is decayed
// before a token adds to it).  The gradients are the same walk:
//     dq: x, y, z = dout, v, k          (state S^T)
//     dk: x, y, z = v, dout, q   and    dv: x, y, z = k, q, dout,
// both from the sequence's end with off = 0 (the state's gradient is read
// before it is decayed; the walk keeps d G).
//
// A sequence is walked in chunks of C tokens: within a chunk the masked
// product P = (X Y^T) o decay and O = P Z; across chunks O += diag(d^i) X E and
// E <- d^C E + Y^T (d^(C-1-s) Z).  All four products run on the matrix cores.
// One workgroup of four waves walks one (segment, head, tile of <= 128 z
// columns); wave w owns a slice of the tile's columns and keeps E's columns of
// that slice in its accumulators for the whole walk, so the state never
// leaves the registers.  The waves share only the chunk's X, Y, Z in LDS:
// every wave recomputes P, whose accumulator layout is the operand layout of
// P Z (rows of Y permuted so that a lane's 8 values are consecutive tokens),
// which costs a third more matrix instructions than sharing P but saves its
// LDS round trip and a barrier.
//
// Rounding (16-bit types): P and the state are rounded to the storage type
// as operands of O (an error like the output's own rounding).  The state is
// an fp32 result, so its update must not lose: d^(C-1-s) Z is split into
// 2 (fp16) or 3 (bf16) storage-type terms that hold it to fp32 precision; in
// fp16, whose second term would fall among the subnormals for |Z| << 1, the
// accumulators hold E times a power of two that follows each chunk's largest |Z|.
//
// A call with few (sequence, head) pairs splits sequences into segments: a
// first pass over y, z gives each segment's own sum, a small kernel chains
// them into the state before each segment, and the walk starts from there.
#pragma once

#include "mma.hpp"
#include "sequence_ops.hpp"

namespace fftconv {

struct SegInfo {
    int64_t start, len;   // the sequence's first token and length
    int64_t seq, index;   // sequence, segment within it
    int64_t count;        // segments of the sequence
    int64_t first;        // block index of the sequence's first segment
};

__device__ __forceinline__ void packed_bounds(const DecayWalk &a, int64_t b, int64_t &start, int64_t &len) {
    // bounds come from device memory: clamped to the tokens there are
    int64_t s = a.cu[b], e = a.cu[b + 1];
    s = s < 0 ? 0 : (s > a.N ? a.N : s);
    e = e < s ? s : (e > a.N ? a.N : e);
    start = s;
    len = e - s;
}

// Segment of block blk (by_seq: of sequence blk, its first segment); false when there is none.
// Called by all 256 threads.
__device__ inline bool find_segment(const DecayWalk &a, int64_t blk, bool by_seq, SegInfo &info) {
    if (!a.cu) {
        const int64_t per = a.N > 0 ? (a.N + a.seglen - 1) / a.seglen : 1;
        info.count = per;
        info.len = a.N;
        info.seq = by_seq ? blk : blk / per;
        info.index = by_seq ? 0 : blk % per;
        info.start = 0;
        info.first = info.seq * per;
        return info.seq < a.B;
    }
    __shared__ int64_t wave_sum[4];
    __shared__ int64_t hit[6];
    if (threadIdx.x == 0) hit[0] = -1;
    int64_t before = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t b0 = 0; b0 < a.B; b0 += 256) {
        const int64_t b = b0 + threadIdx.x;
        int64_t start = 0, len = 0, n = 0;
        if (b < a.B) {
            packed_bounds(a, b, start, len);
            n = len > 0 ? (len + a.seglen - 1) / a.seglen : 1;
        }
        int64_t sum = n;
        for (int s = 1; s < 64; s <<= 1) {
            const int64_t up = __shfl_up(sum, s);
            if (lane >= s) sum += up;
        }
        if (lane == 63) wave_sum[wave] = sum;
        __syncthreads();
        int64_t lead = before;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) lead += wave_sum[w];
            before += wave_sum[w];
        }
        const int64_t first = lead + sum - n;
        const bool mine = by_seq ? b == blk : (blk >= first && blk < first + n);
        if (b < a.B && mine) {
            hit[0] = b;
            hit[1] = by_seq ? 0 : blk - first;
            hit[2] = n;
            hit[3] = start;
            hit[4] = len;
            hit[5] = first;
        }
        __syncthreads();
        if (hit[0] >= 0) break;
    }
    if (a.B == 0) __syncthreads();
    info.seq = hit[0];
    info.index = hit[1];
    info.count = hit[2];
    info.start = hit[3];
    info.len = hit[4];
    info.first = hit[5];
    return info.seq >= 0;
}

// Slot of sequence seq in the state pool, or -1 (no state kept).
__device__ __forceinline__ int64_t state_slot(const int32_t *slots, int64_t n_slots, int64_t seq) {
    if (!slots) return seq;
    const int64_t s = slots[seq];
    return s >= 0 && s < n_slots ? s : -1;
}

__device__ __forceinline__ float decay_power(float log2d, int64_t n) {
    return n <= 0 ? 1.0f : exp2f(log2d * (float)n);
}

constexpr float kLog2e = 1.44269504088896340736f;

// Rows of a chunk from HBM into registers (16 bytes each), zeros outside; then into LDS.
template <typename T, int C, int DP> struct ChunkLoad {
    static constexpr int E = 16 / (int)sizeof(T);        // values of a piece
    static constexpr int PR = DP / E;                    // pieces of a row
    static constexpr int N = C * PR / 256;               // pieces of a thread
    static constexpr int LD = DP + E;                    // LDS row stride: 16 bytes off the banks' period
    static_assert(C * PR % 256 == 0, "whole pieces");
    uint4 r[N];

    // tokens t0 .. t0 + C - 1 of a sequence of len tokens whose first token row is p
    __device__ __forceinline__ void load(const T *p, int64_t stride, int64_t t0, int64_t end, int64_t len, int reverse,
                                         int cols, int col0, int vec) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int idx = i * 256 + threadIdx.x, row = idx / PR, col = col0 + (idx % PR) * E;
            const int64_t t = t0 + row;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (t < end && col < cols) {
                const T *src = p + (reverse ? len - 1 - t : t) * stride + col;
                if (vec) {
                    v = *reinterpret_cast<const uint4 *>(src);
                } else {
                    T e[E];
#pragma unroll
                    for (int j = 0; j < E; ++j) e[j] = col + j < cols ? src[j] : (T)0.0f;
                    __builtin_memcpy(&v, e, 16);
                }
            }
            r[i] = v;
        }
    }
    __device__ __forceinline__ void store(T *tile) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int idx = i * 256 + threadIdx.x;
            *reinterpret_cast<uint4 *>(tile + (idx / PR) * LD + (idx % PR) * E) = r[i];
        }
    }
};

template <typename T> constexpr int decay_chunk() { return sizeof(T) == 2 ? 64 : 32; }

// grid: (nblk, H, z tiles); OUT = false: the segment's own sum only (y, z read), for every
// segment that another follows.  DXP: DX padded; NT: 16-column tiles of E per wave.
template <typename T, typename TO, int DXP, int NT, bool OUT>
__global__ __launch_bounds__(256, DXP <= 128 ? 2 : 1) void decay_walk_kernel(const DecayWalk a) {
    constexpr int C = decay_chunk<T>();
    constexpr int KX = DXP / 32;          // 32-wide contraction steps over DX
    constexpr int KC = C / 32;            // and over a chunk's tokens
    constexpr int RT = C / 16;            // 16-token row tiles of a chunk
    constexpr int DZT = NT * 64;          // z columns of a workgroup
    constexpr int kSplit = Mma<T>::kSplit;
    using LX = ChunkLoad<T, C, DXP>;
    using LZ = ChunkLoad<T, C, DZT>;
    using v8 = typename Mma<T>::v8;
    __shared__ __attribute__((aligned(16))) T sx[OUT ? C * LX::LD : 8];
    __shared__ __attribute__((aligned(16))) T sy[C * LX::LD];
    __shared__ __attribute__((aligned(16))) T sz[C * LZ::LD];
    __shared__ float upd[2 * C];          // u_scale d^(C - off - s): weight of token s in the next state
    __shared__ float row_w[C];            // i_scale d^(i + off): weight of the chunk's first state in row i

    SegInfo si;
    if (!find_segment(a, blockIdx.x, false, si)) return;
    if (!OUT && si.index + 1 >= si.count) return;
    const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, c = lane & 15;
    const int z0 = blockIdx.z * DZT;                     // first z column of the workgroup
    const int zw = wave * NT * 16;                       // this wave's columns within it
    const int64_t t_begin = si.index * a.seglen;
    const int64_t t_end = t_begin + a.seglen < si.len && si.index + 1 < si.count ? t_begin + a.seglen : si.len;
    const int64_t row0 = a.cu ? si.start : 0, batch = a.cu ? 0 : si.seq;
    const T *px = static_cast<const T *>(a.x) + batch * a.xb + row0 * a.xt + (h / a.gx) * a.xh;
    const T *py = static_cast<const T *>(a.y) + batch * a.yb + row0 * a.yt + (h / a.gy) * a.yh;
    const T *pz = static_cast<const T *>(a.z) + batch * a.zb + row0 * a.zt + (h / a.gz) * a.zh;
    const float log2d = a.log_decay[h] * kLog2e;

    for (int i = tid; i < 2 * C; i += 256) upd[i] = i < C ? a.u_scale * decay_power(log2d, C - a.off - i) : 0.0f;
    for (int i = tid; i < C; i += 256) row_w[i] = a.i_scale * decay_power(log2d, i + a.off);

    // z column of accumulator column m of tile t (NT = 2: a lane's two tiles hold 8 neighbours)
    auto zcol = [&](int m, int t) { return zw + (NT == 2 ? (m >> 2) * 8 + t * 4 + (m & 3) : m); };

    // E[kk][r][t]: rows kk * 32 + g * 8 + r * 4 + i, column zcol(c, t)
    f32x4 E[KX][2][NT];
    {
        const float *s0 = nullptr;
        int64_t sx_ = a.s0x, sz_ = a.s0z;
        if (a.seg && OUT) {
            s0 = a.seg + ((int64_t)blockIdx.x * a.H + h) * a.DX * a.DZ;
            sx_ = a.DZ;
            sz_ = 1;
        } else if (OUT && a.state0) {
            const int64_t slot = state_slot(a.slots, a.n_slots, si.seq);
            if (slot >= 0) s0 = a.state0 + (slot * a.H + h) * (int64_t)a.DX * a.DZ;
        }
#pragma unroll
        for (int kk = 0; kk < KX; ++kk)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int dx = kk * 32 + g * 8 + r * 4 + i, dz = z0 + zcol(c, t);
                        E[kk][r][t][i] = s0 && dx < a.DX && dz < a.DZ ? s0[dx * sx_ + dz * sz_] : 0.0f;
                    }
    }
    // decay of P: tile pair at row offset 16 o from its 32 tokens, value (r, i): d^(16 o + c - 8 g - 4 r - i)
    float fac[2 * KC][2][4];
    if (OUT) {
#pragma unroll
        for (int o = 0; o < 2 * KC; ++o)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 16 * o + c - 8 * g - 4 * r - i;
                    fac[o][r][i] = n < 0 ? 0.0f : a.p_scale * decay_power(log2d, n);
                }
    }

    LX lx, ly;
    LZ lz;
    if (OUT) lx.load(px, a.xt, t_begin, t_end, si.len, a.reverse, a.DX, 0, a.vec_x);
    ly.load(py, a.yt, t_begin, t_end, si.len, a.reverse, a.DX, 0, a.vec_y);
    lz.load(pz, a.zt, t_begin, t_end, si.len, a.reverse, a.DZ, z0, a.vec_z);
    int ex = 0;            // the accumulators hold E * 2^ex (fp16 only, else 0)
    for (int64_t t0 = t_begin; t0 < t_end; t0 += C) {
        __syncthreads();
        if (OUT) lx.store(sx);
        ly.store(sy);
        lz.store(sz);
        __syncthreads();
        if (t0 + C < t_end) {
            if (OUT) lx.load(px, a.xt, t0 + C, t_end, si.len, a.reverse, a.DX, 0, a.vec_x);
            ly.load(py, a.yt, t0 + C, t_end, si.len, a.reverse, a.DX, 0, a.vec_y);
            lz.load(pz, a.zt, t0 + C, t_end, si.len, a.reverse, a.DZ, z0, a.vec_z);
        }
        const int n = t_end - t0 < C ? (int)(t_end - t0) : C;
        // this wave's columns of Z, tokens 8 g .. 8 g + 7 of each 32
        v8 zf[KC][NT];
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                zf[kc][t] = lds_col8<T>(sz, LZ::LD, kc * 32 + g * 8,
                                        zw + (NT == 2 ? (lane & 3) * 8 + t * 4 : (lane & 3) * 4), zcol(c, t));
        if (OUT) {
            const float unscale = Mma<T>::kNarrow ? ldexpf(1.0f, -ex) : 1.0f;
            v8 ef[KX][NT];     // the state as an operand: row zcol(c, t), slots 8 g + j
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ef[kk][t][j] = (T)(Mma<T>::kNarrow ? E[kk][j >> 2][t][j & 3] * unscale : E[kk][j >> 2][t][j & 3]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                v8 xf[KX];
#pragma unroll
                for (int kk = 0; kk < KX; ++kk) xf[kk] = lds_row8<T>(sx + (rt * 16 + c) * LX::LD + kk * 32 + g * 8);
                f32x4 o[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) o[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                    for (int t = 0; t < NT; ++t) o[t] = Mma<T>::mma(ef[kk][t], xf[kk], o[t]);
                const float rw = row_w[rt * 16 + c];
#pragma unroll
                for (int t = 0; t < NT; ++t) o[t] *= rw;
#pragma unroll
                for (int kc = 0; kc <= rt / 2; ++kc) {
                    v8 pf;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // rows of Y permuted: accumulator row m is token kc * 32 + 8 (m / 4) + 4 r + m % 4
                        f32x4 p = {0, 0, 0, 0};
                        const T *yr = sy + (kc * 32 + (c >> 2) * 8 + r * 4 + (c & 3)) * LX::LD + g * 8;
#pragma unroll
                        for (int kk = 0; kk < KX; ++kk) p = Mma<T>::mma(lds_row8<T>(yr + kk * 32), xf[kk], p);
#pragma unroll
                        for (int i = 0; i < 4; ++i) pf[r * 4 + i] = (T)(p[i] * fac[rt - 2 * kc][r][i]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) o[t] = Mma<T>::mma(zf[kc][t], pf, o[t]);
                }
                const int row = rt * 16 + c;
                if (row < n && a.out) {
                    const int64_t tok = a.reverse ? si.len - 1 - (t0 + row) : t0 + row;
                    TO *po = static_cast<TO *>(a.out) + batch * a.ob + (row0 + tok) * a.ot + (h / a.go) * a.oh;
                    const int dz = z0 + zw + (NT == 2 ? g * 8 : g * 4);
                    if (a.vec_o && dz + NT * 4 <= a.DZ) {
                        TO w[NT * 4];
#pragma unroll
                        for (int j = 0; j < NT * 4; ++j) w[j] = (TO)o[j >> 2][j & 3];
                        __builtin_memcpy(__builtin_assume_aligned(po + dz, sizeof(TO) * NT * 4 < 16 ? sizeof(TO) * NT * 4 : 16), w,
                                         sizeof w);
                    } else {
#pragma unroll
                        for (int j = 0; j < NT * 4; ++j)
                            if (dz + j < a.DZ) po[dz + j] = (TO)o[j >> 2][j & 3];
                    }
                }
            }
        }
        // E <- d^n E + Y^T (weights Z)
        float dn = decay_power(log2d, n), lift = 1.0f;
        if (Mma<T>::kNarrow) {
            float most = 0.0f;
#pragma unroll
            for (int kc = 0; kc < KC; ++kc)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf((float)zf[kc][t][j]));
            for (int s = 1; s < 64; s <<= 1) most = fmaxf(most, __shfl_xor(most, s));
            most *= fabsf(a.u_scale);
            // the largest term near 2^14; the weights are at most u_scale
            int next = ex;
            if (most > 0.0f) next = 13 - ilogbf(most);
            next = next < -60 ? -60 : (next > 60 ? 60 : next);
            dn = ldexpf(dn, next - ex);
            lift = ldexpf(1.0f, next);
            ex = next;
        }
#pragma unroll
        for (int kk = 0; kk < KX; ++kk)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t) E[kk][r][t] *= dn;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
            v8 zw_[NT][kSplit];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = upd[C - n + kc * 32 + g * 8 + j] * lift;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float rest = (float)zf[kc][t][j] * w[j];
                    // one value for every use: left to itself the compiler rounds the product to fp16 once
                    // through fp32 and once fused, and the two first terms then differ at ties
                    if (kSplit > 1) asm("" : "+v"(rest));
#pragma unroll
                    for (int s = 0; s < kSplit; ++s) {
                        const T part = (T)rest;
                        zw_[t][s][j] = part;
                        rest -= (float)part;
                    }
                }
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    // rows of the state permuted like zcol: row m is kk * 32 + 8 (m / 4) + 4 r + m % 4
                    const v8 yf = lds_col8<T>(sy, LX::LD, kc * 32 + g * 8, kk * 32 + (lane & 3) * 8 + r * 4,
                                              kk * 32 + (c >> 2) * 8 + r * 4 + (c & 3));
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int s = 0; s < kSplit; ++s) E[kk][r][t] = Mma<T>::mma(yf, zw_[t][s], E[kk][r][t]);
                }
        }
    }

    const float unscale = Mma<T>::kNarrow ? ldexpf(1.0f, -ex) : 1.0f;
    float *s1 = nullptr;
    int64_t sx_ = a.s1x, sz_ = a.s1z;
    if (!OUT) {
        s1 = a.seg + ((int64_t)blockIdx.x * a.H + h) * a.DX * a.DZ;
        sx_ = a.DZ;
        sz_ = 1;
    } else if (a.state1 && si.index + 1 == si.count) {
        const int64_t slot = state_slot(a.slots, a.n_slots, si.seq);
        if (slot >= 0) s1 = a.state1 + (slot * a.H + h) * (int64_t)a.DX * a.DZ;
    }
    if (!s1) return;
#pragma unroll
    for (int kk = 0; kk < KX; ++kk)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int dx = kk * 32 + g * 8 + r * 4 + i, dz = z0 + zcol(c, t);
                    if (dx < a.DX && dz < a.DZ) s1[dx * sx_ + dz * sz_] = E[kk][r][t][i] * unscale;
                }
}

// The single-token form: E <- d E + k v^T, out = scale E^T q, one workgroup per (sequence,
// head, tile of LANES * VEC value columns); LANES lanes along a row of the state, the other
// 256 / LANES row groups share its rows, joined through LDS.
template <typename T, int VEC, int LANES>
__global__ __launch_bounds__(256) void decay_step_kernel(const DecayStep a) {
    constexpr int RG = 256 / LANES, U = 8;
    __shared__ float sq[256], sk[256];
    __shared__ float part[RG][LANES * VEC];
    const int tid = threadIdx.x, lc = tid % LANES, rg = tid / LANES;
    const int64_t b = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H;
    const int dv0 = (blockIdx.y * LANES + lc) * VEC;
    const T *q = static_cast<const T *>(a.q) + b * a.qb + h * a.qh;
    const T *k = static_cast<const T *>(a.k) + b * a.kb + (h / a.group) * a.kh;
    const T *v = static_cast<const T *>(a.v) + b * a.vb + (h / a.group) * a.vh;
    const int64_t slot = state_slot(a.slots, a.n_slots, b);
    const float d = expf(a.log_decay[h]);
    for (int i = tid; i < a.Dk; i += 256) {
        sq[i] = a.scale * (float)q[i];
        sk[i] = (float)k[i];
    }
    float vv[VEC], acc[VEC];
    const bool live = dv0 < a.Dv && slot >= 0;   // VEC divides Dv
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        vv[e] = live ? (float)v[dv0 + e] : 0.0f;
        acc[e] = 0.0f;
    }
    __syncthreads();
    typedef float vec __attribute__((ext_vector_type(VEC)));
    if (live) {
        float *s = a.state + (slot * a.H + h) * (int64_t)a.Dk * a.Dv + dv0;
        for (int r0 = rg; r0 < a.Dk; r0 += RG * U) {
            vec e[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r0 + u * RG < a.Dk) e[u] = *reinterpret_cast<const vec *>(s + (int64_t)(r0 + u * RG) * a.Dv);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RG;
                if (r < a.Dk) {
                    const float kr = sk[r], qr = sq[r];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        e[u][i] = d * e[u][i] + kr * vv[i];
                        acc[i] += qr * e[u][i];
                    }
                    *reinterpret_cast<vec *>(s + (int64_t)r * a.Dv) = e[u];
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[rg][lc * VEC + i] = acc[i];
    __syncthreads();
    if (tid < LANES * VEC) {
        const int dv = blockIdx.y * LANES * VEC + tid;
        float sum = 0.0f;
        for (int r = 0; r < RG; ++r) sum += part[r][tid];
        if (dv < a.Dv) static_cast<T *>(a.out)[b * a.ob + h * a.oh + dv] = (T)sum;
    }
}

// Gradients of shared heads: dst (tokens, Hk, D) <- sum over the group of src (tokens, H, D), fp32.
template <typename T>
__global__ __launch_bounds__(256) void decay_group_sum_kernel(const float *src, T *dst, int64_t B, int64_t N, int Hk,
                                                              int group, int D, int64_t db, int64_t dt, int64_t dh) {
    const int64_t n = B * N * Hk * D;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t d = i % D, hk = i / D % Hk, t = i / D / Hk;
        const float *p = src + (t * Hk + hk) * group * D + d;
        float s = 0.0f;
        for (int j = 0; j < group; ++j) s += p[(int64_t)j * D];
        dst[(t / N) * db + (t % N) * dt + hk * dh + d] = (T)s;
    }
}

// State before each segment from the segments' own sums, in place: grid (B, H, pieces of 1024).
static __global__ __launch_bounds__(256) void decay_chain_kernel(const DecayWalk a) {
    SegInfo si;
    if (!find_segment(a, blockIdx.x, true, si)) return;
    const int h = blockIdx.y;
    const int64_t nst = (int64_t)a.DX * a.DZ;
    const float dn = decay_power(a.log_decay[h] * kLog2e, a.seglen);
    const int64_t slot = a.state0 ? state_slot(a.slots, a.n_slots, si.seq) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t e = blockIdx.z * (int64_t)1024 + u * 256 + threadIdx.x;
        if (e >= nst) continue;
        float run = 0.0f;
        if (slot >= 0) {
            const int64_t x = e / a.DZ, z = e % a.DZ;
            run = a.state0[(slot * a.H + h) * nst + x * a.s0x + z * a.s0z];
        }
        float *p = a.seg + (si.first * a.H + h) * nst + e;
        const int64_t step = a.H * nst;
        for (int64_t s = 0; s < si.count; s += 8) {
            float own[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) own[j] = s + j + 1 < si.count ? p[(s + j) * step] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s + j < si.count) {
                    p[(s + j) * step] = run;
                    run = dn * run + own[j];
                }
        }
    }
}

// ---- host side of one storage type ----------------------------------------
template <typename T, typename TO> static hipError_t walk_dispatch(const DecayWalk &a, bool out, hipStream_t stream) {
    const bool narrow = a.DZ <= 64;
    const dim3 grid((unsigned)a.nblk, (unsigned)a.H, (unsigned)((a.DZ + (narrow ? 63 : 127)) / (narrow ? 64 : 128)));
#define FFTCONV_WALK(DXP)                                                                                       \
    do {                                                                                                        \
        if (out) {                                                                                              \
            if (narrow) decay_walk_kernel<T, TO, DXP, 1, true><<<grid, 256, 0, stream>>>(a);                    \
            else decay_walk_kernel<T, TO, DXP, 2, true><<<grid, 256, 0, stream>>>(a);                           \
        } else {                                                                                                \
            if (narrow) decay_walk_kernel<T, T, DXP, 1, false><<<grid, 256, 0, stream>>>(a);                    \
            else decay_walk_kernel<T, T, DXP, 2, false><<<grid, 256, 0, stream>>>(a);                           \
        }                                                                                                       \
    } while (0)
    if (a.DX <= 64) FFTCONV_WALK(64);
    else if (a.DX <= 128) FFTCONV_WALK(128);
    else FFTCONV_WALK(256);
#undef FFTCONV_WALK
    return hipGetLastError();
}

template <typename T> static hipError_t walk_typed(const DecayWalk &a, bool out_f32, hipStream_t stream) {
    if (a.seg) {
        hipError_t e = walk_dispatch<T, T>(a, false, stream);
        if (e != hipSuccess) return e;
        const int64_t nst = (int64_t)a.DX * a.DZ;
        decay_chain_kernel<<<dim3((unsigned)a.B, (unsigned)a.H, (unsigned)((nst + 1023) / 1024)), 256, 0, stream>>>(a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return out_f32 ? walk_dispatch<T, float>(a, true, stream) : walk_dispatch<T, T>(a, true, stream);
}

template <typename T> static hipError_t step_typed(const DecayStep &a, bool vec, hipStream_t stream) {
    const unsigned bh = (unsigned)(a.B * a.H);
    if (!vec) {
        decay_step_kernel<T, 1, 32><<<dim3(bh, (a.Dv + 31) / 32), 256, 0, stream>>>(a);
    } else if (bh < 512) {   // few rows: narrow tiles spread the state over more compute units
        decay_step_kernel<T, 4, 8><<<dim3(bh, (a.Dv + 31) / 32), 256, 0, stream>>>(a);
    } else {
        decay_step_kernel<T, 4, 32><<<dim3(bh, (a.Dv + 127) / 128), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t group_sum_typed(const float *src, void *dst, int64_t B, int64_t N, int Hk, int group, int D,
                                  int64_t db, int64_t dt, int64_t dh, hipStream_t stream) {
    const int64_t n = B * N * Hk * D;
    const int64_t blocks = (n + 255) / 256;
    decay_group_sum_kernel<T><<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(
        src, static_cast<T *>(dst), B, N, Hk, group, D, db, dt, dh);
    return hipGetLastError();
}

#define FFTCONV_DECAY_TYPE(NAME, T)                                                                            \
    hipError_t launch_decay_walk_##NAME(const DecayWalk &a, bool out_f32, hipStream_t s) {                      \
        return walk_typed<T>(a, out_f32, s);                                                                    \
    }                                                                                                           \
    hipError_t launch_decay_step_##NAME(const DecayStep &a, bool vec, hipStream_t s) {                          \
        return step_typed<T>(a, vec, s);                                                                        \
    }                                                                                                           \
    hipError_t launch_decay_group_sum_##NAME(const float *src, void *dst, int64_t B, int64_t N, int Hk, int gr, \
                                             int D, int64_t db, int64_t dt, int64_t dh, hipStream_t s) {        \
        return group_sum_typed<T>(src, dst, B, N, Hk, gr, D, db, dt, dh, s);                                    \
    }

}  // namespace fftconv
