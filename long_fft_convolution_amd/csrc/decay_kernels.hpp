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
// A sequence is walked in chunks of C = 32 tokens: within a chunk the masked
// product P = (X Y^T) o decay and O = P Z; across chunks O += diag(d^i) X E and
// E <- d^C E + Y^T (d^(C-1-s) Z).  All four products run on the matrix cores.
// One workgroup of four waves walks one (segment, head, tile of <= 128 z
// columns); wave w owns a slice of the tile's columns and keeps E's columns of
// that slice in its accumulators for the whole walk, so the state never
// leaves the registers.  The waves share only the chunk's X, Y, Z in LDS:
// every wave recomputes P, whose accumulator layout is the operand layout of
// P Z (rows of Y permuted so that a lane's 8 values are consecutive tokens),
// which costs a fifth more matrix instructions than sharing P but saves its
// LDS round trip and a barrier.
//
// Rounding (16-bit types): P and the state are rounded to the storage type
// as operands of O (an error like the output's own rounding), in fp16 after a
// power of two where they are small or large for its range: the state by its
// largest element in a wave's columns, P row by row.  The state is
// an fp32 result, so its update must not lose: d^(C-1-s) Z is split into
// 2 (fp16) or 3 (bf16) storage-type terms that hold it to fp32 precision (2 in
// bf16 in segments that another follows, whose state only outputs see).
//
// The accumulators hold E times a gain that grows by d^-C a chunk, so that
// decaying the state costs one factor in the chunk's weights instead of a
// multiplication of every accumulator; they are brought back when the gain
// would pass 2^16 (few bits of its exponent, so exp2 of it is exact to a few
// 2^-24), in fp16 also when the terms leave the range that keeps the second
// one out of the subnormals.  Heads that forget more than 2^8 a chunk have
// their accumulators multiplied each time.
//
// A call with few (sequence, head) pairs splits sequences into segments: a
// first pass over y, z gives each segment's own sum, a small kernel chains
// them into the state before each segment, and the walk starts from there.
#pragma once

#include <type_traits>

#include "sequence_device.hpp"
#include "sequence_ops.hpp"

namespace fftconv {

struct SegInfo {
    int64_t start, len;   // the sequence's first token and length
    int64_t seq, index;   // sequence, segment within it
    int64_t count;        // segments of the sequence
    int64_t slot;         // place of the sequence's first state among the segments' states
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
        info.slot = info.seq * ((a.N + a.sublen - 1) / a.sublen);
        return info.seq < a.B;
    }
    __shared__ int64_t wave_sum[4];
    __shared__ int64_t hit[5];
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
    // no two sequences meet: start / sublen + ceil(len / sublen) <= (start + len) / sublen + 1
    info.slot = info.start / a.sublen + info.seq;
    return info.seq >= 0;
}

// Of a sequence's `count` parts, those that precede its last segment.
__device__ __forceinline__ int64_t parts_before_last(const DecayWalk &a, int64_t count) {
    return count > 0 ? (count - 1) / a.parts * a.parts : 0;
}

__device__ __forceinline__ float decay_power(float log2d, int64_t n) {
    return n <= 0 ? 1.0f : exp2f(log2d * (float)n);
}

// Tokens of a chunk.  32 is one contraction step of the 16-bit matrix instruction: with it the
// chunk's own products cost least (a 64-token chunk has half its P blocks to spare) and three
// stages of tiles fit two workgroups on a CU.
constexpr int kChunk = 32;

// A chunk's tile of one operand in LDS: kChunk rows of DP values in 16-byte slots, slot s of row r
// lying at s ^ f(r).  f spreads over the 128 bytes of an LDS cycle what the cycle's lanes read: eight
// neighbouring rows (X), or the permuted rows 8 (c / 4) + c % 4 of eight c (Y), and four groups of four
// columns of four rows (Y, Z: two cycles, the 8-byte groups being of one half of their slots).
template <typename T, int DP, bool PERMUTED> struct ChunkTile {
    static constexpr int E = 16 / (int)sizeof(T);            // values of a slot
    static constexpr int PR = DP / E;                        // slots of a row
    static constexpr int N = kChunk * PR / 256;              // 16-byte loads of a thread
    static constexpr int VALUES = kChunk * DP;
    static_assert(kChunk * PR % 256 == 0, "whole loads");
    static __device__ __forceinline__ int f(int row) {
        if (PERMUTED) return (row & 1) << 2 | (row & 2) | ((row >> 3) & 1);
        return row & 7;
    }
    static __device__ __forceinline__ void source(int i, int &row, int &slot) {
        const int idx = i * 256 + (threadIdx.x & 255);
        row = idx / PR;
        slot = idx % PR ^ f(row);
    }
    static __device__ __forceinline__ const T *at(const T *tile, int row, int slot) {
        return tile + (row * PR + (slot ^ f(row))) * E;
    }
    // 8 values of a row at column col (a multiple of 8)
    static __device__ __forceinline__ typename Mma<T>::v8 row8(const T *tile, int row, int col) {
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const typename Mma<T>::v8 *>(at(tile, row, col / 8));
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(at(tile, row, col / 4));
            const f32x4 b = *reinterpret_cast<const f32x4 *>(at(tile, row, col / 4 + 1));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Rows 8 g + j of this lane's own column, mine.  16-bit types: two transposing reads, in which 16
    // lanes read four rows of four 4-column groups and lane c receives column c % 4 of group c / 4;
    // group is the start of the group that lanes of this c % 4 read.  fp32: value by value.
    static __device__ __forceinline__ typename Mma<T>::v8 col8(const T *tile, int group, int mine) {
        const int lane = threadIdx.x & 63, g = lane >> 4;
        if constexpr (sizeof(T) == 2) {
            const int row = g * 8 + ((lane & 15) >> 2);
            const T *p = at(tile, row, group / 8) + group % 8;     // f(row + 4) = f(row)
            typedef typename Mma<T>::v4 v4;
            const v4 a = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p)));
            const v4 b = __builtin_bit_cast(v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(FFTCONV_LDS_CAST(s16x4, p + 4 * DP)));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typename Mma<T>::v8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = at(tile, g * 8 + j, mine / 4)[mine % 4];
            return v;
        }
    }
};

// Brings a tensor's chunks into LDS.  VEC: loads with an LDS destination (rows of whole, aligned
// 16-byte pieces; a piece outside the chunk or the columns reads zero by the buffer unit's range
// check); else value by value through registers.
template <typename T, int DP, bool PERMUTED, bool VEC> struct ChunkSource {
    using Tile = ChunkTile<T, DP, PERMUTED>;
    const T *p;            // the sequence's first row
    int64_t stride, len;
    int cols, col0, reverse;
    uint32_t off[VEC ? Tile::N : 1];

    __device__ __forceinline__ void init(const void *base, int64_t batch, int64_t sb, int64_t row0, int64_t st, int64_t head,
                                         int64_t sh, int64_t len_, int cols_, int col0_, int reverse_) {
        p = static_cast<const T *>(base) + batch * sb + row0 * st + head * sh;
        stride = st;
        len = len_;
        cols = cols_, col0 = col0_, reverse = reverse_;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < Tile::N; ++i) {
                int row, slot;
                Tile::source(i, row, slot);
                const int col = col0 + slot * Tile::E;
                off[i] = col < cols ? (uint32_t)(((reverse ? kChunk - 1 - row : row) * stride + col) * (int64_t)sizeof(T))
                                    : kSkip;
            }
        }
    }
    // tokens t0 .. t0 + n - 1 (n <= kChunk) into the tile; the rest becomes zero
    __device__ __forceinline__ void bring(int64_t t0, int n, T *tile) const {
        if constexpr (VEC) {
            const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x & 255) >> 6);
            const T *first = p + (reverse ? len - t0 - kChunk : t0) * stride;
#pragma unroll
            for (int i = 0; i < Tile::N; ++i) {
                uint32_t o = off[i];
                if (n < kChunk) {
                    int row, slot;
                    Tile::source(i, row, slot);
                    if (row >= n) o = kSkip;
                }
                lds_load16(first, tile + (i * 256 + wave * 64) * Tile::E, o);
            }
        } else {
            const auto view = wide_view(p + (reverse ? len - t0 - kChunk : t0) * stride);
#pragma unroll
            for (int i = 0; i < Tile::N; ++i) {
                int row, slot;
                Tile::source(i, row, slot);
                const int col = col0 + slot * Tile::E;
                const uint32_t at = (uint32_t)(((reverse ? kChunk - 1 - row : row) * stride + col) * (int64_t)sizeof(T));
                T e[Tile::E];
#pragma unroll
                for (int j = 0; j < Tile::E; ++j)
                    e[j] = view_load<T>(view, (row < n) & (col + j < cols) ? at + j * (uint32_t)sizeof(T) : kSkip);
                __builtin_memcpy(tile + (i * 256 + (threadIdx.x & 255)) * Tile::E, e, 16);
            }
        }
    }
};

// Work item of workgroup id: ids go to the 8 XCDs in turn, so runs of set.share items are dealt to
// one XCD, whose L2 then holds what they have in common.
__device__ __forceinline__ void work_of(const DecaySet &set, uint32_t id, int &kind, int &zt, int &h, int64_t &blk) {
    const uint32_t run = set.share, round = id / (8 * run), in = id % (8 * run);
    uint32_t w = (round * 8 + in % 8) * run + in / 8;
    kind = w % set.kinds, w /= set.kinds;
    zt = w % set.ztiles, w /= set.ztiles;
    h = w % set.w[0].H;
    blk = w / set.w[0].H;
}

// Stages of tiles in LDS: the chunk in use and those on their way.  Three where two workgroups of
// them fit a CU's 160 KB, else two; without LDS-destination loads one.
constexpr int walk_stages(int bytes, bool vec) { return !vec ? 1 : (3 * bytes <= 78 * 1024 ? 3 : (2 * bytes <= 150 * 1024 ? 2 : 1)); }

// The walk.  MODE kSums: the part's own sum only (y, z read), for every part that another segment
// follows; kOut: outputs in the storage type; kOutAny: in it or fp32, by the walk (the choice costs
// registers, so the plain prompt has a kernel without it).  DXP: DX padded; NT: 16-column tiles of E per
// wave.  grid: work items (see work_of).
//
// What bounds it: 20 heads of 128 x 128 in bf16, 131072 tokens: 632 us for 2.69 GB read and written, 4.3 TB/s, so
// near the memory; the sums before it 335 to 362 us for 1.34 GB.  With few tokens a walk the serial chunk does:
// 1.8 us at 128 x 128 with one walk a CU (the gradients of 4 x 4096 tokens: 230 us for 128 chunks, the matrix
// units a quarter of the time busy).  Two workgroups a CU overlap little where heads share k and v and memory
// is no bound: packed prompts take 84 us for 22 chunks.  P is computed by each of the four waves: sharing it
// through LDS would put a barrier and a round trip between a chunk's products (not tried).
//
// fp16's look at the sizes of the state and of P costs instructions where two workgroups compete for a SIMD:
// gradients of 8 x 1000 tokens, 12 heads of 64: 67 us without, 70 with it; elsewhere it is hidden (prompts of
// 4 x 4096 and 131072 tokens, gradients of 4 x 4096: within 1 %).
enum WalkMode : int { kSums = 0, kOut = 1, kOutAny = 2 };
template <typename T, int DXP, int NT, int MODE, bool VEC>
__global__ __launch_bounds__(256, DXP <= 128 ? 2 : 1) void decay_walk_kernel(const DecaySet set) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass, which cannot take the scalar operands, needs the stub alone
    constexpr bool OUT = MODE != kSums;
    constexpr int KX = DXP / 32;          // 32-wide contraction steps over DX
    constexpr int DZT = NT * 64;          // z columns of a workgroup
    using TX = ChunkTile<T, DXP, false>;
    using TY = ChunkTile<T, DXP, true>;
    using TZ = ChunkTile<T, DZT, true>;
    using v8 = typename Mma<T>::v8;
    constexpr int kBytes = ((OUT ? 2 : 1) * TY::VALUES + TZ::VALUES) * (int)sizeof(T);
    constexpr int S = walk_stages(kBytes, VEC);
    constexpr int kLoads = (OUT ? 2 : 1) * TY::N + TZ::N;
    __shared__ __attribute__((aligned(128))) T x0[OUT ? TX::VALUES : 8], y0[TY::VALUES], z0[TZ::VALUES];
    __shared__ __attribute__((aligned(128))) T x1[OUT && S > 1 ? TX::VALUES : 8], y1[S > 1 ? TY::VALUES : 8], z1[S > 1 ? TZ::VALUES : 8];
    __shared__ __attribute__((aligned(128))) T x2[OUT && S > 2 ? TX::VALUES : 8], y2[S > 2 ? TY::VALUES : 8], z2[S > 2 ? TZ::VALUES : 8];
    __shared__ __attribute__((aligned(16))) float upd[2 * kChunk];   // u_scale d^(C - off - s): weight of token s in the next state
    __shared__ float row_w[kChunk];       // i_scale d^(i + off): weight of the chunk's first state in row i

    int kind, h, zt;
    int64_t blk;
    work_of(set, blockIdx.x, kind, zt, h, blk);
    const DecayWalk &a = set.w[kind];
    SegInfo si;
    if (blk >= a.nblk || zt * DZT >= a.DZ || !find_segment(a, blk, false, si)) return;
    si.seq = scalar(si.seq), si.index = scalar(si.index), si.count = scalar(si.count);
    si.start = scalar(si.start), si.len = scalar(si.len), si.slot = scalar(si.slot);
    if (!OUT && si.index >= parts_before_last(a, si.count)) return;
    // The final state comes from the last segment, of the walks that may be asked for one: whether it is
    // asked for changes no output's bits.
    const bool exact = !OUT || (a.keeps && si.index + 1 == si.count);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int col0 = zt * DZT;                   // first z column of the workgroup
    const int zw = wave * NT * 16;                       // this wave's columns within it
    const int64_t t_begin = si.index * a.seglen;
    const int64_t t_end = t_begin + a.seglen < si.len && si.index + 1 < si.count ? t_begin + a.seglen : si.len;
    const int64_t row0 = a.cu ? si.start : 0, batch = a.cu ? 0 : si.seq;
    const float log2d = a.log_decay[h] * kLog2e;

    for (int i = tid; i < 2 * kChunk; i += 256) upd[i] = i < kChunk ? a.u_scale * decay_power(log2d, kChunk - a.off - i) : 0.0f;
    for (int i = tid; i < kChunk; i += 256) row_w[i] = a.i_scale * decay_power(log2d, i + a.off);

    ChunkSource<T, DXP, false, VEC> src_x;
    ChunkSource<T, DXP, true, VEC> src_y;
    ChunkSource<T, DZT, true, VEC> src_z;
    if (OUT) src_x.init(a.x, batch, a.xb, row0, a.xt, h / a.gx, a.xh, si.len, a.DX, 0, a.reverse);
    src_y.init(a.y, batch, a.yb, row0, a.yt, h / a.gy, a.yh, si.len, a.DX, 0, a.reverse);
    src_z.init(a.z, batch, a.zb, row0, a.zt, h / a.gz, a.zh, si.len, a.DZ, col0, a.reverse);
    auto bring = [&](int64_t t, T *x, T *y, T *z) __attribute__((always_inline)) {
        const int n = t_end - t < kChunk ? (int)(t_end - t) : kChunk;
        if (OUT) src_x.bring(t, n, x);
        src_y.bring(t, n, y);
        src_z.bring(t, n, z);
    };
    if (S > 1 && t_begin < t_end) bring(t_begin, x0, y0, z0);
    if (S > 2 && t_begin + kChunk < t_end) bring(t_begin + kChunk, x1, y1, z1);

    // z column of accumulator column m of tile t (NT = 2: a lane's two tiles hold 8 neighbours)
    auto zcol = [&](int m, int t) { return zw + (NT == 2 ? (m >> 2) * 8 + t * 4 + (m & 3) : m); };

    // E[kk][r][t]: rows kk * 32 + g * 8 + r * 4 + i, column zcol(c, t)
    f32x4 E[KX][2][NT];
    {
        const float *s0 = nullptr;
        uint32_t sx_ = (uint32_t)a.s0x, sz_ = (uint32_t)a.s0z;
        if (a.seg && OUT) {
            s0 = a.seg + ((si.slot + si.index * (a.seglen / a.sublen)) * a.H + h) * (int64_t)a.DX * a.DZ;
            sx_ = (uint32_t)a.segx;
            sz_ = (uint32_t)a.segz;
        } else if (OUT && a.state0) {
            const int64_t slot = state_slot(a.slots, a.n_slots, si.seq);
            if (slot >= 0) s0 = a.state0 + (slot * a.H + h) * (int64_t)a.DX * a.DZ;
        }
        const auto view = wide_view(s0);
        if (OUT && a.seg && a.segx == 1 && a.DX % 4 == 0) {      // the segments' states: four rows of a column together
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int dx = kk * 32 + g * 8 + r * 4, dz = col0 + zcol(c, t);
                        E[kk][r][t] = view_load_wide<f32x4>(view, (dx < a.DX) & (dz < a.DZ) ? (uint32_t)(dx + dz * sz_) * 4u : kSkip);
                    }
        } else {
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int dx = kk * 32 + g * 8 + r * 4 + i, dz = col0 + zcol(c, t);
                            const uint32_t at = (uint32_t)(dx * sx_ + dz * sz_) * 4u;
                            E[kk][r][t][i] = view_load<float>(view, (s0 != nullptr) & (dx < a.DX) & (dz < a.DZ) ? at : kSkip);
                        }
        }
    }
    // decay of P in row tile rt, accumulator (r, i): d^(16 rt + c - 8 g - 4 r - i), 0 above the diagonal
    float fac[2][2][4];
    if (OUT) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 16 * rt + c - 8 * g - 4 * r - i;
                    fac[rt][r][i] = n < 0 ? 0.0f : a.p_scale * decay_power(log2d, n);
                }
    }
    const bool slow = __builtin_amdgcn_readfirstlane(fabsf(log2d) * kChunk <= 8.0f);   // the gain carries the decay
    const int zl = col0 + zw + (NT == 2 ? g * 8 : g * 4);      // this lane's first column of the output
    const int out_cols = a.DZ - zl;                             // and how many are left
    const uint32_t out_e = MODE == kOutAny && a.out_f32 ? 4u : (uint32_t)sizeof(T);
    char *out0 = static_cast<char *>(a.out) + (OUT ? (batch * a.ob + row0 * a.ot + (h / a.go) * a.oh) * out_e : 0);
    uint32_t out_off[2];        // this lane's places in a chunk's rows
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        const int row = rt * 16 + c;
        out_off[rt] = (out_cols > 0) & (a.out != nullptr) ? (uint32_t)((a.reverse ? kChunk - 1 - row : row) * a.ot + zl) * out_e : kSkip;
    }
    float grown = 0.0f;    // the accumulators hold E * 2^(grown + ex); grown = -log2 d * held
    int held = 0;
    int ex = 0;            // (ex: fp16 only, else 0)

    // one chunk at token t in (x, y, z); (nx, ny, nz) is free for the chunk S - 1 ahead
    auto chunk = [&](int64_t t, const T *x, const T *y, const T *z, T *nx, T *ny, T *nz) __attribute__((always_inline)) {
        if constexpr (S == 1) {
            __syncthreads();
            bring(t, nx, ny, nz);
            __syncthreads();
        } else {
            // this chunk's loads are the oldest; with three stages the next chunk's, if there is one,
            // may still travel (vmcnt retires in order; it counts the stores of the chunk before as well, so
            // as many of those loads have arrived, too).  The wait on LDS reads keeps every wave's
            // reads of the freed stage before the loads into it.
            if (S == 3 && t + kChunk < t_end) wait_loads_and_barrier<kLoads>();
            else wait_loads_and_barrier<0>();
            if (t + (S - 1) * kChunk < t_end) bring(t + (S - 1) * kChunk, nx, ny, nz);
        }
        const int n = t_end - t < kChunk ? (int)(t_end - t) : kChunk;
        // this wave's columns of Z, tokens 8 g .. 8 g + 7
        v8 zf[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q)
            zf[q] = TZ::col8(z, zw + (NT == 2 ? (lane & 3) * 8 + q * 4 : (lane & 3) * 4), zcol(c, q));
        if (OUT) {
            // fp16: the state is an operand as it is where the largest element in this wave's columns has room in the
            // type's range, else with that element at its upper end; outputs are brought back in fp32
            float unscale = Mma<T>::kNarrow ? ldexpf(__builtin_amdgcn_exp2f(-grown), -ex) : __builtin_amdgcn_exp2f(-grown), to = 1.0f;
            if (Mma<T>::kNarrow) {
                float top = 0.0f;
#pragma unroll
                for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(E[kk][j >> 2][q][j & 3]));
                const float size = top * unscale;
                const bool low = __ballot(size >= kFp16LowAll) == 0, high = __ballot(!(size <= kFp16High)) != 0;
                to = unscale;
                unscale = 1.0f;
                if (__builtin_expect(low | high, 0)) {
                    const int shift = fp16_shift(wave_max(size));
                    to = ldexpf(to, shift);
                    unscale = ldexpf(1.0f, -shift);
                }
            }
            v8 ef[KX][NT];     // the state as an operand: row zcol(c, q), slots 8 g + j
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float e = E[kk][j >> 2][q][j & 3];
                        ef[kk][q][j] = (T)(Mma<T>::kNarrow ? e * to : e);
                    }
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                f32x4 o[NT], p[2];
#pragma unroll
                for (int q = 0; q < NT; ++q) o[q] = f32x4{0, 0, 0, 0};
                p[0] = p[1] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kk = 0; kk < KX; ++kk) {
                    const v8 xf = TX::row8(x, rt * 16 + c, kk * 32 + g * 8);
#pragma unroll
                    for (int q = 0; q < NT; ++q) o[q] = Mma<T>::mma(ef[kk][q], xf, o[q]);
                    // rows of Y permuted: accumulator row m is token 8 (m / 4) + 4 r + m % 4
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        p[r] = Mma<T>::mma(TY::row8(y, (c >> 2) * 8 + r * 4 + (c & 3), kk * 32 + g * 8), xf, p[r]);
                }
                const float rw = row_w[rt * 16 + c] * unscale;
                float pw[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) pw[j] = p[j >> 2][j & 3] * fac[rt][j >> 2][j & 3];
                v8 pf;
                bool room = true;
                float top = 0.0f;
                if (Mma<T>::kNarrow) {      // P likewise, each row (one of the output's, the lanes of one c) by itself
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(pw[j]));
                    // (no short-circuit: one branch)
                    room = ((~rows_vote(top >= kFp16Low) & 0xffff) | (__ballot(!(top <= kFp16High)) != 0)) == 0;
                }
                if (__builtin_expect(room, 1)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) pf[j] = (T)pw[j];
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        o[q] *= rw;
                        o[q] = Mma<T>::mma(zf[q], pf, o[q]);
                    }
                } else {
                    const int shift = fp16_shift(rows_max(top));
                    const float rw_p = ldexpf(rw, shift), from = ldexpf(1.0f, -shift);
#pragma unroll
                    for (int j = 0; j < 8; ++j) pf[j] = (T)ldexpf(pw[j], shift);
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        o[q] *= rw_p;
                        o[q] = Mma<T>::mma(zf[q], pf, o[q]);
                        o[q] *= from;
                    }
                }
                {
                    const auto view = wide_view(out0 + (a.reverse ? si.len - t - kChunk : t) * a.ot * out_e);
                    const uint32_t off = rt * 16 + c < n ? out_off[rt] : kSkip;
                    if (MODE == kOutAny && a.out_f32) put_row<float, NT, VEC && sizeof(T) == 2>(view, off, o, a.vec_o, out_cols);
                    else put_row<T, NT, VEC && sizeof(T) == 2>(view, off, o, a.vec_o, out_cols);
                }
            }
        }
        // The gain after this chunk; brought back first where that leaves its range.  (Behind the outputs, which do not
        // wait for Z's largest value then: fp16, 4 x 4096 tokens of 20 x 128: gradients 285 against 294 us.)
        const float growth = slow ? (float)n * -log2d : 0.0f;
        held = slow ? held + n : 0;
        float next = slow ? (float)held * -log2d : 0.0f, most = 0.0f;
        bool back = fabsf(next) > 16.0f;
        float w[8], terms[NT][8];       // (terms: fp16)
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = upd[kChunk - n + g * 8 + j];
        if (Mma<T>::kNarrow) {
            // the largest of the terms themselves: a head that forgets fast may weigh all that a chunk holds by very little
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    terms[q][j] = (float)zf[q][j] * w[j];
                    most = fmaxf(most, fabsf(terms[q][j]));
                }
            most = wave_max(most);
            const float top = ldexpf(most * __builtin_amdgcn_exp2f(next), ex);
            back = back || top > 32768.0f || (top < 16.0f && most > 0.0f);
        }
        if (__builtin_amdgcn_readfirstlane(back)) {
            int e1 = 0;
            if (Mma<T>::kNarrow) {
                e1 = most > 0.0f ? 13 - ilogbf(most) - (int)ceilf(growth) : ex;     // the largest term near 2^14
                e1 = e1 < -60 ? -60 : (e1 > 60 ? 60 : e1);
            }
            const float r = ldexpf(__builtin_amdgcn_exp2f(-grown), e1 - ex);
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int r2 = 0; r2 < 2; ++r2)
#pragma unroll
                    for (int q = 0; q < NT; ++q) E[kk][r2][q] *= r;
            ex = e1;
            grown = 0.0f;
            held = slow ? n : 0;
            next = growth;
        }
        const float gain = Mma<T>::kNarrow ? ldexpf(__builtin_amdgcn_exp2f(next), ex) : __builtin_amdgcn_exp2f(next);
        // E <- d^n E + Y^T (weights Z), in units of the gain
        if (!slow) {
            const float dn = decay_power(log2d, n);
#pragma unroll
            for (int kk = 0; kk < KX; ++kk)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int q = 0; q < NT; ++q) E[kk][r][q] *= dn;
        }
        grown = next;
        if (!Mma<T>::kNarrow) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= gain;
        }
        auto update = [&](auto count) __attribute__((always_inline)) {
            constexpr int TERMS = decltype(count)::value;
            v8 zs[NT][TERMS];
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                float weighted[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) weighted[j] = Mma<T>::kNarrow ? terms[q][j] * gain : (float)zf[q][j] * w[j];
                split8<T, TERMS>(weighted, zs[q]);
            }
            // terms outermost: an accumulator's next product comes 2 NT instructions later, past their latency
#pragma unroll
            for (int kk = 0; kk < KX; ++kk) {
                // rows of the state permuted like zcol: row m is kk * 32 + 8 (m / 4) + 4 r + m % 4
                v8 yf[2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    yf[r] = TY::col8(y, kk * 32 + (lane & 3) * 8 + r * 4, kk * 32 + (c >> 2) * 8 + r * 4 + (c & 3));
#pragma unroll
                for (int p = 0; p < TERMS * Mma<T>::kParts; ++p)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int q = 0; q < NT; ++q)
                            E[kk][r][q] = Mma<T>::mma(yf[r], zs[q][p / Mma<T>::kParts], E[kk][r][q], p % Mma<T>::kParts);
            }
        };
        constexpr int kExact = Mma<T>::kExactTerms, kTerms = Mma<T>::kTerms;
        if (!OUT || kExact == kTerms || exact) update(std::integral_constant<int, kExact>{});
        else update(std::integral_constant<int, kTerms>{});
    };
    __syncthreads();       // the tables above
    for (int64_t t = t_begin; t < t_end; t += S * kChunk) {
        if constexpr (S == 1) {
            chunk(t, x0, y0, z0, x0, y0, z0);
        } else if constexpr (S == 2) {
            chunk(t, x0, y0, z0, x1, y1, z1);
            if (t + kChunk < t_end) chunk(t + kChunk, x1, y1, z1, x0, y0, z0);
        } else {
            chunk(t, x0, y0, z0, x2, y2, z2);
            if (t + kChunk < t_end) chunk(t + kChunk, x1, y1, z1, x0, y0, z0);
            if (t + 2 * kChunk < t_end) chunk(t + 2 * kChunk, x2, y2, z2, x1, y1, z1);
        }
    }

    const float unscale = ldexpf(exp2f(-grown), -ex);
    float *s1 = nullptr;
    uint32_t sx_ = (uint32_t)a.s1x, sz_ = (uint32_t)a.s1z;
    if (!OUT) {
        s1 = a.seg + ((si.slot + si.index) * a.H + h) * (int64_t)a.DX * a.DZ;
        sx_ = (uint32_t)a.segx;
        sz_ = (uint32_t)a.segz;
    } else if (a.state1 && si.index + 1 == si.count) {
        const int64_t slot = state_slot(a.slots, a.n_slots, si.seq);
        if (slot >= 0) s1 = a.state1 + (slot * a.H + h) * (int64_t)a.DX * a.DZ;
    }
    if (!s1) return;
    const auto view = wide_view(s1);
    if (!OUT && sx_ == 1 && a.DX % 4 == 0) {
#pragma unroll
        for (int kk = 0; kk < KX; ++kk)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int dx = kk * 32 + g * 8 + r * 4, dz = col0 + zcol(c, t);
                    const f32x4 e = E[kk][r][t] * unscale;
                    view_store(view, (dx < a.DX) & (dz < a.DZ) ? (uint32_t)(dx + dz * sz_) * 4u : kSkip, e);
                }
        return;
    }
#pragma unroll
    for (int kk = 0; kk < KX; ++kk)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int dx = kk * 32 + g * 8 + r * 4 + i, dz = col0 + zcol(c, t);
                    const uint32_t at = (uint32_t)(dx * sx_ + dz * sz_) * 4u;
                    const float e = E[kk][r][t][i] * unscale;
                    view_store(view, (dx < a.DX) & (dz < a.DZ) ? at : kSkip, e);
                }
#endif
}

// The single-token form: E <- d E + k v^T, out = scale E^T q, one workgroup per (sequence,
// head, tile of LANES * VEC value columns); LANES lanes along a row of the state, the other
// 256 / LANES row groups share its rows, joined through LDS.  Bound by the state, which is read and
// written once: U rows of it are on their way in each lane.  256 sequences x 20 heads of 128 x 128 (676 MB):
// 137 us, 4.9 TB/s, what a copy of 2 GiB reaches; 12 heads of one sequence: 3.3 us, a launch.
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

// grid (blocks, tensors): a thread sums the group's values of V neighbouring columns, in the heads' order (no
// atomics).  Bound by the fp32 parts it reads: 8 x 1000 tokens, 12 heads of 64 in groups of 3, both tensors (57 MB
// in and out): 10 us.
template <typename T, int V> __global__ __launch_bounds__(256) void decay_group_sum_kernel(const DecayGroupSum a) {
    const int k = blockIdx.y;
    if (!a.dst[k] || (V == 4) != (a.vec[k] != 0)) return;
    typedef float vec __attribute__((ext_vector_type(V)));
    const int D = a.D[k], Q = D / V;
    // sequences lie one behind another: the tokens between the first bound and the last, clamped like the walks'
    int64_t first = 0, end = a.B * a.N;
    if (a.cu) {
        const int64_t s = a.cu[0], e = a.cu[a.seqs];
        first = s < 0 ? 0 : (s > a.N ? a.N : s);
        end = e < first ? first : (e > a.N ? a.N : e);
    }
    const int64_t n = (end - first) * a.Hk * Q;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int d = (int)(i % Q) * V;
        const int64_t head = i / Q + first * a.Hk, hk = head % a.Hk, t = head / a.Hk;
        const float *p = a.src[k] + head * a.group * D + d;
        vec s = 0.0f;
        for (int j = 0; j < a.group; ++j) s += *reinterpret_cast<const vec *>(p + (int64_t)j * D);
        T *q = static_cast<T *>(a.dst[k]) + t / a.N * a.db[k] + t % a.N * a.dt[k] + hk * a.dh[k] + d;
        T w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = (T)s[j];
        __builtin_memcpy(__builtin_assume_aligned(q, V * sizeof(T)), w, sizeof w);
    }
}

// State before each segment from the parts' own sums, in place:
// grid (B, H, kinds x pieces of 256 V values).  V = 4: Dx * Dz a multiple of 4.  A thread follows its values
// through all parts of a sequence, eight parts' loads ahead.  Latency bound: 15 us at 131072 tokens x 20
// heads of 128 x 128.
template <int V> static __global__ __launch_bounds__(256) void decay_chain_kernel(const DecaySet set) {
    const DecayWalk &a = set.w[blockIdx.z % set.kinds];
    typedef float vec __attribute__((ext_vector_type(V)));
    SegInfo si;
    if (!find_segment(a, blockIdx.x, true, si)) return;
    const int h = blockIdx.y;
    const uint32_t nst = (uint32_t)(a.DX * a.DZ), e = (blockIdx.z / set.kinds * 256 + threadIdx.x) * V;
    if (e >= nst) return;
    // place in a state whose element (x, z) is at x sx + z sz of what lies at e + i in a segment's
    auto place = [&](int i, uint32_t sx, uint32_t sz) {
        const uint32_t row = (uint32_t)(a.segx == 1 ? a.DX : a.DZ), hi = (e + i) / row, lo = e + i - hi * row;
        return a.segx == 1 ? lo * sx + hi * sz : hi * sx + lo * sz;
    };
    const float log2d = a.log_decay[h] * kLog2e;
    const float dn = decay_power(log2d, a.seglen);
    const int64_t slot = state_slot(a.slots, a.n_slots, si.seq);
    vec run = 0.0f;
    if (slot >= 0 && a.state0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            run[i] = a.state0[(slot * a.H + h) * nst + place(i, (uint32_t)a.s0x, (uint32_t)a.s0z)];
    }
    float *p = a.seg + (si.slot * a.H + h) * nst + e;
    const int64_t step = (int64_t)a.H * nst;
    const int64_t sums = parts_before_last(a, si.count);     // the state behind them is the last segment's
    constexpr int U = 8;
    int to_state = 0;       // parts until the next segment starts
    for (int64_t s = 0; s <= sums; s += U) {
        vec own[U];
#pragma unroll
        for (int j = 0; j < U; ++j) own[j] = s + j < sums ? *reinterpret_cast<const vec *>(p + (s + j) * step) : (vec)0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (s + j <= sums) {
                if (to_state == 0) *reinterpret_cast<vec *>(p + (s + j) * step) = run;
                to_state = to_state == 0 ? a.parts - 1 : to_state - 1;
                run = dn * run + own[j];
            }
    }
}

// ---- host side of one storage type ----------------------------------------
template <typename T, int MODE, bool VEC> static hipError_t walk_launch(const DecaySet &set, hipStream_t stream) {
    bool narrow = true;
    int dx = 0;
    for (int i = 0; i < set.kinds; ++i) {
        narrow = narrow && set.w[i].ztile == 64;
        dx = set.w[i].DX > dx ? set.w[i].DX : dx;
    }
    const int64_t items = set.w[0].nblk * set.w[0].H * set.ztiles * set.kinds, round = 8 * (int64_t)set.share;
    const unsigned grid = (unsigned)((items + round - 1) / round * round);
    // (rows wider than 128 leave registers for 64 z columns only: decay_z_tile)
    if (dx > 128) {
        if (!narrow) return hipErrorInvalidValue;
        decay_walk_kernel<T, 256, 1, MODE, VEC><<<grid, 256, 0, stream>>>(set);
    } else if (dx > 64) {
        if (narrow) decay_walk_kernel<T, 128, 1, MODE, VEC><<<grid, 256, 0, stream>>>(set);
        else decay_walk_kernel<T, 128, 2, MODE, VEC><<<grid, 256, 0, stream>>>(set);
    } else {
        if (narrow) decay_walk_kernel<T, 64, 1, MODE, VEC><<<grid, 256, 0, stream>>>(set);
        else decay_walk_kernel<T, 64, 2, MODE, VEC><<<grid, 256, 0, stream>>>(set);
    }
    return hipGetLastError();
}

template <typename T> static hipError_t walks_typed(const DecaySet &set, hipStream_t stream) {
    bool vec = true, any = false;
    for (int i = 0; i < set.kinds; ++i) {
        vec = vec && set.w[i].vec_x && set.w[i].vec_y && set.w[i].vec_z && set.w[i].vec_o;
        any = any || set.w[i].out_f32;
    }
    if (!vec) return walk_launch<T, kOutAny, false>(set, stream);
    return any ? walk_launch<T, kOutAny, true>(set, stream) : walk_launch<T, kOut, true>(set, stream);
}

template <typename T> static hipError_t sums_typed(const DecaySet &set, hipStream_t stream) {
    if (!set.w[0].seg) return hipSuccess;
    bool vec = true;
    for (int i = 0; i < set.kinds; ++i) vec = vec && set.w[i].vec_y && set.w[i].vec_z;
    const hipError_t e = vec ? walk_launch<T, kSums, true>(set, stream) : walk_launch<T, kSums, false>(set, stream);
    if (e != hipSuccess) return e;
    const int64_t nst = (int64_t)set.w[0].DX * set.w[0].DZ;
    const bool quads = nst % 4 == 0;
    const unsigned pieces = (unsigned)((nst + (quads ? 1023 : 255)) / (quads ? 1024 : 256));
    const dim3 grid((unsigned)set.w[0].B, (unsigned)set.w[0].H, pieces * set.kinds);
    if (quads) decay_chain_kernel<4><<<grid, 256, 0, stream>>>(set);
    else decay_chain_kernel<1><<<grid, 256, 0, stream>>>(set);
    return hipGetLastError();
}

template <typename T> static hipError_t step_typed(const DecayStep &a, bool vec, hipStream_t stream) {
    const unsigned bh = (unsigned)(a.B * a.H);
    if (!vec) {
        decay_step_kernel<T, 1, 32><<<dim3(bh, (a.Dv + 31) / 32), 256, 0, stream>>>(a);
    } else if (bh * ((a.Dv + 127) / 128) < 352) {
        // few states: tiles of 32 columns spread them over more compute units.  128 x 128 states, back to
        // back, narrow against wide: 3.3 against 4.1 us for 12, 6.3 / 6.9 for 256, 7.1 / 7.7 for 320, 10.8 / 10.2
        // for 384, 11.1 / 10.0 for 512; 256 x 256: 15.0 / 15.6 for 160, 17.8 / 17.5 for 192.
        decay_step_kernel<T, 4, 8><<<dim3(bh, (a.Dv + 31) / 32), 256, 0, stream>>>(a);
    } else {
        decay_step_kernel<T, 4, 32><<<dim3(bh, (a.Dv + 127) / 128), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T> static hipError_t group_sum_typed(const DecayGroupSum &a, hipStream_t stream) {
    int64_t most[2] = {0, 0};     // threads of the tensors met value by value, and four at a time
    for (int k = 0; k < 2; ++k)
        if (a.dst[k]) {
            const int64_t n = a.B * a.N * a.Hk * a.D[k] / (a.vec[k] ? 4 : 1);
            most[a.vec[k] != 0] = n > most[a.vec[k] != 0] ? n : most[a.vec[k] != 0];
        }
    auto grid = [](int64_t n) { return dim3((unsigned)(n / 256 < 4096 ? n / 256 + 1 : 4096), 2); };
    if (most[1]) decay_group_sum_kernel<T, 4><<<grid(most[1]), 256, 0, stream>>>(a);
    if (most[0]) decay_group_sum_kernel<T, 1><<<grid(most[0]), 256, 0, stream>>>(a);
    return hipGetLastError();
}

#define FFTCONV_DECAY_TYPE(NAME, T)                                                                                      \
    hipError_t launch_decay_sums_##NAME(const DecaySet &set, hipStream_t s) { return sums_typed<T>(set, s); }             \
    hipError_t launch_decay_walks_##NAME(const DecaySet &set, hipStream_t s) { return walks_typed<T>(set, s); }           \
    hipError_t launch_decay_step_##NAME(const DecayStep &a, bool vec, hipStream_t s) { return step_typed<T>(a, vec, s); } \
    hipError_t launch_decay_group_sum_##NAME(const DecayGroupSum &a, hipStream_t s) { return group_sum_typed<T>(a, s); }

}  // namespace fftconv
