// sequence_ops.hpp -- what the host side of the decay-attention and
// linear-product operators (sequence_ops.cpp) passes to their kernels
// (decay_kernels.hpp, linear_kernels.hpp), and the launchers per storage type.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fftconv {

// z columns of a workgroup's state: 128 (two 16-column tiles for each of four waves), 64 where no more are
// needed or the state's rows leave no registers for more.
inline int decay_z_tile(int64_t dx, int64_t dz) { return dz <= 64 || dx > 128 ? 64 : 128; }

// One walk over sequences: the prompt form, or one gradient (decay_kernels.hpp).
struct DecayWalk {
    const void *x, *y, *z;
    void *out;
    int64_t xb, xt, xh, yb, yt, yh, zb, zt, zh, ob, ot, oh;   // strides (batch, token, head), elements
    int gx, gy, gz, go;              // heads that share one x / y / z / out head
    const float *log_decay;          // (H)
    const float *state0;             // initial state or null; (slots or B, H) matrices of DX * DZ
    float *state1;                   // final state or null
    int64_t s0x, s0z, s1x, s1z;      // element strides of a state along DX and DZ
    const int32_t *slots;            // state slot of each sequence or null
    int64_t n_slots;
    const int32_t *cu;               // packed sequences' bounds (B + 1) or null
    int64_t B, N;                    // N: tokens of each sequence, or of all when packed
    int H, DX, DZ;
    int ztile;                       // z columns of a workgroup
    int64_t seglen;                  // tokens per segment, a multiple of sublen
    int64_t sublen;                  // tokens per part that has a sum of its own, a multiple of the chunk
    int parts;                       // seglen / sublen of the walks
    int64_t nblk;                    // segments launched (an upper bound when packed)
    float *seg;                      // state before each part, (parts, H) matrices, null when one segment each
    int64_t segx, segz;              // their strides along DX and DZ
    float p_scale, u_scale, i_scale;
    int off, reverse;
    int keeps;                       // this kind of walk can return its final state
    int vec_x, vec_y, vec_z, vec_o;  // 16-byte access allowed
    int out_f32;                     // out is fp32 (a part of a sum over heads), else the storage type
};

// Walks that one launch runs side by side: they have the same sequences, segments and H, and the same
// padded widths.  Work is dealt to the chip in runs of `share` neighbours (walk fastest, then z tile,
// head, segment), which read the same tensors and land on one XCD.
struct DecaySet {
    DecayWalk w[3];
    int kinds;       // walks in use
    int ztiles;      // z tiles of a walk (of the widest)
    int share;
};

// One single-token step (decay_kernels.hpp).
struct DecayStep {
    const void *q, *k, *v;
    void *out;
    int64_t qb, qh, kb, kh, vb, vh, ob, oh;
    const float *log_decay;
    float *state;
    const int32_t *slots;
    int64_t n_slots, B;
    int H, group, Dk, Dv;
    float scale;
};

// Gradients of shared heads: dst (tokens, Hk, D) <- sum over each group of src (tokens, H, D), fp32.  When packed,
// of the tokens that belong to a sequence: src holds nothing for the others, and dst keeps what it has there.
struct DecayGroupSum {
    const float *src[2];
    void *dst[2];                    // up to two tensors; null: none
    int D[2], vec[2];                // vec: four values at a time
    int64_t db[2], dt[2], dh[2];     // strides of dst
    int64_t B, N;
    const int32_t *cu;               // packed sequences' bounds (seqs + 1) or null
    int64_t seqs;
    int Hk, group;
};

enum LinearAct : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
enum LinearLayout : int { LAYOUT_NT = 0, LAYOUT_NN = 1, LAYOUT_TN = 2 };

// One product C[m][n] = sum_k A(m, k) B(n, k) with its epilogue (linear_kernels.hpp).
struct LinearGemm {
    const void *A, *B;
    int64_t lda, ldb;
    int64_t M, N, K;
    void *C;
    int64_t ldc;
    const void *bias, *res;   // null: none
    int64_t ldr;
    void *pre;                // null: not kept
    int64_t ldp;
    int act;
    int vec_c, vec_r, vec_p, vec_b;   // 4-value access allowed
    int quads;                // N a multiple of 4, 4-value access everywhere, a tile's rows within 31 bits
    // Tiles below `full` are computed whole; each of the others in `splits` parts of kper of K (whole
    // stages), whose sums go to part (tile-sized matrices, fp32) and are joined by a second kernel.
    int64_t tiles, full;
    int splits;
    int64_t kper;
    float *part;
};

// dz = dout * act'(pre) into rows of ldz (zeros behind N), and column sums of slabs of rows.
struct LinearDz {
    const void *dout, *pre;
    int64_t ldo, ldp, M, N;
    int act;
    void *dz;          // null: not written (act none, dout itself is used)
    int64_t ldz;
    float *colsum;     // slabs x N, null: no bias gradient
    int64_t rows;      // rows of a slab
    int vec;           // rows of whole 16-byte pieces
};

// sums of segments and their chain (nothing when the walks are not segmented), then the walks
hipError_t launch_decay_sums_f16(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_walks_f16(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_step_f16(const DecayStep &a, bool vec, hipStream_t stream);
hipError_t launch_decay_group_sum_f16(const DecayGroupSum &a, hipStream_t stream);
hipError_t launch_linear_gemm_f16(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t stream);
hipError_t launch_linear_vector_f16(const LinearGemm &a, bool vec, hipStream_t stream);
hipError_t launch_linear_dz_f16(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t stream);
// sums of segments and their chain (nothing when the walks are not segmented), then the walks
hipError_t launch_decay_sums_bf16(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_walks_bf16(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_step_bf16(const DecayStep &a, bool vec, hipStream_t stream);
hipError_t launch_decay_group_sum_bf16(const DecayGroupSum &a, hipStream_t stream);
hipError_t launch_linear_gemm_bf16(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t stream);
hipError_t launch_linear_vector_bf16(const LinearGemm &a, bool vec, hipStream_t stream);
hipError_t launch_linear_dz_bf16(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t stream);
// sums of segments and their chain (nothing when the walks are not segmented), then the walks
hipError_t launch_decay_sums_f32(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_walks_f32(const DecaySet &s, hipStream_t stream);
hipError_t launch_decay_step_f32(const DecayStep &a, bool vec, hipStream_t stream);
hipError_t launch_decay_group_sum_f32(const DecayGroupSum &a, hipStream_t stream);
hipError_t launch_linear_gemm_f32(const LinearGemm &a, int layout, int tile, bool vec, hipStream_t stream);
hipError_t launch_linear_vector_f32(const LinearGemm &a, bool vec, hipStream_t stream);
hipError_t launch_linear_dz_f32(const LinearDz &a, int64_t slabs, void *dbias, hipStream_t stream);

}  // namespace fftconv
