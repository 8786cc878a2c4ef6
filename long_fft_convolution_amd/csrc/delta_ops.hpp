// delta_ops.hpp -- what the host side of the gated delta rule (delta_ops.cpp)
// passes to its kernels (delta_kernels.hpp), and the launchers per storage type.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sequence_ops.hpp"

namespace fftconv {

constexpr int kDeltaChunk = 64;      // tokens of a chunk

// What the walks read of one (chunk, head), written by the first kernel, in pieces of 1 KB (16 bytes a lane): the
// inverse as 6 operands of three bf16 terms, 4 vectors of the tokens, the masked products as 6 operands of `terms`
// terms; padded to a multiple of four.
constexpr int kDeltaInverse = 18, kDeltaVectors = 1;
constexpr int delta_pieces(int terms) { return (kDeltaInverse + kDeltaVectors + 6 * terms + 3) / 4 * 4; }
// terms of the masked products, as of all else that outputs see: two for 16 bits (one would be a rounding as large as a
// bf16 result's own), three for fp32
constexpr int delta_terms(int elem_bytes) { return elem_bytes == 4 ? 3 : 2; }
// The backward call's record: the inverse of I + C diag(beta), the vectors, then, as operands over tokens from the
// other side, the inverse of I + C^T diag(beta) in three terms and P^T in fp32 (two halves of an operand).
constexpr int kDeltaBackProducts = 12;
constexpr int kDeltaBackPieces = (2 * kDeltaInverse + kDeltaVectors + kDeltaBackProducts + 3) / 4 * 4;

struct DeltaArgs {
    const void *q, *k, *v;           // q and k have H / group heads, v and out H
    void *out;
    int64_t qb, qt, qh, kb, kt, kh, vb, vt, vh, ob, ot, oh;   // strides (batch, token, head), elements
    const float *log_decay, *beta;   // (B, N, H) or (N, H)
    float scale;
    const int32_t *cu;               // packed sequences' bounds (B + 1) or null
    int64_t B, N;                    // N: tokens of each sequence, or of all when packed
    int H, group, Dk, Dv;
    const float *state0;             // initial states or null
    float *state1;                   // final states or null
    const int32_t *slots;            // state slot of each sequence or null
    int64_t n_slots;
    int64_t chunks;                  // places for chunks (an upper bound when packed)
    int64_t seg_chunks, segs;        // chunks of a segment, places for segments
    char *rec;                       // (chunks, H) records
    int64_t rec_bytes;
    // (segs, H) matrices of padded rows: a segment's own sum, what it makes of the state before it, and that state;
    // null: one segment each
    float *seg_sum, *seg_map, *seg_state;
    int sum_ld, map_ld;              // row lengths: seg_sum and seg_state, seg_map
    int vec;                         // rows of the tensors in whole aligned 16-byte pieces
    int wide;                        // 128 columns of the state a workgroup, else 64

    // backward
    const void *dout;
    int64_t gb, gt, gh;
    const float *dstate1;            // gradients of the final states or null
    float *dstate0;                  // gradients of the initial states or null
    int dkp, dvp;                    // padded widths of what follows
    float *states, *grads;           // (chunks, H) dkp x dvp: state before a chunk, gradient of the state behind it
    float *wrong, *dright;           // (chunks, H) 64 x dvp: w, and the gradient of u (its own and what later tokens of the chunk add)
    void *dq, *dk, *dv;              // null = skip; dq and dk fp32 (tokens, H, Dk) parts where heads share them
    int64_t dqb, dqt, dqh, dkb, dkt, dkh, dvb, dvt, dvh;
    int parts;                       // dq and dk are such parts
    float *dlog_decay, *dbeta;       // null = skip
};

struct DeltaStep {
    const void *q, *k, *v;
    void *out;
    int64_t qb, qh, kb, kh, vb, vh, ob, oh;
    const float *log_decay, *beta;   // (B, H)
    float *state;
    const int32_t *slots;
    int64_t n_slots, B;
    int H, group, Dk, Dv;
    float scale;
};

#define FFTCONV_DELTA_LAUNCHERS(NAME)                                                       \
    hipError_t launch_delta_prepare_##NAME(const DeltaArgs &a, hipStream_t stream);         \
    hipError_t launch_delta_fwd_##NAME(const DeltaArgs &a, hipStream_t stream);             \
    hipError_t launch_delta_bwd_##NAME(const DeltaArgs &a, hipStream_t stream);             \
    hipError_t launch_delta_step_##NAME(const DeltaStep &a, bool vec, hipStream_t stream);
FFTCONV_DELTA_LAUNCHERS(f32)
FFTCONV_DELTA_LAUNCHERS(f16)
FFTCONV_DELTA_LAUNCHERS(bf16)
#undef FFTCONV_DELTA_LAUNCHERS

}  // namespace fftconv
