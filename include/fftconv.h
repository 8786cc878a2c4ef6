/*
 * fftconv.h -- C ABI of the MI355X (gfx950) exact long causal FFT convolution.
 *
 * The operation (FlashFFTConv summary page, "Summary": a fused kernel that
 * computes *exact* FFT convolutions for long sequences, with partial and
 * frequency-sparse variants; "Problem": filters as long as the sequence;
 * "Measured effects", row on fusing gating into the convolution: the gated
 * form) is, for every batch row b and channel h,
 *
 *     out[b,h,t] = v[b,h,t] * sum_{s=0}^{min(t, L-1)} k[h,s] * u[b,h,t-s] * w[b,h,t-s]
 *                = v * irfft( rfft(pad(u*w, 2N)) * rfft(pad(k, 2N)) )[:N]      (t < N)
 *
 * computed through the convolution theorem with an FFT of size 2N.  With a
 * frequency mask ("Approach": sparsity realised by skipping blocks of the
 * matmuls; "Key results": 79 % of frequency-domain filter entries zeroed) the
 * filter spectrum's bins in zeroed blocks are treated as zero:
 *
 *     out = v * irfft( rfft(pad(u*w, 2N)) * (mask o rfft(pad(k, 2N))) )[:N]
 *
 * Mask blocks: the N+1 rfft bins f in [0, N] form 128 blocks of N/128 bins
 * (block = min(f / (N/128), 127), so the Nyquist bin N joins block 127); the
 * Hermitian mirror 2N-f of each bin follows it.
 *
 * Conventions for every function below:
 *  - Tensors are DEVICE pointers owned by the caller, dense and row-major:
 *      u, w, v, out : (B, H, N)  storage dtype
 *      k            : (H, L)     storage dtype
 *      mask         : (H, fftconv_mask_blocks(N)) uint8, 1 = keep, 0 = zero
 *    Every tensor pointer must be 16-byte aligned.  `out` must not overlap
 *    any input.
 *  - K_f (the prepared filter) is a caller-allocated device buffer of
 *    fftconv_filter_bytes() bytes.  Its contents are library-defined and
 *    opaque: a header (magic, version, N, H, L, dtype), one fp32 scale per
 *    channel, then the filter spectrum in the order the forward kernels read
 *    it (fp32 bins for FFTCONV_F32, scaled fp16 bins for FFTCONV_F16 and
 *    FFTCONV_BF16).  It depends on N and dtype, not on B.
 *  - Workspace: sequences longer than the largest on-chip size stream through
 *    HBM in several passes and need fftconv_workspace_bytes() bytes of device
 *    scratch, owned by the caller; 0 bytes (and a NULL pointer) suffice
 *    otherwise.
 *  - Supported sizes: N a power of two in [1024, 4194304]; 1 <= L <= N;
 *    B, H >= 0 (B*H == 0 enqueues nothing and returns FFTCONV_OK).
 *  - Every call is asynchronous on `stream` (a HIP stream, NULL = the default
 *    stream) unless stated otherwise, and returns a status; arguments are
 *    validated before anything is enqueued, so on any error status nothing
 *    was launched.  fftconv_last_error() gives the detail of the calling
 *    thread's last non-OK status.  Calls on different streams may run
 *    concurrently; the library's only shared state is a per-device cache of
 *    constant tables (twiddles, DFT operand tiles) guarded by a mutex.
 *  - Range (fp16 and bf16 storage).  Every size runs on the matrix-core
 *    kernels (N = 1024; N = 2048 .. 16384; the row pass of N > 16384, and its
 *    column passes for N >= 2^21), which round every transform stage to fp16
 *    (fp32 accumulation); power-of-two factors folded into their DFT tables
 *    keep the stage results within a small factor of the input (about
 *    rms(u*w) for a zero-mean input).  Overflow needs |u*w| near the fp16
 *    maximum 65504 (bf16 magnitudes beyond it are not representable on these
 *    paths), or a mean m of u*w whose zero-frequency bin passes it: 32 m at
 *    N = 1024, 64 m to 256 m at N = 2048 .. 16384, at most 4096 m for
 *    N > 16384 (|m| < 15 is safe at every N).  Nothing is clamped: an
 *    overflow gives inf / NaN.  fp32 storage has fp32 range.
 *  - The constant tables of a device are built once, by fftconv_init() or by
 *    the first fftconv_prepare_filter / fftconv_prepare_short_filter on that
 *    device: that one call allocates device memory and copies synchronously.
 *    After it, no call of this library allocates device memory or waits for
 *    the GPU (apart from the functions marked SYNCHRONOUS), so the forward
 *    and backward calls may be captured into a HIP graph.  A forward or
 *    backward call on a device where neither ran builds the tables itself,
 *    allocating and blocking like fftconv_init.
 */
#ifndef FFTCONV_H
#define FFTCONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same opaque type as HIP's hipStream_t. */
typedef struct ihipStream_t *hipStream_t;

typedef enum {
    FFTCONV_F32 = 0,  /* fp32 storage, fp32 arithmetic                          */
    FFTCONV_F16 = 1,  /* fp16 storage, fp32 accumulation                        */
    FFTCONV_BF16 = 2  /* bf16 storage, fp32 accumulation                        */
} fftconv_dtype_t;

typedef enum {
    FFTCONV_OK = 0,
    FFTCONV_ERR_INVALID_ARGUMENT = 1, /* null/misaligned pointer, bad size, overlap  */
    FFTCONV_ERR_UNSUPPORTED = 2,      /* N not a supported power of two, bad dtype   */
    FFTCONV_ERR_WORKSPACE = 3,        /* workspace smaller than required             */
    FFTCONV_ERR_FILTER_MISMATCH = 4,  /* K_f prepared for another N, H, L or dtype   */
    FFTCONV_ERR_HIP = 5               /* a HIP runtime call or kernel launch failed  */
} fftconv_status_t;

/* Bytes of the prepared-filter buffer K_f for H channels at sequence length N.
 * Returns 0 for unsupported N, dtype or H < 1. */
size_t fftconv_filter_bytes(int64_t H, int64_t N, fftconv_dtype_t dtype);

/* Bytes of device scratch fftconv_fwd needs for B*H sequences of length N
 * (fftconv_prepare_filter needs the value for B = 1).  0 when the whole
 * sequence fits on chip.  Returns 0 for unsupported arguments. */
size_t fftconv_workspace_bytes(int64_t B, int64_t H, int64_t N, fftconv_dtype_t dtype);

/* Number of frequency blocks per channel the mask addresses (128 for every
 * supported N; 0 for unsupported N). */
int64_t fftconv_mask_blocks(int64_t N);

/* Transform the time-domain filter k (H, L_filter) into K_f for sequences of
 * length N: K_f holds rfft(pad(k, 2N)) ("Approach": the filter spectrum the
 * convolution multiplies by; partial convolution = L_filter < N, where only
 * the L_filter taps are read and the padding is implicit).  fp16 / bf16 at
 * N = 2048 .. 16384 transform on the matrix cores with fp16 stages (about
 * 1e-3 relative error of the stored spectrum, like the forward call's own
 * stages); other sizes and fp32 in fp32.  Needs workspace of
 * fftconv_workspace_bytes(1, H, N, dtype) bytes for N beyond the on-chip
 * size.  K_f_bytes must be >= fftconv_filter_bytes(H, N, dtype). */
fftconv_status_t fftconv_prepare_filter(const void *k, int64_t H, int64_t L_filter, int64_t N,
                                        fftconv_dtype_t dtype, void *K_f, size_t K_f_bytes,
                                        void *workspace, size_t workspace_bytes,
                                        hipStream_t stream);

/* Gated causal FFT convolution (formula in the file header).
 *   u        input (B, H, N), required
 *   K_f      filter prepared by fftconv_prepare_filter for the same H, L_filter,
 *            N and dtype (checked against its header only when the
 *            environment variable FFTCONV_CHECK=1 is set, since that check
 *            synchronises)
 *   w, v     input and output gates (B, H, N); NULL = no gate
 *   out      output (B, H, N)
 *   sparsity_mask  (H, fftconv_mask_blocks(N)) uint8 device array, or NULL
 *            for a dense filter spectrum
 *   workspace / workspace_bytes  device scratch, see fftconv_workspace_bytes */
fftconv_status_t fftconv_fwd(const void *u, const void *K_f, const void *w, const void *v,
                             void *out, int64_t B, int64_t H, int64_t N, int64_t L_filter,
                             const uint8_t *sparsity_mask, fftconv_dtype_t dtype,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): fftconv_fwd
 * with the same arguments except the workspace, which comes from a static
 * device array of the library (fftconv_fwd_noalloc_scratch_bytes() bytes,
 * one copy per device, held until the process ends).  fftconv_init() must
 * have run on the calling thread's current device (else
 * FFTCONV_ERR_INVALID_ARGUMENT); the call then allocates nothing.  Sequences
 * longer than the on-chip size run through the scratch in chunks of as many
 * sequences as it holds (every supported N fits one sequence); the results are
 * those of fftconv_fwd bit for bit.  Every call on one device shares that
 * device's scratch, which keeps the last call's contents (nothing in it needs
 * to start at zero): calls that may overlap in time on one device (other
 * streams, other threads) race and must be serialised by the caller. */
fftconv_status_t fftconv_fwd_noalloc(const void *u, const void *K_f, const void *w, const void *v,
                                     void *out, int64_t B, int64_t H, int64_t N, int64_t L_filter,
                                     const uint8_t *sparsity_mask, fftconv_dtype_t dtype, hipStream_t stream);

/* Bytes of the static scratch of fftconv_fwd_noalloc (72 MiB). */
size_t fftconv_fwd_noalloc_scratch_bytes(void);

/* Device scratch bytes fftconv_fwd_taps needs: the prepared spectrum of the
 * H filters (fftconv_filter_bytes, rounded up to 256 bytes) followed by the
 * larger of the prepare's and the forward call's scratch.  0 for unsupported
 * N or dtype, H < 1 or B < 0. */
size_t fftconv_fwd_taps_workspace_bytes(int64_t B, int64_t H, int64_t N, fftconv_dtype_t dtype);

/* Forward call from the time-domain filter ("Approach", FlashFFTConv summary
 * page: a partial convolution's filter has fewer taps than the sequence, and
 * only the blocks that hold taps are transformed).  Equivalent to
 * fftconv_prepare_filter(k -> a spectrum in the workspace) followed by
 * fftconv_fwd on it, both enqueued on `stream` by this one call, so the
 * caller keeps no prepared filter; the results equal that pair of calls bit
 * for bit.
 *   k         (H, L_filter) device array of taps, same dtype as u, read only
 *   u, w, v, out, sparsity_mask  as in fftconv_fwd; w, v may be NULL
 *   workspace device scratch of fftconv_fwd_taps_workspace_bytes bytes,
 *             16-byte aligned, overlapping no argument; it holds the spectrum
 *             until the forward kernels have read it, so it must not be reused
 *             by another stream before this call's work completes
 * Errors as fftconv_prepare_filter and fftconv_fwd, plus
 * FFTCONV_ERR_WORKSPACE for a short workspace.  B = 0 or H = 0: nothing is
 * enqueued. */
fftconv_status_t fftconv_fwd_taps(const void *u, const void *k, const void *w, const void *v,
                                  void *out, int64_t B, int64_t H, int64_t N, int64_t L_filter,
                                  const uint8_t *sparsity_mask, fftconv_dtype_t dtype,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Device scratch bytes fftconv_bwd needs for this shape (0 for unsupported
 * N or dtype).  It holds room for a conjugated spectrum, u*w, the spectra of the
 * B*H sequences u*w, their correlations with v*dy, and the forward
 * workspace; at N = 1024 with fp16 or bf16 storage only the conjugated
 * spectrum (dk is accumulated on chip there); at N = 2048 .. 16384 with fp16
 * or bf16 storage the conjugated spectrum, the spectra of the batch-row pairs
 * of u*w with their scales, and one correlation row per pair and channel. */
size_t fftconv_bwd_workspace_bytes(int64_t B, int64_t H, int64_t N, fftconv_dtype_t dtype);

/* Backward pass of fftconv_fwd: the gradients of sum(dy * out) (the
 * convolutions are trained, FlashFFTConv summary page, "Key results"), with
 * x = u*w and g = v*dy:
 *   dv = dy * conv(x, k)                       (needs v; NULL = skip)
 *   du = w * corr(g, k),  dw = u * corr(g, k)  (dw needs w; NULL = skip)
 *   dk[h, s] = sum_b sum_t g[b,h,t] x[b,h,t-s], s < L_filter  (NULL = skip)
 * where corr(g, k)[t] = sum_s k[s] g[t+s] is the adjoint of the causal
 * convolution: the forward kernels run on the conjugated spectrum of K_f
 * (at N = 1024 .. 16384 in fp16 / bf16 with both du and dw asked for, one
 * kernel forms both and conjugates the bins as it reads K_f; otherwise a
 * conjugated copy is made in the workspace).  At N = 16384 in fp16 / bf16
 * with dv and dk asked for, dv comes from the same pass over u, w as the
 * spectra dk needs.  With a sparsity mask the gradients are those of the
 * masked forward pass.
 *   dy, u, w, v  (B, H, N) device arrays as in fftconv_fwd (w, v may be NULL)
 *   K_f          the spectrum fftconv_fwd used (same H, L_filter, N, dtype)
 *   du, dw, dv   (B, H, N) outputs; dk (H, L_filter) output, all in dtype
 *   workspace    at least fftconv_bwd_workspace_bytes(B, H, N, dtype) bytes
 * Asynchronous on stream; outputs must not overlap inputs. */
fftconv_status_t fftconv_bwd(const void *dy, const void *u, const void *K_f, const void *w, const void *v,
                             void *du, void *dk, void *dw, void *dv, int64_t B, int64_t H, int64_t N,
                             int64_t L_filter, const uint8_t *sparsity_mask, fftconv_dtype_t dtype,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- Chunked short-filter path (overlap-save) --------------------------
 * For a filter of at most 1024 taps (the FlashFFTConv summary page, table of
 * measured effects: filters shortened to 2K keep model quality) the
 * convolution needs no transform of the whole sequence.  The sequence is
 * covered by windows of 2048 samples overlapping by half (zeros before the
 * sequence start); each window's 2048-point circular convolution with the
 * filter runs on the matrix cores and keeps the second half of its outputs,
 * which no filter tap wraps around to.  The result is the same causal
 * convolution as fftconv_fwd with this filter.  fp16 and bf16 storage only;
 * no frequency mask (the spectrum is the 2048-point one of the filter).  Its
 * backward pass is fftconv_bwd_short. */

/* Bytes of a short-filter spectrum for H channels (0 for fp32 or H < 1). */
size_t fftconv_short_filter_bytes(int64_t H, fftconv_dtype_t dtype);

/* k (H, L_filter) device array, 1 <= L_filter <= 1024, fp16 or bf16 ->
 * K_s, K_s_bytes >= fftconv_short_filter_bytes(H, dtype).  Asynchronous. */
fftconv_status_t fftconv_prepare_short_filter(const void *k, int64_t H, int64_t L_filter,
                                              fftconv_dtype_t dtype, void *K_s, size_t K_s_bytes,
                                              hipStream_t stream);

/* out = v * causal_conv(u * w, k) with the prepared short filter K_s.
 *   u, w, v, out  (B, H, N) device arrays, N a positive multiple of 1024
 *                 (not necessarily a power of two); w, v may be NULL
 *   L_filter      the filter length K_s was prepared with (<= 1024)
 * Asynchronous on stream; no workspace; out must not overlap the inputs. */
fftconv_status_t fftconv_fwd_short(const void *u, const void *K_s, const void *w, const void *v,
                                   void *out, int64_t B, int64_t H, int64_t N, int64_t L_filter,
                                   fftconv_dtype_t dtype, hipStream_t stream);

/* Backward pass of fftconv_fwd_short (the convolutions are trained,
 * FlashFFTConv summary page, "Key results"): the gradients of sum(dy * out)
 * with x = u*w and g = v*dy,
 *   dv = dy * conv(x, k)                       (needs v; NULL = skip)
 *   du = w * corr(g, k),  dw = u * corr(g, k)  (dw needs w; NULL = skip)
 *   dk[h, s] = sum_b sum_t g[b,h,t+s] x[b,h,t], s < L_filter  (NULL = skip)
 * with corr(g, k)[t] = sum_s k[s] g[t+s] (zero past the sequence end), the
 * same quantities as fftconv_bwd.  dv runs the windowed forward kernel with
 * dy as the output gate; corr takes, for the outputs of block j, the window
 * of blocks j and j+1 and its 2048-point circular correlation with the
 * filter (the conjugated spectrum, first half of the outputs: no
 * wrap-around); dk accumulates, per channel on chip, the spectrum products
 * of those windows of g with the zero-padded blocks of x.
 *   dy, u, w, v   (B, H, N) device arrays, N a positive multiple of 1024;
 *                 w, v may be NULL (absent gates, as in the forward call)
 *   K_s           the short-filter spectrum of the forward call
 *   du, dw, dv    (B, H, N) outputs, dk (H, L_filter) output, all in dtype;
 *                 each may be NULL; none may overlap an input
 * No workspace.  B = 0: dk is set to zero, nothing else is written.
 * Asynchronous on stream. */
fftconv_status_t fftconv_bwd_short(const void *dy, const void *u, const void *K_s, const void *w,
                                   const void *v, void *du, void *dk, void *dw, void *dv, int64_t B,
                                   int64_t H, int64_t N, int64_t L_filter, fftconv_dtype_t dtype,
                                   hipStream_t stream);

/* ---- Group-axis circular convolution (Flash EQ-Linear) ------------------
 * The Flash EQ-Linear abstract page: an equivariant linear layer is a
 * circular convolution along the group dimension composed with a linear map
 * along the channels, computed through the Fourier convolution theorem along
 * the group axis with the real DFT's conjugate symmetry, in FP32 and in FP16
 * precision.  Here, for a cyclic group of order T:
 *   y[n, t, d] = sum_{s < T} sum_{c < C_in} W[s, d, c] x[n, (t - s) mod T, c]
 * x (N, T, C_in), W (T, C_out, C_in), y (N, T, C_out), contiguous, fp32, fp16
 * or bf16 storage; T in {4, 8, 16}; C_in and C_out positive multiples of 32.
 * The per-frequency channel products run on the matrix cores: fp32 operands
 * for fp32 storage, fp16 operands for fp16 and bf16 storage, fp32
 * accumulation throughout. */

/* Bytes of the transformed weights (T/2 + 1 complex matrices, fp32 for fp32
 * storage and fp16 otherwise); 0 when unsupported. */
size_t fftconv_eqlinear_weight_bytes(int64_t T, int64_t C_out, int64_t C_in, fftconv_dtype_t dtype);

/* W (T, C_out, C_in) device array -> W_f (W_f_bytes >= fftconv_eqlinear_weight_bytes).
 * Asynchronous on stream. */
fftconv_status_t fftconv_eqlinear_prepare(const void *W, int64_t T, int64_t C_out, int64_t C_in,
                                          fftconv_dtype_t dtype, void *W_f, size_t W_f_bytes,
                                          hipStream_t stream);

/* y = the group convolution of x with the prepared weights W_f (prepared for the
 * same dtype).  Asynchronous on stream; y must not overlap x or W_f. */
fftconv_status_t fftconv_eqlinear_fwd(const void *x, const void *W_f, void *y, int64_t N, int64_t T,
                                      int64_t C_in, int64_t C_out, fftconv_dtype_t dtype, hipStream_t stream);

/* ---- Decay attention -----------------------------------------------------
 * Linear attention with a decay for each head: the mixer that hybrid models
 * set beside the long convolution, and the one with a recurrent form for
 * single tokens.  With d_h = exp(log_decay[h]) and, per sequence and head, an
 * fp32 state S (Dk x Dv, row-major):
 *
 *     S_t = d S_{t-1} + k_t v_t^T,     out_t = scale * S_t^T q_t
 *
 * that is out_t = scale * sum_{j <= t} d^(t-j) (q_t . k_j) v_j, plus the carried
 * state's scale * d^(t+1) S_0^T q_t.  log_decay is an fp32 device array of H
 * values <= 0 (0: no decay, -inf: d = 0); it is a constant of the model, with no gradient.
 *
 * Heads: q and out have H heads, k and v have Hk, H a multiple of Hk; head h
 * uses k/v head h / (H / Hk).  Widths: 1 <= Dk, Dv <= 256.
 * Layouts: q (B, N, H, Dk), k (B, N, Hk, Dk), v (B, N, Hk, Dv), out (B, N, H, Dv).
 * `strides` gives (batch, token, head) in elements for each tensor in the
 * order of the arguments, NULL = dense; rows of Dk or Dv values are contiguous.
 * Results share no element with each other or an input; blocks of one buffer that repeat by a
 * common stride (dq, dk, dv as heads of a fused buffer) are told apart, others by their spans.
 * Pointers need the alignment of their elements only; rows at 16-byte aligned
 * addresses of whole 16-byte pieces are the fast case.
 * Packed sequences: with cu_seqlens (device int32, B + 1 ascending values from
 * 0 to the total) the tensors hold N tokens in all, (N, H, D), sequence b is
 * tokens cu_seqlens[b] .. cu_seqlens[b+1] - 1, and batch strides are ignored.
 * Bounds outside [0, N] are clamped; tokens of no sequence are not written.
 * Precision: products of fp16 / bf16 storage run on the matrix cores with fp32
 * accumulation; the products q k^T and the state are rounded to the storage
 * type where they meet v and q, and the state itself is kept and returned to
 * fp32 precision.  fp32 storage uses fp32 matrix instructions throughout.
 * Range: nothing is clamped; results beyond the storage type become infinite.  q k^T and the
 * states may be of any size that fp32 holds, in fp16 too: they are scaled by powers of two
 * where they are rounded (elements below 2^-12 of a state's largest may keep fewer bits there).
 * A NaN or infinity in a token may reach every output of its sequence and head from its
 * block of 32 tokens on (blocks are counted from the sequence's start, in dk and dv from
 * its end), never another sequence.
 * Refused with FFTCONV_ERR_UNSUPPORTED: token strides of 32 MiB or more, and
 * calls whose (sequence or segment, head) pairs pass 2^24. */

/* Device scratch bytes of fftconv_decay_fwd for T tokens in all (B * N, or N
 * when packed); 0 where none is needed or an argument is unsupported. */
size_t fftconv_decay_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype);

/* Prompt form over whole sequences.
 *   strides      int64[12] host array: q, k, v, out (or NULL)
 *   state_in     initial states, fp32 (B, H, Dk, Dv), or NULL (zero)
 *   state_out    receives the states after the last token, or NULL; may be state_in
 *   state_slots  NULL, or device int32 (B): state_in and state_out are pools
 *                (n_slots, H, Dk, Dv) and sequence b uses slot state_slots[b].
 *                A slot outside [0, n_slots) means no state: zero, and none kept.
 *                Slots of one call must differ.
 * An empty sequence passes its state on.  Asynchronous on stream; out and the
 * workspace must not overlap any argument. */
fftconv_status_t fftconv_decay_fwd(const void *q, const void *k, const void *v, const float *log_decay, void *out,
                                   const int64_t *strides, const float *state_in, float *state_out,
                                   const int32_t *state_slots, int64_t n_slots, const int32_t *cu_seqlens, int64_t B,
                                   int64_t N, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                   fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* One token of each of B sequences: q (B, H, Dk), k (B, Hk, Dk), v (B, Hk, Dv),
 * out (B, H, Dv); the states are updated in place.  strides: int64[8] host
 * array, (batch, head) of q, k, v, out, or NULL.  state and state_slots as
 * above; a row whose slot is outside [0, n_slots) gets zeros.  No workspace. */
fftconv_status_t fftconv_decay_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                                    void *out, const int64_t *strides, const int32_t *state_slots, int64_t n_slots,
                                    int64_t B, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                    fftconv_dtype_t dtype, hipStream_t stream);

/* As above, for fftconv_decay_bwd. */
size_t fftconv_decay_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype);

/* Gradients of sum(dout * out) + sum(dstate_out * state_out) of the prompt form:
 * with G_t = scale q_t dout_t^T + d G_{t+1} (dstate_out in place of d G behind the last token),
 *   dq_t = scale S_t dout_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   dstate_in = d G_0,
 * dk and dv summed over the heads that share a key/value head.  dq, dk, dv and
 * dstate_in may each be NULL (skipped); dstate_out NULL = zero.  States are
 * fp32 (B, H, Dk, Dv).  strides: int64[21], dout, q, k, v, dq, dk, dv, or NULL. */
fftconv_status_t fftconv_decay_bwd(const void *dout, const void *q, const void *k, const void *v,
                                   const float *log_decay, void *dq, void *dk, void *dv, const int64_t *strides,
                                   const float *state_in, const float *dstate_out, float *dstate_in,
                                   const int32_t *cu_seqlens, int64_t B, int64_t N, int64_t H, int64_t Hk, int64_t Dk,
                                   int64_t Dv, float scale, fftconv_dtype_t dtype, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* ---- Gated delta rule --------------------------------------------------------
 * Linear attention whose state forgets by a factor of each token and is corrected by what it got wrong,
 * beside decay attention.  With a_t = exp(log_decay_t), beta_t, and per sequence and head an fp32 state
 * S (Dk x Dv, row-major):
 *
 *     u_t = beta_t (v_t - a_t S_{t-1}^T k_t),    S_t = a_t S_{t-1} + k_t u_t^T,    out_t = scale * S_t^T q_t
 *
 * log_decay and beta are fp32 (B, N, H), dense: logarithms <= 0 (below -104, -inf among them: the state is cleared
 * before the token), and any weight.  The rule is stable while beta |k|^2 <= 2: keys are meant to be normed (fftconv_norm_fwd over
 * the heads' rows, weight 1 / sqrt(Dk)).
 * Heads: v, out, log_decay, beta and the states have H heads, q and k Hk, H a multiple of Hk; head h uses q/k
 * head h / (H / Hk).  Widths 1 <= Dk, Dv <= 256.
 * Layouts: q, k (B, N, Hk, Dk), v, out (B, N, H, Dv); `strides` (batch, token, head), alignment, separation of
 * results, packed sequences (cu_seqlens) and state pools (state_slots) as for decay attention; a call names a slot
 * at most once (of a slot that two sequences name, the state and those sequences' outputs are undefined).
 * Precision: operands are exact sums of bf16 terms and products are accumulated in fp32; the states, and
 * everything a state depends on, keep fp32 precision.  Outputs in 16 bits see the state, u and the products q k^T in
 * two bf16 terms each (2^-15 of a value).
 * A NaN or infinity in a token may reach every output of its sequence and head from its block of 64 tokens on,
 * never another sequence; one in a state that is passed in may reach all of them, unless the first token clears it.
 * Refused with FFTCONV_ERR_UNSUPPORTED: token strides of 16 MiB or more, and calls whose (64 tokens, head) pairs
 * pass 2^24 or whose (sequence, head) pairs pass 2^20. */

/* Device scratch bytes of fftconv_delta_fwd for T tokens in all (B * N, or N when packed); 0 where none is needed or
 * an argument is unsupported. */
size_t fftconv_delta_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype);

/* Prompt form over whole sequences; arguments as fftconv_decay_fwd, with beta.  strides: int64[12], q, k, v, out. */
fftconv_status_t fftconv_delta_fwd(const void *q, const void *k, const void *v, const float *log_decay, const float *beta,
                                   void *out, const int64_t *strides, const float *state_in, float *state_out,
                                   const int32_t *state_slots, int64_t n_slots, const int32_t *cu_seqlens, int64_t B,
                                   int64_t N, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                   fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* One token of each of B sequences: q, k (B, Hk, Dk), v, out (B, H, Dv), log_decay, beta (B, H); the states are
 * updated in place.  strides: int64[8] host array, (batch, head) of q, k, v, out, or NULL.  state and state_slots as
 * for fftconv_decay_step.  No workspace. */
fftconv_status_t fftconv_delta_step(const void *q, const void *k, const void *v, const float *log_decay,
                                    const float *beta, float *state, void *out, const int64_t *strides,
                                    const int32_t *state_slots, int64_t n_slots, int64_t B, int64_t H, int64_t Hk,
                                    int64_t Dk, int64_t Dv, float scale, fftconv_dtype_t dtype, hipStream_t stream);

/* As above, for fftconv_delta_bwd. */
size_t fftconv_delta_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype);

/* Gradients of sum(dout * out) + sum(dstate_out * state_out) of the prompt form.  dq, dk and dv are in the storage
 * type, dq and dk summed over the heads that share a q/k head; dlog_decay and dbeta are fp32 (B, N, H), dense.  All of
 * them and dstate_in may each be NULL (skipped); dstate_out NULL = zero.  States are fp32 (B, H, Dk, Dv).  The call
 * recomputes what it needs of the forward pass; its workspace holds the state and the state's gradient of every 64
 * tokens.  strides: int64[21], dout, q, k, v, dq, dk, dv, or NULL.  Results repeat bit by bit.
 * dlog_decay_t is the sum of q_i . dq_i - v_i . dv_i over the tokens i >= t of t's block of 64 and of <G, S> behind the
 * block (the state and its gradient), in fp32: its error is some 2^-20 of those terms, which do not shrink with the
 * decay, so that little is left of a gradient that a small a_t makes small.  It is 0 where the token clears the state. */
fftconv_status_t fftconv_delta_bwd(const void *dout, const void *q, const void *k, const void *v, const float *log_decay,
                                   const float *beta, void *dq, void *dk, void *dv, float *dlog_decay, float *dbeta,
                                   const int64_t *strides, const float *state_in, const float *dstate_out,
                                   float *dstate_in, const int32_t *cu_seqlens, int64_t B, int64_t N, int64_t H,
                                   int64_t Hk, int64_t Dk, int64_t Dv, float scale, fftconv_dtype_t dtype,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- Linear product ---------------------------------------------------------
 * The dense products around a mixer, with what follows them fused:
 *     pre = x W^T + bias,     out = act(pre) + residual
 * x (M, K), W (N, K), bias (N), residual, out, pre (M, N), one storage type,
 * fp32 accumulation, everything after the product in fp32, one rounding.
 * Activations and their slopes (each of the slope's two summands) have relative errors of at
 * most 2^-20 with fp32 storage (the tanh form: and 2^-22 for each unit of the exponential's
 * argument) and 2^-15 before the rounding with 16-bit storage.  Rows
 * are contiguous; `strides` gives the row strides in elements (NULL = dense).
 * Any sizes and element-aligned pointers; 16-byte aligned rows of whole 16-byte pieces are
 * the fast case.  Results repeat bit by bit.  Sizes are below 2^31, N at most 2^28 - 16; products of
 * more than 2^23 tiles (64 to 256 wide) are refused with FFTCONV_ERR_UNSUPPORTED. */
typedef enum {
    FFTCONV_ACT_NONE = 0,
    FFTCONV_ACT_RELU = 1,
    FFTCONV_ACT_GELU = 2,      /* z/2 (1 + erf(z / sqrt 2))                                  */
    FFTCONV_ACT_GELU_TANH = 3, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))              */
    FFTCONV_ACT_SILU = 4       /* z / (1 + exp(-z))                                          */
} fftconv_activation_t;

/* Device scratch bytes of fftconv_linear_fwd; 0 where none is needed or an argument is unsupported. */
size_t fftconv_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, fftconv_dtype_t dtype);

/* bias, residual and pre may be NULL; pre receives x W^T + bias for the
 * backward call.  out may be the residual itself (same pointer and stride), and
 * overlaps nothing else.  strides: int64[5], x, W, residual, out, pre. */
fftconv_status_t fftconv_linear_fwd(const void *x, const void *W, const void *bias, const void *residual, void *out,
                                    void *pre, const int64_t *strides, int64_t M, int64_t N, int64_t K,
                                    fftconv_activation_t activation, fftconv_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* As above, for fftconv_linear_bwd. */
size_t fftconv_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, fftconv_dtype_t dtype);

/* Gradients of sum(dout * out), with dz = dout * act'(pre):
 *     dx = dz W,   dW = dz^T x,   dbias = sum over rows of dz      (the residual's is dout)
 * each NULL = skipped.  pre may be NULL for FFTCONV_ACT_NONE; relu's slope at 0
 * is 0.  dz is rounded to the storage type where it meets W and x (in fp16, gradients below 2^-14
 * keep fewer bits there: scale the loss); dbias sums it unrounded.
 * strides: int64[6], dout, x, W, pre, dx, dW. */
fftconv_status_t fftconv_linear_bwd(const void *dout, const void *x, const void *W, const void *pre, void *dx, void *dW,
                                    void *dbias, const int64_t *strides, int64_t M, int64_t N, int64_t K,
                                    fftconv_activation_t activation, fftconv_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* ---- Root-mean-square norm ----------------------------------------------------
 * The norm before a mixer or MLP with the residual stream's addition, over rows of any width (also the
 * heads' own: queries and keys of the delta rule):
 *     t = x + residual,    y = t / sqrt(mean(t^2) + eps) * weight
 * x, residual, sum (M, G, D) rows of D values in (M, G) groups, weight (D) or NULL (ones), one storage
 * type, 1 <= D <= 2^20, M * G < 2^31.  Everything is fp32 (squares beyond fp32's range make the row 0);
 * `sum` receives t rounded once, out receives y, of the unrounded t.
 *   scales  NULL: out (M, G, D) holds y in the storage type.  Else fp32 (M, G): out holds 8 bits (e4m3,
 *           largest value 448) with y ~ scale * out, scale = max|y| / 448 of the row, at least 2^-126;
 *           a row with a NaN has the scale NaN.
 *   strides int64[8], (row, group) in elements of x, residual, out, sum, or NULL = dense; rows are contiguous.
 * residual and sum may be NULL; sum may be the residual or x itself (same pointer and strides), else no
 * result overlaps anything.  No workspace.  Asynchronous on stream. */
fftconv_status_t fftconv_norm_fwd(const void *x, const void *residual, const void *weight, void *out, void *sum,
                                  float *scales, const int64_t *strides, int64_t M, int64_t G, int64_t D, float eps,
                                  fftconv_dtype_t dtype, hipStream_t stream);

/* Device scratch bytes of fftconv_norm_bwd for `rows` = M * G; 0 where none is needed or an argument is unsupported. */
size_t fftconv_norm_bwd_workspace_bytes(int64_t rows, int64_t D);

/* Gradients of sum(dout * out) + sum(dsum * sum) with x the sum that the forward call normed (its x without a
 * residual): r = 1 / sqrt(mean(x^2) + eps), u = weight dout,
 *     dx = r (u - x r^2 mean(u x)) + dsum,    dweight = sum over rows of dout x r
 * dx is the gradient of x and of the residual alike.  weight, dsum, dx and dweight may be NULL; dx may be dsum
 * itself.  dweight is summed in fp32 in one order (results repeat bit by bit) and is zero without rows.
 * strides: int64[8], dout, x, dsum, dx, or NULL. */
fftconv_status_t fftconv_norm_bwd(const void *dout, const void *x, const void *weight, const void *dsum, void *dx,
                                  void *dweight, const int64_t *strides, int64_t M, int64_t G, int64_t D, float eps,
                                  fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Static text for a status code. */
const char *fftconv_status_string(fftconv_status_t status);

/* Detail of the calling thread's last non-OK status ("" if none). */
const char *fftconv_last_error(void);

/* Test helper, SYNCHRONOUS: decode K_f into natural-order rfft bins
 * K[h, f] = rfft(pad(k[h], 2N))[f], f in [0, N], as float64 (re, im) pairs in
 * host memory host_out[(H, N+1, 2)]. */
fftconv_status_t fftconv_export_filter_rfft(const void *K_f, int64_t H, int64_t N,
                                            fftconv_dtype_t dtype, double *host_out,
                                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FFTCONV_H */
