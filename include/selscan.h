/*
 * libselscan -- the selective state-space scan (Mamba's selective SSM) on AMD
 * Instinct MI355X (gfx950).  Plain C ABI: device pointers, sizes, a HIP stream.
 *
 * The operation (all passages are on the reference pages):
 *
 *   Delta[b,l,d] = softplus(delta[b,l,d] + delta_bias[d])
 *       velog.io Mamba review, section 3.2 "Improving SSMs with Selection":
 *       the step is a projection plus a learned parameter passed through softplus,
 *       with shape (B, L, D); A has shape (D, N); B and C have shape (B, L, N).
 *   Abar = exp(Delta A),  Bbar = (Delta A)^-1 (exp(Delta A) - I) Delta B
 *       velog.io review, section "2 State Space Models", "Discretization"
 *       (zero-order hold; A is diagonal, so both are elementwise per (d, n):
 *       Bbar[b,l,d,n] = (exp(Delta A[d,n]) - 1) / A[d,n] * B[b,l,n], and
 *       Delta * B[b,l,n] in the limit A[d,n] = 0).
 *   h_l = Abar_l h_{l-1} + Bbar_l x_l,   y_l = C_l . h_l + D x_l,   y_l *= silu(z_l)
 *       velog.io review, "Discretization" item 3 (state and output equations);
 *       skip term and gate: gh.r-mj.com Mamba_Model_Report.md, sections 3
 *       (MambaBlock.forward: y * silu(z)) and 4.2 (y = y + D * x).
 *   Single-token recurrent step on a carried state [B, D, N]:
 *       Mamba_Model_Report.md, section 6 (ssm_step).
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller, dense and
 *    row-major (last index fastest).  The library never frees or retains them.
 *  - Token tensors x, delta, z, y, and B, C use the element type `dtype`
 *    (SSCAN_F32 = float32, SSCAN_BF16 = bfloat16 stored as 16-bit words).
 *    A, D, delta_bias and every state tensor are float32.
 *  - Arithmetic is float32 in registers (state included); y is rounded to
 *    `dtype` with round-to-nearest-even.
 *  - Calls are asynchronous on `stream` (a hipStream_t; NULL is the null
 *    stream).  The library allocates no device memory and never synchronizes
 *    (sscan_fwd_noalloc's static scratch array comes with the loaded code object).
 *  - Errors: a nonzero sscan_status is returned and nothing is launched;
 *    sscan_last_error() gives a message (per calling thread).  Arguments are
 *    checked on the host before any launch.  Values are not checked: NaN and
 *    Inf propagate.  SSCAN_ERR_HIP reports a failed launch.
 *  - Outputs must not overlap inputs, except where stated (in-place state).
 *  - dstate (N) must be in [1, SSCAN_MAX_DSTATE]; seqlen at most SSCAN_MAX_SEQLEN.
 *  - `flags` selects variants of the method (SSCAN_FLAG_*); 0 is the method
 *    as defined above.
 * The gated linear recurrence and the 8-bit activations, and what stands around
 * the recurrence in a layer (norm, 8-bit products, convolution), at the end of this header
 * follow the same conventions, with shapes of their own and no flags.
 */
#ifndef SELSCAN_H
#define SELSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSCAN_VERSION 430
#define SSCAN_MAX_DSTATE 16
#define SSCAN_MAX_DCONV 4
/* Longest sequence sscan_fwd* and sscan_bwd* accept (2^30 steps): the kernels count
 * the steps of one sequence segment in 32-bit integers.  Longer ones are rejected
 * with SSCAN_ERR_INVALID_ARG. */
#define SSCAN_MAX_SEQLEN (1LL << 30)

/*
 * Bits of the `flags` argument.
 *
 * SSCAN_FLAG_EULER: discretize B with the first-order (Euler) rule
 *   Bbar = Delta * B   instead of the zero-order hold (Abar is exp(Delta A) either way).
 *   This is the rule the page-3 report's code uses (section 4.2,
 *   selective_scan / selective_scan_seq: deltaB = delta * B, BX = deltaB * x).
 * Unknown bits are rejected with SSCAN_ERR_UNSUPPORTED.
 */
#define SSCAN_FLAG_EULER 1u

/*
 * SSCAN_FLAG_STRUCTURED_A: the caller states that A is rank one, A[d, n] = c_d a_n --
 *   as the S4D-Real initialisation A = -(n + 1) of every channel (Mamba_Model_Report.md,
 *   section 3, MambaBlock: A = -exp(A_log) with A_log = log(1 .. N) for each channel).
 *   Then x B / A = (x / c_d)(B / a_n), and the forward stages x / c_d and B / a_n once
 *   per token instead of dividing per state.  A hint, never a change of the result:
 *   each channel tile checks the form exactly (c_d = A[d, 0], a_n = A[d0, n] / A[d0, 0]
 *   for the tile's first channel d0, and c_d a_n == A[d, n] with no rounding) and runs
 *   the plain form where it does not hold; results agree with the flag's absence to
 *   float32 rounding.  Used by sscan_fwd, sscan_fwd_segmented and sscan_fwd_noalloc with
 *   the zero-order hold when the launch takes the row layout (grids of at most one
 *   workgroup per compute unit); ignored otherwise and by the other entry points.
 */
#define SSCAN_FLAG_STRUCTURED_A 2u

typedef enum {
  SSCAN_OK = 0,
  SSCAN_ERR_INVALID_ARG = 1,  /* bad size, null required pointer, overlap, misalignment */
  SSCAN_ERR_UNSUPPORTED = 2,  /* dstate outside [1, SSCAN_MAX_DSTATE], unknown dtype   */
  SSCAN_ERR_HIP = 3           /* a HIP launch or runtime call failed                  */
} sscan_status;

typedef enum {
  SSCAN_F32 = 0,
  SSCAN_BF16 = 1
} sscan_dtype;

/* Library version (SSCAN_VERSION of the build). */
int sscan_version(void);

/* Message describing the last error returned to the calling thread ("" if none). */
const char* sscan_last_error(void);

/*
 * Workspace bytes that let sscan_fwd split long sequences into independently
 * scanned segments joined by a carry pass (a two-level scan over the sequence).
 * Returns 0 when the shape needs no split.  Pass at least this many bytes to
 * sscan_fwd to get the full split; fewer bytes give fewer segments (possibly
 * one), which is slower but equally correct.  The part of the workspace a call
 * uses must not overlap any tensor of that call (SSCAN_ERR_INVALID_ARG).
 */
size_t sscan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate,
                                int dtype);

/*
 * Forward selective scan over whole sequences.
 *
 *   x, delta, z, y : [batch, seqlen, dim]     (dtype)
 *   A              : [dim, dstate]            (float32; real, normally negative)
 *   B, C           : [batch, seqlen, dstate]  (dtype)
 *   D, delta_bias  : [dim]                    (float32)
 *   initial_state  : [batch, dim, dstate]     (float32)
 *   last_state     : [batch, dim, dstate]     (float32) state after the last step
 *
 * Optional (NULL allowed): D (no skip term), z (no gate), delta_bias (zero),
 * initial_state (zero state), last_state (not written), workspace (no split).
 * last_state may be the same buffer as initial_state.
 * Result: y[b,l,d] as defined at the top of this header.  With seqlen == 0,
 * last_state receives the initial state (zeros when absent).
 * Alignment: dtype-size alignment for token tensors, 4 bytes for float32 ones.
 */
sscan_status sscan_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                       unsigned int flags, const void* x, const void* delta, const float* A, const void* B, const void* C,
                       const float* D, const void* z, const float* delta_bias,
                       const float* initial_state, void* y, float* last_state,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes that give sscan_fwd_segmented the split it asks for: num_segments
 * after the same clamping the call applies (to whole 16-step chunks of seqlen and at
 * least one segment).  num_segments == 0 gives sscan_fwd_workspace_size.  Returns 0
 * when that plan has one segment, or for a negative num_segments or an invalid shape.
 */
size_t sscan_fwd_segmented_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate,
                                          int dtype, int64_t num_segments);

/*
 * Same as sscan_fwd, with the number of sequence segments chosen by the caller
 * (num_segments >= 1; it is clamped to what the workspace and seqlen allow).
 * num_segments == 0 means "choose automatically" and equals sscan_fwd.
 * For tuning and testing the two-level split; results agree with sscan_fwd
 * up to float32 rounding.
 */
sscan_status sscan_fwd_segmented(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                                 unsigned int flags, const void* x, const void* delta, const float* A, const void* B,
                                 const void* C, const float* D, const void* z, const float* delta_bias,
                                 const float* initial_state, void* y, float* last_state,
                                 void* workspace, size_t workspace_bytes, int64_t num_segments,
                                 void* stream);

/*
 * sscan_fwd for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Arguments, results
 * and errors are those of sscan_fwd without the workspace; the two-level split's
 * scratch (carries, segment end states, step sums) lives instead in a static device
 * array of SSCAN_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it runs
 * on until the process ends.  The call allocates nothing (no hipMalloc, no
 * allocating library routine).  It chooses the same split as sscan_fwd with a
 * workspace of sscan_fwd_workspace_size bytes, so its results equal that call's bit
 * for bit; a shape whose split needs more scratch than the array holds is rejected
 * with SSCAN_ERR_INVALID_ARG before anything runs.  Every call on one GPU shares
 * that GPU's array: calls that overlap in time on one GPU (other streams, other
 * threads) race on it and must be serialized by the caller.
 */
#define SSCAN_NOALLOC_SCRATCH_BYTES (32u << 20)
sscan_status sscan_fwd_noalloc(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                               unsigned int flags, const void* x, const void* delta, const float* A,
                               const void* B, const void* C, const float* D, const void* z,
                               const float* delta_bias, const float* initial_state, void* y,
                               float* last_state, void* stream);

/*
 * One recurrent step for a single token per batch row (decode).
 *
 *   state          : [batch, dim, dstate]  (float32) read, then overwritten in place
 *   x, delta, z, y : [batch, dim]          (dtype)
 *   A              : [dim, dstate]         (float32)
 *   B, C           : [batch, dstate]       (dtype)
 *   D, delta_bias  : [dim]                 (float32)
 *
 * Optional (NULL allowed): D, z, delta_bias.  Equivalent to sscan_fwd with
 * seqlen = 1, initial_state = last_state = state.
 */
sscan_status sscan_step(int64_t batch, int64_t dim, int64_t dstate, int dtype, unsigned int flags,
                        float* state, const void* x, const void* delta, const float* A,
                        const void* B, const void* C, const float* D, const void* z,
                        const float* delta_bias, void* y, void* stream);

/*
 * sscan_fwd with the short convolution that precedes the scan in a Mamba block,
 * fused into the scan's load: the page-3 report's MambaBlock.forward
 * (Mamba_Model_Report.md, section 3) passes the x branch through a causal depthwise
 * conv1d over time (kernel d_conv, padding d_conv - 1, output cropped to the first
 * L steps) and a SiLU before the selective scan:
 *   u[b,l,d] = silu(conv_b[d] + sum_{k<dconv} conv_w[d,k] * xx[b, l - (dconv-1) + k, d])
 * where xx is x preceded along time by conv_state_in (the dconv - 1 raw inputs
 * before the sequence, oldest first; zeros when NULL).  The scan, skip term and gate
 * then use u in place of x.  conv_state_out receives the last dconv - 1 raw inputs
 * (the cache that MambaBlock.step keeps, section 6), so a prefill hands over to
 * sscan_step_conv.
 *
 *   x              : [batch, seqlen, dim]    (dtype) raw inputs of the convolution
 *   conv_w         : [dim, dconv]            (float32) taps, conv_w[:, dconv-1] on the current input
 *   conv_b         : [dim]                   (float32) or NULL
 *   conv_state_in  : [batch, dim, dconv - 1] (float32) or NULL
 *   conv_state_out : [batch, dim, dconv - 1] (float32) or NULL; may be conv_state_in
 *   other arguments: as sscan_fwd.
 * 1 <= dconv <= SSCAN_MAX_DCONV (else SSCAN_ERR_UNSUPPORTED).  The backward pass does
 * not include the convolution: sscan_bwd differentiates the scan with respect to u.
 */
sscan_status sscan_fwd_conv(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int64_t dconv,
                            int dtype, unsigned int flags, const void* x, const float* conv_w,
                            const float* conv_b, const float* conv_state_in, float* conv_state_out,
                            const void* delta, const float* A, const void* B, const void* C,
                            const float* D, const void* z, const float* delta_bias,
                            const float* initial_state, void* y, float* last_state, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * sscan_step with the convolution prologue: the page-3 report's MambaBlock.step
 * (section 6) convolves the cached dconv - 1 raw inputs and the new one, applies
 * SiLU, runs the SSM step on the result, and updates the cache by dropping its
 * oldest entry and appending the new raw input.
 *
 *   conv_state : [batch, dim, dconv - 1] (float32) read, then updated in place
 *                (may be NULL only when dconv == 1)
 *   x          : [batch, dim] (dtype) raw input
 *   conv_w, conv_b, dconv: as sscan_fwd_conv; other arguments: as sscan_step.
 */
sscan_status sscan_step_conv(int64_t batch, int64_t dim, int64_t dstate, int64_t dconv, int dtype,
                             unsigned int flags, float* state, float* conv_state, const void* x,
                             const float* conv_w, const float* conv_b, const void* delta, const float* A,
                             const void* B, const void* C, const float* D, const void* z,
                             const float* delta_bias, void* y, void* stream);

/*
 * Workspace bytes sscan_bwd needs for a shape (0 for an empty problem).  The
 * backward pass cannot run without it: it holds the state checkpoints (one per
 * 8 timesteps), per-channel-tile partial sums of dB and dC, per-batch-row
 * partial sums of dA, dD and ddelta_bias, and the sequence-split buffers of the
 * checkpoint pass.  Contents are scratch: nothing is kept between calls.
 */
size_t sscan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate,
                                int dtype);

/*
 * Backward pass of sscan_fwd: gradients of a scalar loss with respect to every
 * input, given dy = dLoss/dy and, optionally, dlast_state = dLoss/d(last_state).
 *
 * The gradients are the chain rule through the forward definition at the top of
 * this header, run backwards in time: the reverse recurrence
 *   g_l = gyo_l C_l + Abar_{l+1} g_{l+1},   gyo_l = dy_l silu(z_l)   (elementwise in N)
 * that the page-3 report's PScan.backward computes with its reverse scan
 * pscan_rev (Mamba_Model_Report.md, section 4.1), with the forward states
 * recomputed rather than stored (the recomputation that the lengnian.github.io
 * notes, "Part3: Mamba - A Selective SSM", list in the hardware-aware algorithm).
 * Gradients then follow per step (phi = Bbar / B):
 *   dx = gyo D + sum_n g phi B        dB = sum_d g phi x        dC = sum_d gyo h
 *   dz = dy (C.h + D x) silu'(z)      dD = sum_{b,l} gyo x
 *   ddelta = sigmoid(delta + delta_bias) sum_n g (A Abar h_{l-1} + dphi/dDelta B x)
 *   dA = sum_{b,l} g (Delta Abar h_{l-1} + dphi/dA B x),  ddelta_bias = sum_{b,l} ddelta
 *   dinitial_state = Abar_0 g_0
 * (zero-order hold: phi = (Abar - 1)/A, dphi/dDelta = Abar, dphi/dA = (Delta Abar - phi)/A,
 * Delta^2/2 at A = 0; SSCAN_FLAG_EULER: phi = Delta, dphi/dDelta = 1, dphi/dA = 0).
 *
 *   inputs  : as sscan_fwd (x, delta, A, B, C, D, z, delta_bias, initial_state, flags)
 *   dy      : [batch, seqlen, dim]    (dtype)
 *   dlast_state : [batch, dim, dstate] (float32), NULL = zero
 *   dx, ddelta, dz : [batch, seqlen, dim]    (dtype)
 *   dB, dC         : [batch, seqlen, dstate] (dtype)
 *   dA             : [dim, dstate]           (float32)
 *   dD, ddelta_bias: [dim]                   (float32)
 *   dinitial_state : [batch, dim, dstate]    (float32)
 *
 * Required: x, delta, A, B, C, dy, dx, ddelta, dA, dB, dC and the workspace
 * (at least sscan_bwd_workspace_size bytes, 256-byte aligned).  dz is required
 * exactly when z is given; dD may be given only with D; ddelta_bias and
 * dinitial_state are optional whether or not delta_bias / initial_state are
 * (they are then the gradients at a zero bias / zero initial state).
 * Outputs must not overlap inputs, each other or the workspace.  Reductions run
 * in a fixed order: results are bitwise reproducible.
 */
sscan_status sscan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                       unsigned int flags, const void* x, const void* delta, const float* A, const void* B,
                       const void* C, const float* D, const void* z, const float* delta_bias,
                       const float* initial_state, const void* dy, const float* dlast_state, void* dx,
                       void* ddelta, float* dA, void* dB, void* dC, float* dD, void* dz,
                       float* ddelta_bias, float* dinitial_state, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Saved checkpoints for a training step.  The lengnian.github.io notes ("Part3:
 * Mamba - A Selective SSM") list recomputation among the means by which the
 * hardware-aware algorithm keeps intermediate results small; sscan_bwd recomputes
 * the forward states from scratch.  A training step that runs the forward anyway
 * can instead keep the state at a coarse grain: sscan_fwd_checkpointed writes the
 * state entering every block of 8 timesteps (1/8 of the four-dimensional state,
 * nothing in between), and sscan_bwd_checkpointed starts its reverse pass from
 * those states instead of running the forward recurrence again.
 *
 * Layout: checkpoints[b][j][n][d], float32, j = 0 .. ceil(seqlen / 8) - 1, holding
 * h_{8j-1}, the state entering timestep 8j (the initial state for j = 0).
 */

/* Bytes of the checkpoint array for a shape (0 for an empty problem). */
size_t sscan_checkpoint_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate);

/*
 * sscan_fwd that also writes the checkpoints.
 *   checkpoints      : written; at least sscan_checkpoint_bytes bytes, 4-byte aligned,
 *                      overlapping no other tensor or the workspace
 *   checkpoint_bytes : its size in bytes
 * Other arguments, results and errors: as sscan_fwd (there is no convolution
 * prologue here: the backward pass does not cover it).  y and last_state equal
 * sscan_fwd's bit for bit.
 */
sscan_status sscan_fwd_checkpointed(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                                    unsigned int flags, const void* x, const void* delta, const float* A,
                                    const void* B, const void* C, const float* D, const void* z,
                                    const float* delta_bias, const float* initial_state, void* y,
                                    float* last_state, void* workspace, size_t workspace_bytes,
                                    float* checkpoints, size_t checkpoint_bytes, void* stream);

/* Workspace bytes sscan_bwd_checkpointed needs: sscan_bwd's less the checkpoint array. */
size_t sscan_bwd_checkpointed_workspace_size(int64_t batch, int64_t seqlen, int64_t dim,
                                             int64_t dstate, int dtype);

/*
 * sscan_bwd from checkpoints that sscan_fwd_checkpointed wrote for the same x,
 * delta, A, B, C, delta_bias, initial_state and flags.  The initial state reaches
 * the backward pass through checkpoint block 0, so it is not an argument here;
 * dinitial_state is still produced.
 *   checkpoints      : read; at least sscan_checkpoint_bytes bytes, 4-byte aligned
 *   workspace        : at least sscan_bwd_checkpointed_workspace_size bytes
 * Other arguments, results and errors: as sscan_bwd.  The gradients equal
 * sscan_bwd's to rounding: sscan_bwd's own recomputation may split the sequence
 * differently from the forward, which rounds the states differently.
 */
sscan_status sscan_bwd_checkpointed(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                                    unsigned int flags, const void* x, const void* delta, const float* A,
                                    const void* B, const void* C, const float* D, const void* z,
                                    const float* delta_bias, const float* checkpoints,
                                    size_t checkpoint_bytes, const void* dy, const float* dlast_state,
                                    void* dx, void* ddelta, float* dA, void* dB, void* dC, float* dD,
                                    void* dz, float* ddelta_bias, float* dinitial_state, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * The gated linear recurrence: one state per channel whose decay is a gate of the
 * token, in place of the selective scan's step size and fixed A.  For channel d:
 *
 *   rho_t  = sigmoid(r_t + r_bias[d])      iota_t = sigmoid(i_t + i_bias[d])
 *   a_t    = exp(-decay_scale softplus(lam[d]) rho_t)
 *   h_t    = a_t h_{t-1} + sqrt(1 - a_t^2) (iota_t x_t)
 *   y_t    = h_t, or h_t silu(z_t) with a gate z
 *
 * r and i are the pre-activations of the two gates (projections of the token), lam a
 * parameter per channel, decay_scale > 0 a constant of the model.  The square root
 * keeps the state at the size of the input whatever the decay; 1 - a^2 is formed
 * without cancellation for decays near 1.
 *
 * Shapes.  Dense: x, r, i, z, y are [batch, seqlen, dim], every batch row a sequence.
 * Packed (offsets given): batch is 1, and request s holds the tokens offsets[s] ..
 * offsets[s + 1] - 1 of the seqlen tokens.  offsets is a device array of num_seqs + 1
 * int32, non-decreasing, starting at 0 and ending at most at seqlen; equal neighbours
 * are an empty request, whose last state is its initial one.  Tokens at or past
 * offsets[num_seqs] are padding: y is zero there, and so are their gradients,
 * whatever the inputs hold.  No state passes from one request to the next, infinities
 * and NaN included (activations kept in 8 bits share groups, see there).  The host does not read offsets; an array that breaks these rules
 * gives unspecified results, with no access outside the tensors.  "Sequences" below
 * are the batch rows, or the num_seqs requests.
 *
 * strides: host array of 4 token strides of x, r, i, z in elements (each at least
 * dim), so that the inputs can be columns of one projection's output: token t of
 * batch row b is at (b seqlen + t) stride.  NULL: all dense.  y and dy are dense.
 *
 * Limits: seqlen at most SSCAN_MAX_SEQLEN, dim at most 2^28, and batch ceil(seqlen / 64)
 * ceil(dim / 64) below 2^31 (for one token: seqlen 1).
 */

/* Tokens between the saved states of sscan_glr_fwd's checkpoints. */
#define SSCAN_GLR_BLOCK 64

/*
 * Activations in 8 bits.  Every channel's 16 consecutive tokens of a batch row (the
 * last group of a row may be shorter) share one power of two 2^e, e = floor(log2 max|v|)
 * held as e + 127 in a byte (the exponent field of the largest magnitude), and each
 * value is held as the whole number nearest to v 2^(6 - e) (ties to even), at most 127
 * in magnitude: the error is at most 2^(e - 7), except for magnitudes within
 * 2^(e - 7) of 2^(e + 1), where it is below 2^(e - 6).  Magnitudes below 2^-126 share
 * e = -126.  A group with an infinity or NaN has the byte 255 and comes back as NaN.
 *
 * Groups are cut by position, tokens 16 k .. 16 k + 15, whatever packed requests they
 * belong to.  Two requests that meet inside a group share its power of two: beside large
 * values of one the other's are held with less relative precision, and an infinity or NaN
 * of one turns the other's tokens in the group to NaN, and in a backward pass from 8 bits
 * their gradients and those that depend on them.  Requests that start at multiples of 16
 * share nothing.  (The forward's outputs do not come from the 8 bits.)
 *
 * One packed tensor [batch, seqlen, dim] is sscan_act8_bytes bytes: the codes (int8)
 * [batch][seqlen][dim], then, from the next multiple of 256 bytes, the exponent bytes
 * [batch][ceil(seqlen / 16)][dim]; the total is a multiple of 256.
 */
#define SSCAN_ACT8_GROUP 16

/* Bytes of one packed tensor (0 for an empty one, and for invalid sizes). */
size_t sscan_act8_bytes(int64_t batch, int64_t seqlen, int64_t dim);

/*
 * Pack x [batch, seqlen, dim] (dtype, token stride x_stride in elements, at least dim,
 * 0 for dense) into `packed`, and back into a dense x.  The values that come back are
 * rounded to dtype (bfloat16 holds every packed value exactly).  packed must be
 * 256-byte aligned, of packed_bytes >= sscan_act8_bytes, and overlap no tensor.
 * batch ceil(seqlen / 16) dim is at most 2^39 - 257.
 */
sscan_status sscan_act8_pack(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x,
                             int64_t x_stride, void* packed, size_t packed_bytes, void* stream);
sscan_status sscan_act8_unpack(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* packed,
                               size_t packed_bytes, void* x, void* stream);

/* Bytes of the state checkpoints (float32, [batch][ceil(seqlen / SSCAN_GLR_BLOCK)][dim]:
 * the state entering each block of tokens) and of the activations saved in 8 bits
 * (x, r, i and, if gated, z, each as one packed tensor of sscan_act8_bytes, in this order). */
size_t sscan_glr_checkpoint_bytes(int64_t batch, int64_t seqlen, int64_t dim);
size_t sscan_glr_saved_bytes(int64_t batch, int64_t seqlen, int64_t dim, int gated);

/* Workspace bytes of sscan_glr_fwd (0: none needed) and of sscan_glr_bwd. */
size_t sscan_glr_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim);
size_t sscan_glr_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim);

/*
 * Forward over whole sequences.
 *
 *   x, r, i, z     : as above (dtype); z NULL: no gate
 *   lam, r_bias, i_bias : [dim] (float32); a NULL bias is zero
 *   initial_state  : [sequences, dim] (float32), NULL: zero
 *   y              : [batch, seqlen, dim] (dtype)
 *   last_state     : [sequences, dim] (float32), NULL: not written; may be initial_state
 *   checkpoints    : for a backward pass: sscan_glr_checkpoint_bytes, NULL: not written
 *   saved          : for a backward pass from 8 bits: sscan_glr_saved_bytes, 256-byte
 *                    aligned, NULL: not written
 *   workspace      : sscan_glr_fwd_workspace_size, 256-byte aligned; scratch, nothing is
 *                    kept in it between calls
 * Results are bitwise reproducible.
 */
sscan_status sscan_glr_fwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r,
                           const void* i, const void* z, const int64_t* strides, const float* lam,
                           const float* r_bias, const float* i_bias, float decay_scale,
                           const float* initial_state, const int32_t* offsets, int64_t num_seqs, void* y,
                           float* last_state, float* checkpoints, size_t checkpoint_bytes, void* saved,
                           size_t saved_bytes, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass, given dy = dLoss/dy and optionally dlast_state = dLoss/d(last_state):
 * with the reverse recurrence g_t = dy_t silu(z_t) + a_{t+1} g_{t+1} within a sequence,
 *   dlog_a = g (a h_{t-1} - iota x a^2 / sqrt(1 - a^2))
 *   dx = g sqrt(1 - a^2) iota             di = g sqrt(1 - a^2) x iota (1 - iota)
 *   dr = -decay_scale softplus(lam) dlog_a rho (1 - rho)
 *   dz = dy h silu'(z)                    dinitial_state = a g of the first token
 *   dlam = -decay_scale sigmoid(lam) sum dlog_a rho     (bias gradients: sums of dr and di)
 * These hold also where a rounds to 1, since 1 - a^2 comes from the decay rate itself.
 * Only the square root stays at 1e-18 or above, for its reciprocal: where 1 - a^2 is less
 * than 1e-36 the terms with it vanish with the rate (and iota x up to 1e20 overflows in
 * none).
 *
 *   checkpoints    : what sscan_glr_fwd wrote for the same inputs (required)
 *   x, r, i, z     : the forward's inputs, or all NULL with `saved`, what the forward
 *                    wrote there; dz then says whether it was gated.  From `saved`,
 *                    every gradient is the formula's at the values the 8 bits stand
 *                    for, except that the states entering the blocks are the
 *                    forward's own (those of the inputs as they were).
 *   initial_state  : the forward's (read only with offsets; a dense forward's comes
 *                    with the checkpoints), NULL: zero
 *   dx, dr, di, dz : (dtype) token strides in grad_strides (host array of 4, NULL:
 *                    dense); dz is required exactly when z is given
 *   dlam, dr_bias, di_bias : [dim] (float32); the bias gradients may be NULL
 *   dinitial_state : [sequences, dim] (float32), NULL: not written; an empty
 *                    request's is its dlast_state
 *   workspace      : sscan_glr_bwd_workspace_size, 256-byte aligned
 * The remaining arguments as in sscan_glr_fwd.  Results are bitwise reproducible.
 */
sscan_status sscan_glr_bwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r,
                           const void* i, const void* z, const int64_t* strides, const void* saved,
                           size_t saved_bytes, const float* lam, const float* r_bias, const float* i_bias,
                           float decay_scale, const float* initial_state, const int32_t* offsets, int64_t num_seqs,
                           const float* checkpoints, size_t checkpoint_bytes, const void* dy,
                           const float* dlast_state, void* dx, void* dr, void* di, void* dz,
                           const int64_t* grad_strides, float* dlam, float* dr_bias, float* di_bias,
                           float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for every row of a decode batch.
 *
 *   state          : [num_slots, dim] (float32), a pool of request states
 *   slots          : device array [batch] of int32: row b continues state slots[b]; a row
 *                    whose slot is outside [0, num_slots) holds no request: its y is zero
 *                    and no state changes.  NULL: row b has slot b (batch <= num_slots).
 *   slots_out      : device array [batch] of int32: where row b's new state goes (nowhere
 *                    if outside [0, num_slots)); NULL: back to its own slot.  With other
 *                    slots a state can be continued more than one way, or a drafted
 *                    token taken back.  No two rows may write one slot, and no row may
 *                    read a slot that another writes.
 *   x, r, i, z     : [batch, dim] (dtype), strides as above; y [batch, dim] dense
 */
sscan_status sscan_glr_step(int64_t batch, int64_t dim, int dtype, float* state, int64_t num_slots,
                            const int32_t* slots, const int32_t* slots_out, const void* x, const void* r,
                            const void* i, const void* z, const int64_t* strides, const float* lam,
                            const float* r_bias, const float* i_bias, float decay_scale, void* y, void* stream);

/*
 * What stands around the recurrence in a layer: the norm with the residual's addition,
 * projections in 8-bit integers, and the short convolution for packed requests and with
 * its backward pass.  Conventions as above; "rows" are tokens (batch * seqlen of them, or
 * a decode batch), and a row stride is in elements, 0 for dense.
 */

/* From here on a tensor with a row stride extends from its first byte to its last: outputs and
 * inputs that are different columns of one tensor count as overlapping.
 *
 * Channels of a row that sscan_rms_fwd, sscan_rms_bwd and sscan_i8_quant accept. */
#define SSCAN_RMS_MAX_DIM 32768

/*
 * Root-mean-square norm with the residual's addition.  For each row:
 *
 *   s = x + residual, rounded to residual_dtype (what is kept, and what is normed)
 *   r = 1 / sqrt(mean(s^2) + eps)          y = s r weight
 *
 *   x            : [rows, dim] (dtype), row stride x_stride
 *   residual     : [rows, dim] (residual_dtype), NULL: s = x rounded to residual_dtype
 *   weight       : [dim] (float32), NULL: ones
 *   y            : [rows, dim] (dtype), NULL: not written
 *   residual_out : [rows, dim] (residual_dtype), s, NULL: not written; may be residual (and
 *                  x too, if x is that tensor, dense and of its type); apart from all else
 *   codes, scales: y in 8 bits as sscan_i8_quant gives it (from y before its rounding to
 *                  dtype), both or neither; codes has the row stride codes_stride
 *                  (with dim == 0 nothing is written: sscan_i8_quant has those rows' scales)
 * residual_dtype is SSCAN_F32, or dtype.  eps is at least 0 and finite.  Sums are float32:
 * a row whose sum of squares passes float32's range has r = 0, and one whose mean(s^2) + eps
 * is below its normal numbers (2^-126; never with eps of that size) has r infinite.
 */
sscan_status sscan_rms_fwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* x, int64_t x_stride,
                           const void* residual, const float* weight, float eps, void* y, void* residual_out,
                           int8_t* codes, int64_t codes_stride, float* scales, void* stream);

/* Workspace bytes of sscan_rms_bwd; no less for more rows or channels. */
size_t sscan_rms_bwd_workspace_size(int64_t rows, int64_t dim);

/*
 * Backward pass of sscan_rms_fwd, given dy = dLoss/dy and, optionally, dresidual_out =
 * dLoss/ds from the layers that follow.  With g = dy weight:
 *
 *   ds = dresidual_out + r g - s r^3 mean(g s)        dweight = sum over rows of dy s r
 *
 * ds is the gradient of x and of the residual alike (the rounding of s passes it on).
 *
 *   s             : [rows, dim] (residual_dtype), what the forward kept (x itself, of type
 *                   residual_dtype, if there was no residual), row stride s_stride
 *   dy            : [rows, dim] (dtype)
 *   dresidual_out : [rows, dim] (residual_dtype), NULL: zero
 *   dx            : [rows, dim] (dtype), row stride dx_stride, NULL: not written
 *   dresidual     : [rows, dim] (residual_dtype), NULL: not written; may be dresidual_out (and
 *                   s or dy too, if dense and of its type); apart from all else
 *   dweight       : [dim] (float32), NULL: not written
 *   workspace     : sscan_rms_bwd_workspace_size, 256-byte aligned (needed for dweight)
 * Results are bitwise reproducible.
 */
sscan_status sscan_rms_bwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* s, int64_t s_stride,
                           const float* weight, float eps, const void* dy, const void* dresidual_out, void* dx,
                           int64_t dx_stride, void* dresidual, float* dweight, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Rows in 8-bit integers with a float32 scale for each:
 *
 *   scale = max(max |x| / 127, 2^-126)     code = the whole number nearest to x / scale
 *
 * (the quotient of the real numbers, ties to even; at most 127 in magnitude).  A row with
 * an infinity or NaN has the scale NaN and codes 0, so it comes out of a product as NaN.
 * A row without channels (dim == 0; x and codes may be NULL) has the scale 2^-126.
 * Weights are brought into this form once, each output's row by itself; activations at each
 * call, or by sscan_rms_fwd.
 *
 *   x      : [rows, dim] (dtype), row stride x_stride
 *   codes  : [rows, dim] (int8), row stride codes_stride; bytes between rows are not written
 *   scales : [rows] (float32)
 */
sscan_status sscan_i8_quant(int64_t rows, int64_t dim, int dtype, const void* x, int64_t x_stride, int8_t* codes,
                            int64_t codes_stride, float* scales, void* stream);

/* Products of a row that sscan_i8_matmul sums: any codes (-128 included) stay inside 32 bits. */
#define SSCAN_I8_MAX_K 131071

/*
 * Product of rows in 8-bit integers, with the scales of both sides:
 *
 *   out[i, j] = (sum_l a[i, l] b[j, l]) * (a_scales[i] * b_scales[j]) + bias[j]
 *
 * The sums are whole numbers of 32 bits, exact in any order; the rest is float32, rounded
 * once to dtype at the end.
 *
 *   a, a_scales : [m, k] (int8), row stride a_stride; [m] (float32)
 *   b, b_scales : [n, k] (int8), row stride b_stride; [n] (float32)
 *   bias        : [n] (float32), NULL: zero
 *   out         : [m, n] (dtype), row stride out_stride
 * Any strides and alignment work; rows at multiples of 16 bytes with k a multiple of 128 are
 * read fastest.  k is at most SSCAN_I8_MAX_K, m and n at most 2^31 - 1, and ceil(m / 16) ceil(n / 16)
 * at most 2^31 - 1 as well.  With k == 0 the sums are zero.
 */
sscan_status sscan_i8_matmul(int64_t m, int64_t n, int64_t k, const int8_t* a, int64_t a_stride,
                             const float* a_scales, const int8_t* b, int64_t b_stride, const float* b_scales,
                             const float* bias, int dtype, void* out, int64_t out_stride, void* stream);

/*
 * Depthwise causal convolution over time, the prologue of sscan_fwd_conv as an operator of
 * its own: in front of either recurrence, for packed requests, and with a backward pass.
 *
 *   v[t] = conv_b + sum_{k < dconv} conv_w[k] xx[t - (dconv - 1) + k]
 *   y[t] = v[t], or silu(v[t]) with silu != 0
 *
 * where xx is the sequence's x with initial_state (its dconv - 1 raw inputs before, oldest
 * first; zeros when NULL) in front.  Dense batches or packed requests, offsets and padding
 * as in sscan_glr_fwd; no value passes from one request to the next.
 *
 *   x              : [batch, seqlen, dim] (dtype), token stride x_stride (0: dense)
 *   conv_w, conv_b : [dim, dconv], [dim] (float32); conv_b NULL: zero
 *   initial_state  : [sequences, dim, dconv - 1] (float32), NULL: zeros
 *   y              : [batch, seqlen, dim] (dtype)
 *   last_state     : [sequences, dim, dconv - 1] (float32): the last dconv - 1 raw inputs
 *                    (of the initial state where the sequence is shorter), NULL: not
 *                    written; apart from initial_state
 * 1 <= dconv <= SSCAN_MAX_DCONV (else SSCAN_ERR_UNSUPPORTED).  Limits as sscan_glr_fwd's.
 */
sscan_status sscan_dwconv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu,
                              const void* x, int64_t x_stride, const float* conv_w, const float* conv_b,
                              const float* initial_state, const int32_t* offsets, int64_t num_seqs, void* y,
                              float* last_state, void* stream);

/* Workspace bytes of sscan_dwconv_bwd; no less when any of the sizes grows. */
size_t sscan_dwconv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv);

/*
 * Backward pass, given dy and optionally dlast_state = dLoss/d(last_state).  With
 * dv = dy, or dy silu'(v), and within each sequence:
 *
 *   dx[u] = sum_k conv_w[k] dv[u + (dconv - 1) - k]   (+ dlast_state of the tokens it holds)
 *   dconv_w[k] = sum_t dv[t] xx[t - (dconv - 1) + k]     dconv_b = sum_t dv[t]
 *   dinitial_state: the same as dx, of the tokens before the sequence
 *
 *   x, conv_w, conv_b, initial_state, offsets, silu: the forward's
 *   dy             : [batch, seqlen, dim] (dtype)
 *   dx             : [batch, seqlen, dim] (dtype), token stride dx_stride (0: dense)
 *   dconv_w        : [dim, dconv] (float32), dconv_b [dim] (NULL: not written)
 *   dinitial_state : [sequences, dim, dconv - 1] (float32), NULL: not written
 *   workspace      : sscan_dwconv_bwd_workspace_size, 256-byte aligned
 * Padding has zero gradients whatever the inputs hold there.  Results are bitwise
 * reproducible.
 */
sscan_status sscan_dwconv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu,
                              const void* x, int64_t x_stride, const float* conv_w, const float* conv_b,
                              const float* initial_state, const int32_t* offsets, int64_t num_seqs, const void* dy,
                              const float* dlast_state, void* dx, int64_t dx_stride, float* dconv_w, float* dconv_b,
                              float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for every row of a decode batch, against a pool of states:
 *
 *   state            : [num_slots, dim, dconv - 1] (float32; may be NULL when dconv == 1)
 *   slots, slots_out : as in sscan_glr_step
 *   x, y             : [batch, dim] (dtype), x with the row stride x_stride
 */
sscan_status sscan_dwconv_step(int64_t batch, int64_t dim, int64_t dconv, int dtype, int silu, float* state,
                               int64_t num_slots, const int32_t* slots, const int32_t* slots_out, const void* x,
                               int64_t x_stride, const float* conv_w, const float* conv_b, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_H */
