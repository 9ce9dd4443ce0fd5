/*
 * qmixer.h -- C ABI of the operators around the recurrent state (sm_100a).
 * Library: bit_recurrent_state_decode_b200/libqmixer.so.
 *
 * qstate.h steps a low-bit recurrent state by one token.  A Mamba2 layer needs
 * more around that step, and this file has it: the short causal convolution
 * and the selective scan of a prompt, both for single tokens too, the
 * handover of a prompt's float32 state into the low-bit object, the operands
 * of qstate_step from the layer's own quantities, and the root-mean-square
 * norm in front of and behind the mixer.
 *
 * ARITHMETIC.  All sums, norms, decays and states are binary32; inputs and
 * outputs are binary32 or bfloat16 (`dtype`), rounded once, at the end.
 *   time step  dt = softplus(raw + dt_bias) with QMIXER_SOFTPLUS, else
 *              raw + dt_bias (dt_bias may be NULL: 0)
 *   decay      a = exp(dt A)
 *   scan       S <- a S + dt B x^T,  y = S^T C + D x   (D may be NULL: 0)
 *   conv       z_t = bias + sum_k weight[k] x_{t-W+1+k};  y = z / (1 + e^-z)
 *              with QMIXER_SILU, else z   (bias may be NULL: 0)
 *   norm       h = x + residual, x silu(gate) or x;
 *              y = h / sqrt(mean(h^2) + eps) * weight
 * The prompt scan of bfloat16 inputs forms its matrix products over chunks of
 * 128 tokens on the tensor cores, with binary32 sums.  Its states keep 24 bits.
 * For y alone it rounds two factors to bfloat16: (C B^T) decays dt, and the copy
 * of S that C multiplies.  Each is off by at most 2^-8 of a term of y, so y by
 * 2^-7 of the sum of its terms' magnitudes, beside its own rounding: 0.0018 to
 * 0.0020 in the 2-norm where the rounding of y alone gives 0.0017.  C B^T, dt x
 * and the products of up to 128 decays are formed by themselves there, and in
 * either form of a long prompt the products of a whole segment's decays: these
 * have to stay inside binary32 (products of decays of at most 1 do).  In the
 * form for bfloat16 a token whose x is not a finite number makes its column of y
 * and of the state NaN from its own row on, where the binary32 form may keep an
 * infinity; no other column and no earlier token depends on it in either.
 *
 * SEQUENCES.  The token axis of the prompt calls holds `sequences` sequences
 * one behind the other.  seq_starts (device, int32 [sequences + 1], ascending,
 * seq_starts[0] >= 0) gives the first token of each and the end of the last;
 * tokens behind the last sequence are neither read nor written.  NULL: equal
 * sequences of tokens / sequences each.  A sequence may be empty.  Values
 * outside [0, tokens] are taken as the nearest bound; with a descending pair
 * the sequences concerned have no defined result, and nothing outside the
 * given buffers is touched.
 * With QMIXER_INITIAL a sequence continues from its row of `state`, else from
 * zeros; its row receives the state behind its last token (of an empty
 * sequence: what it started from).
 *
 * LAYOUTS (row-major device memory; a stride counts elements from one token's
 * row to the next; inside a row the elements are contiguous)
 *   conv    x, y [tokens][channels], weight [channels][width],
 *           bias [channels], state [sequences][width - 1][channels], oldest
 *           token first
 *   scan    x, y [tokens][heads][d_v], dt [tokens][heads], A, D, dt_bias
 *           [heads] binary32, B, C [tokens][groups][d_k] (head h reads group
 *           h / (heads / groups)), state [sequences][heads][d_k][d_v]
 *           binary32 -- the tile layout of qstate_dequant
 *   norm    x, other, y [rows][columns], weight [columns], scales
 *           [rows][columns / group] binary32 ([rows] for group 0)
 * Outputs must not overlap inputs, other than the state and the residual,
 * which are updated in place.  The state of scan and scan_step and the
 * buffers of quantize start on 16-byte boundaries, as do x, B and C of the
 * scans, whose strides are multiples of 16 bytes (QMIXER_EINVAL otherwise);
 * conv and norm take any alignment that their element type has.
 *
 * ERRORS.  The return codes and their names are qstate.h's.  Invalid
 * arguments are rejected before any CUDA call.  Calls are asynchronous on
 * `stream`, allocate nothing, keep nothing between calls and may be captured
 * into a CUDA graph.  Buffers belong to the current device.  The waits inside
 * the prompt scan of bfloat16 inputs are bounded: where one runs out, y and the
 * state of its segment and of what follows in its sequence are NaN, and
 * qmixer_scan_timeouts counts it.
 */
#ifndef QMIXER_H
#define QMIXER_H

#include <stdint.h>

#include "qstate.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    QMIXER_INITIAL = 1,   /* prompts: continue from `state` */
    QMIXER_SILU = 2,      /* conv: activate the output */
    QMIXER_SOFTPLUS = 4   /* scan: dt is given before its softplus */
};

typedef enum { QMIXER_BEFORE_NONE = 0, QMIXER_BEFORE_RESIDUAL = 1, QMIXER_BEFORE_GATE = 2 } qmixer_before;
typedef enum { QMIXER_OUT_SAME = 0, QMIXER_OUT_INT8 = 1, QMIXER_OUT_E4M3 = 2 } qmixer_out;

/* Causal convolution of width 2 to 4 over a prompt.  state may be NULL
 * without QMIXER_INITIAL (it is then not kept). */
typedef struct qmixer_conv_args {
    const void* x;
    int64_t x_stride;
    const void* weight;
    const void* bias;
    void* state;
    void* y;
    int64_t y_stride;
    const int32_t* seq_starts;
    int32_t sequences;
    int64_t tokens;
    int32_t channels, width, dtype, flags;
} qmixer_conv_args;
int qmixer_conv(const qmixer_conv_args* args, qstate_stream stream);

/* The same for one token of each sequence: x, y [batch][channels]; every row
 * of state moves on by one token. */
typedef struct qmixer_conv_step_args {
    const void* x;
    int64_t x_stride;
    const void* weight;
    const void* bias;
    void* state;
    void* y;
    int64_t y_stride;
    int32_t batch, channels, width, dtype, flags;
} qmixer_conv_step_args;
int qmixer_conv_step(const qmixer_conv_step_args* args, qstate_stream stream);

/* Selective scan of a prompt.  d_k and d_v 64 or 128, groups dividing heads.
 * dtype is the type of x, B, C and y, dt_dtype that of dt.  state may be NULL
 * without QMIXER_INITIAL.  workspace: qmixer_scan_workspace() bytes of device
 * memory on a 16-byte boundary, used by this call alone until it has run (two
 * graphs that may run at once need one each); QSTATE_EINVAL if it is smaller. */
typedef struct qmixer_scan_args {
    const void* x;
    int64_t x_stride;
    const void* dt;
    int64_t dt_stride;
    const float* A;
    const void* B;
    int64_t B_stride;
    const void* C;
    int64_t C_stride;
    const float* D;
    const float* dt_bias;
    float* state;
    void* y;
    int64_t y_stride;
    const int32_t* seq_starts;
    int32_t sequences;
    int64_t tokens;
    int32_t heads, groups, d_k, d_v, dtype, dt_dtype, flags;
    void* workspace;
    int64_t workspace_bytes;
} qmixer_scan_args;
int qmixer_scan(const qmixer_scan_args* args, qstate_stream stream);

/* Bytes of workspace that qmixer_scan needs for these sizes on the current
 * device; a negative return code for sizes that it refuses. */
int64_t qmixer_scan_workspace(int32_t sequences, int64_t tokens, int32_t heads, int32_t groups,
                              int32_t d_k, int32_t d_v, int32_t dtype);

/* How many thread blocks of prompt scans on the current device have given up a
 * bounded wait since the library was loaded: 0, unless the GPU was withheld from
 * a running kernel for seconds.  Waits for `stream`; not while it is captured. */
int qmixer_scan_timeouts(uint64_t* count, qstate_stream stream);

/* Fault injection for tests of the bounded waits, for all prompt scans of the
 * process that follow: each wait takes at most `wait_polls` polls (default 2^24,
 * several seconds), and the inputs of a segment's chunks of 128 tokens from
 * drop_from_chunk on are never loaded, so that the waits for them run out; -1
 * loads all again.  The context stays usable.  QSTATE_EINVAL for wait_polls 0. */
int qmixer_debug_set(int32_t drop_from_chunk, uint32_t wait_polls);

/* The same for one token of each sequence on binary32 states: x, y
 * [batch][heads][d_v]; every state moves on by one token. */
typedef struct qmixer_scan_step_args {
    const void* x;
    int64_t x_stride;
    const void* dt;
    int64_t dt_stride;
    const float* A;
    const void* B;
    int64_t B_stride;
    const void* C;
    int64_t C_stride;
    const float* D;
    const float* dt_bias;
    float* state;
    void* y;
    int64_t y_stride;
    int32_t batch, heads, groups, d_k, d_v, dtype, dt_dtype, flags;
} qmixer_scan_step_args;
int qmixer_scan_step(const qmixer_scan_step_args* args, qstate_stream stream);

/* One token of each sequence on a low-bit state: these operands, qstate_step
 * of a QSTATE_MAMBA2 object of one layer, then qmixer_step_output.  Writes
 * q = C and k = B of each head's group, v = dt x (qkv_dtype) and the gate
 * a = exp(dt A) (gate_dtype) in qstate_step's layouts. */
typedef struct qmixer_step_operands_args {
    const void* x;
    int64_t x_stride;
    const void* dt;
    int64_t dt_stride;
    const float* A;
    const void* B;
    int64_t B_stride;
    const void* C;
    int64_t C_stride;
    const float* dt_bias;
    void* q;
    void* k;
    void* v;
    void* gates;
    int32_t batch, heads, groups, d_k, d_v, dtype, dt_dtype, qkv_dtype, gate_dtype, flags;
} qmixer_step_operands_args;
int qmixer_step_operands(const qmixer_step_operands_args* args, qstate_stream stream);

/* y = out + D x: out [batch][heads][d_v] binary32 as qstate_step leaves it. */
typedef struct qmixer_step_output_args {
    const float* out;
    const void* x;
    int64_t x_stride;
    const float* D;
    void* y;
    int64_t y_stride;
    int32_t batch, heads, d_v, dtype;
} qmixer_step_output_args;
int qmixer_step_output(const qmixer_step_output_args* args, qstate_stream stream);

/* Root-mean-square norm.  before: QMIXER_BEFORE_RESIDUAL adds x to `other`
 * (the residual, which receives the sum in its own type) and normalises the
 * unrounded sum; QMIXER_BEFORE_GATE normalises x silu(other).  out: the
 * inputs' type, or 8-bit codes with binary32 scales of each row (group 0) or
 * of each `group` consecutive columns (a power of two from 8 to 256 dividing
 * columns).  scale = max|y| / Qmax, Qmax 127 (int8) or 448 (e4m3), code = y /
 * scale, both quotients rounded to binary32 first, the code then half to even
 * (int8) or to nearest even (e4m3), and clamped to Qmax.  (y's own binary32
 * value is not the rounded one: the reciprocal root is off by up to 2 units, the
 * silu of bfloat16 inputs by up to 10 + 2.4 |gate| of 2^-24.)  Where max|y| is 0
 * the scale and codes are 0, where it is not a finite number the scale is NaN
 * and the codes 0.  columns 1 to 32768. */
typedef struct qmixer_norm_args {
    const void* x;
    int64_t x_stride;
    void* other;
    int64_t other_stride;
    const void* weight;
    void* y;
    int64_t y_stride;
    float* scales;
    int64_t rows;
    int32_t columns, group;
    float eps;
    int32_t dtype, before, out;
} qmixer_norm_args;
int qmixer_norm(const qmixer_norm_args* args, qstate_stream stream);

/* Quantise binary32 states S [rows][heads][d_k][d_v] (rows = layers * batch)
 * into codes and scales in qstate's layouts, ready for qstate_import: scale =
 * cvt(max|S| / Qmax) of each group, code = clamp(round_half_even(S * inv)),
 * the dynamic rule of qstate.h on a fresh state.  head_bits: NULL, or a HOST
 * array [heads] of 2/4/6/8 that overrides bits (at most 512 heads).  bits 32
 * copies.  rotation 1: the rotated state S H is quantised; `ref` (NULL, or
 * the yoked reference [rows][heads][d_k][d_v]) receives what is quantised.  A
 * group that holds a NaN gets the scale NaN, so that all its values read back
 * as NaN and the next step counts its tile; one that holds an infinity gets
 * the scale infinity, in binary16 65504, at which such scales saturate, and
 * unspecified codes (neither is counted here). */
typedef struct qmixer_quantize_args {
    const float* S;
    void* codes;
    void* scales;
    float* ref;
    int64_t rows;
    int32_t heads, d_k, d_v, bits;
    const uint8_t* head_bits;
    int32_t group, scale_dtype, rotation;
} qmixer_quantize_args;
int qmixer_quantize(const qmixer_quantize_args* args, qstate_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* QMIXER_H */
