/*
 * ssd_mixer.h -- C ABI of the operators around the Mamba2 SSD scan of
 * ssd_scan.h: what a Mamba2 mixer computes between its in-projection and its
 * out-projection, for packed prompts and for single tokens, and a state cache
 * held in 8 bits.
 *
 *   ssd_conv_varlen   prompts: short causal convolution of the packed x, B, C
 *                     channels, split into the scan's dense inputs
 *   ssd_step          single tokens: convolution, dt, state update, read-out
 *                     and gate of one token per request, in one launch
 *   ssd_gated_norm    RMS norm with the SiLU gate, after the scan or the step
 *   ssd_state_store   states into an 8-bit cache (quantised as written)
 *   ssd_state_load    states back out of it
 *
 * A prompt runs ssd_conv_varlen, ssd_scan_varlen, ssd_gated_norm; a decoded
 * token ssd_step, ssd_gated_norm.  With an 8-bit cache the prompt's initial
 * states come through ssd_state_load and its final states leave through
 * ssd_state_store.
 *
 * Common rules, as in ssd_scan.h: the caller owns every buffer; a call checks
 * its arguments on the host, enqueues exactly one kernel (none for an empty
 * batch) on `stream`, a stream of the calling thread's current device, on which
 * the buffers lie too, and returns; nothing is allocated, synchronised or read
 * back, so a call may be captured in a CUDA graph; no call needs a workspace.
 * Invalid arguments return an error status and launch nothing.  Faults in
 * device-resident metadata make the kernel skip that request or sequence and
 * OR a bit into *device_status (if not NULL); the kernels never trap.  All
 * arithmetic is in fp32, rounded once where a value is stored.  SiLU goes through
 * approximations of 2^v and 1 / v: relative error below 2^-20 + |v| 2^-23, zero
 * below about v = -87.3 (results below 2^-119); ssd_step says where its
 * convolution does not.  Every pointer must be aligned to its element type, else
 * SSD_ERR_INVALID_ARG; 16-byte aligned rows take the wide paths, others are
 * computed as exactly.
 *
 * Slots: slot_idx entry s is at slot_idx[s * slot_idx_stride] (0 = 1).  The
 * slots of one call must be distinct (entries of -1 may repeat); of two requests
 * that name one slot it is unspecified what either reads there and which one's
 * write stays.  -1 marks padding in ssd_step alone; to the other entry points it
 * is a bad slot like any that the cache does not have.
 */
#ifndef SSD_MIXER_H_
#define SSD_MIXER_H_

#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit storage of a state cache, beside SSD_F32, SSD_BF16 and SSD_F16.  The
 * N values of a state row [slot, h, p, :] are codes times one fp32 scale:
 *   m = max |h_n|;  inv = (1 / m) lim;  code_n = round(h_n inv);
 *   scale = m (1 / lim)
 * (each operation, also of the rules below, rounded to fp32 by itself).
 * with lim 448 (E4M3, codes are e4m3 numbers) or 127 (I8, codes are signed
 * integers).  A row with m < 2^-100 is held as zeros with scale 0; a row with
 * an infinity or a NaN gets the scale NaN, so that it reads back as NaN.
 * Rounding is to nearest even, or with sr_seed stochastic: element e (flat
 * index in the cache) takes byte e & 15 of the sixteen bytes of Philox4x32-10
 * with key (seed, seed >> 32) and counter (e >> 4, e >> 36, 2, 0), byte 0
 * being the lowest of word 0.
 *   I8:   code = floor(h inv + (byte + 0.5) / 256)
 *   E4M3: h inv / 256 is rounded to fp16, whose magnitude bits, plus
 *         the low 7 bits of the byte, are cut to e4m3's (fp16 keeps 7 bits
 *         more than e4m3 over the whole range, subnormals included).      */
#define SSD_E4M3 3
#define SSD_I8 4

/* bit of *device_status: start_pos[s] or pos[b] negative */
#define SSD_DEV_BAD_POS 32

/* Largest convolution width. */
#define SSD_CONV_MAX_WIDTH 8

/* ------------------------------------------------------------------------
 * Short causal convolution of packed prompts.  For token t of sequence s
 * (0 <= t < len_s, the sequence's own position start_pos[s] + t) and channel c:
 *
 *   u_t[c] = act(bias[c] + sum_{k < width} weight[c, width-1-k] xbc_{t-k}[c])
 *
 * act is SiLU or the identity.  Inputs from before this call (t - k < 0) come
 * from the convolution cache, or are zero where the sequence has no such
 * token (start_pos[s] + t - k < 0).  The convolution cache is a ring per
 * slot: row (position mod conv_rows) holds the raw input of the token at that
 * position.  The call leaves the last width - 1 inputs of the sequence there
 * (as many of them as the call has).  With start_pos = 0 nothing of a slot is
 * read, so slots need no clearing.
 * Channels [0, split0) go to out0, the next split1 to out1, the rest to out2,
 * each dense: the x, B and C of ssd_scan_varlen.  dt, in io_dtype, is widened
 * to the scan's fp32 out_dt by the same launch.
 * Tokens of no valid sequence are written in no output.
 * Layouts:
 *   xbc    [T, channels]  io_dtype, row stride xbc_stride elements
 *   dt     [T, nheads]    io_dtype, row stride dt_stride, or NULL
 *   weight [channels, width], bias [channels]  io_dtype (bias may be NULL)
 *   conv_cache [num_slots, conv_rows, channels] io_dtype, conv_rows >= width,
 *              or NULL: then start_pos must be NULL too and nothing is kept
 * Outputs must not overlap inputs.                                         */
typedef struct {
    int64_t total_tokens;       /* T                                          */
    int32_t num_seqs;
    int32_t channels;
    int32_t width;              /* 1 .. SSD_CONV_MAX_WIDTH                    */
    int32_t io_dtype;           /* SSD_F32 or SSD_BF16                        */
    int32_t activation;         /* 1: SiLU, 0: none                           */
    int32_t split0, split1;
    int32_t nheads;             /* columns of dt, 0 without                   */
    int32_t num_slots;
    int32_t conv_rows;
    const void *xbc;
    int64_t xbc_stride;
    const void *weight;
    const void *bias;           /* may be NULL                                */
    const int32_t *cu_seqlens;  /* [S+1], as in ssd_scan_params               */
    const int32_t *start_pos;   /* [S] tokens before this call, NULL = all 0  */
    const int32_t *slot_idx;    /* [S], may be NULL without conv_cache        */
    int64_t slot_idx_stride;
    void *conv_cache;
    void *out0, *out1, *out2;   /* NULL where they have no channels           */
    const void *dt;
    int64_t dt_stride;
    float *out_dt;              /* [T, nheads] dense, NULL without dt         */
    int32_t *device_status;
} ssd_conv_params;

ssd_status ssd_conv_varlen(const ssd_conv_params *params, struct CUstream_st *stream);

/* ------------------------------------------------------------------------
 * One token for each of `batch` requests.  For request b in slot q at
 * position pos[b], head h of group g = h / (nheads / ngroups):
 *
 *   u      = act(bias + sum_k weight[:, width-1-k] xbc at position pos - k)
 *   x, B, C = u[0 : H P], u[H P : H P + G N], u[H P + G N :]
 *   dt'    = softplus(dt + dt_bias)  (or dt + dt_bias)
 *   h[p,n] = exp(dt' A) h[p,n] + dt' x[p] B[n]      (the cache's state; 0 if
 *                                                    pos[b] = 0)
 *   y[p]   = sum_n C[n] h[p,n] + D x[p], times SiLU(z[p]) where z is given
 *
 * y uses h before it is rounded for the cache.  The convolution cache is the
 * ring of ssd_conv_varlen; the call writes row pos mod conv_rows.  The state
 * cache is rewritten in place, rounded to nearest even, or stochastically
 * with sr_seed (SSD_F16: the rule of ssd_scan_params.sr_seed with stream 0;
 * 8-bit: the rule above; other types ignore it).  Use a new seed each step.
 * With an 8-bit cache, with an SSD_F16 cache and sr_seed, and with SSD_F32
 * activations and any cache below fp32, every operation up to the stored state is
 * rounded to fp32 by itself, in the order of the formulas (taps from the oldest
 * on, then the bias; SiLU as v / (1 + e^-v)), so that a plain fp32 program stores
 * the same bits; otherwise products and sums may be fused.
 * slot -1 marks a padding request (a batch of fixed size in a CUDA graph):
 * its y is zero and nothing else of it is read or written.
 * Layouts:
 *   xbc [batch, H P + 2 G N] io_dtype, row stride xbc_stride
 *   z   [batch, H P] io_dtype, row stride z_stride, or NULL
 *   dt  [batch, H] io_dtype, row stride dt_stride
 *   weight, bias, conv_cache as above with H P + 2 G N channels
 *   A, dt_bias, D [H] fp32 (the last two may be NULL)
 *   state_cache [num_slots, H, P, N] state_dtype
 *   state_scale [num_slots, H, P] fp32, 8-bit caches only
 *   out_y [batch, H, P] io_dtype, dense, must not overlap any input
 * dstate up to 256 (SSD_ERR_UNSUPPORTED above).                            */
typedef struct {
    int32_t batch;
    int32_t nheads, headdim, dstate, ngroups;
    int32_t width;
    int32_t io_dtype;
    int32_t state_dtype;        /* SSD_F32, _BF16, _F16, _E4M3 or _I8         */
    int32_t activation;
    int32_t dt_softplus;
    int32_t num_slots;
    int32_t conv_rows;
    const void *xbc;
    int64_t xbc_stride;
    const void *z;
    int64_t z_stride;
    const void *dt;
    int64_t dt_stride;
    const void *weight;
    const void *bias;
    const float *A, *dt_bias, *D;
    const int32_t *pos;         /* [batch] tokens of the request before this  */
    const int32_t *slot_idx;    /* [batch]                                    */
    int64_t slot_idx_stride;
    void *conv_cache;
    void *state_cache;
    float *state_scale;
    const uint64_t *sr_seed;    /* device, or NULL                            */
    void *out_y;
    int32_t *device_status;
} ssd_step_params;

ssd_status ssd_step(const ssd_step_params *params, struct CUstream_st *stream);

/* ------------------------------------------------------------------------
 * Gated RMS norm over groups of group_size columns:
 *   norm_before_gate = 0:  out = rms(y SiLU(z)) weight
 *   norm_before_gate = 1:  out = rms(y) weight SiLU(z)
 * with rms(v) = v / sqrt(mean(v^2 over the group) + eps); without z the gate
 * is 1.  y, z, out: [rows, columns] io_dtype with row strides; weight
 * [columns] io_dtype or NULL (ones).  out may be y (the same pointer and
 * stride) and otherwise must not overlap an input.                         */
typedef struct {
    int64_t rows;
    int32_t columns;
    int32_t group_size;         /* divides columns                            */
    int32_t io_dtype;
    int32_t norm_before_gate;
    float eps;                  /* >= 0                                       */
    int32_t reserved0;
    const void *y;
    int64_t y_stride;
    const void *z;
    int64_t z_stride;
    const void *weight;
    void *out;
    int64_t out_stride;
} ssd_gated_norm_params;

ssd_status ssd_gated_norm(const ssd_gated_norm_params *params, struct CUstream_st *stream);

/* ------------------------------------------------------------------------
 * States [num_states, H, P, N] (SSD_F32 or SSD_BF16, dense) to and from
 * the slots of an 8-bit cache (state_cache [num_slots, H, P, N], state_scale
 * [num_slots, H, P]), in the form described at SSD_E4M3.  A state of a bad slot
 * is skipped: the store writes nothing for it, the load leaves its part of
 * states as it was.  has_init (uint8 [num_states], NULL = all 1) is used by
 * ssd_state_load alone: where it is 0 the state becomes zeros and the slot is
 * not looked at.  sr_seed is used by ssd_state_store alone.  dstate up to 256. */
typedef struct {
    int32_t num_states;
    int32_t nheads, headdim, dstate;
    int32_t dense_dtype;        /* of states: SSD_F32 or SSD_BF16             */
    int32_t state_dtype;        /* SSD_E4M3 or SSD_I8                         */
    int32_t num_slots;
    int32_t reserved0;
    void *states;               /* read by store, written by load             */
    void *state_cache;
    float *state_scale;
    const int32_t *slot_idx;
    int64_t slot_idx_stride;
    const uint8_t *has_init;
    const uint64_t *sr_seed;
    int32_t *device_status;
} ssd_state_params;

ssd_status ssd_state_store(const ssd_state_params *params, struct CUstream_st *stream);
ssd_status ssd_state_load(const ssd_state_params *params, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_MIXER_H_ */
