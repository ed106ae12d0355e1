/*
 * ssd_layer.h -- C ABI of the operators at a Mamba2 layer's edges and of the
 * decoding loop around it: what a layer computes before its mixer and in its
 * projections when few tokens are decoded, and what a multi-token round does
 * after the model's last layer.
 *
 *   ssd_residual_norm  residual addition and RMS norm, before the in-projection;
 *                      its output also in 8 bits with scales
 *   ssd_matvec4        products of few rows with 4-bit weights: the projections,
 *                      and the head of the vocabulary
 *   ssd_verify_drafts  which drafted tokens of each window stand, and the token
 *                      that follows them; advances ssd_replay_mtp's ring counts
 *
 * A decoded token or window runs ssd_residual_norm, ssd_matvec4 (which reads the
 * norm's 8-bit output as it is), ssd_step or ssd_conv_varlen and ssd_replay_mtp,
 * ssd_gated_norm, ssd_matvec4; a round of windows ends with ssd_verify_drafts.
 *
 * Common rules as in ssd_mixer.h: the caller owns every buffer; a call checks
 * its arguments on the host, enqueues exactly one kernel (none where there is
 * nothing to do) on `stream`, a stream of the calling thread's current device,
 * on which the buffers lie too, and returns; nothing is allocated, synchronised
 * or read back, no workspace is needed, and a call may be captured in a CUDA
 * graph.  Invalid arguments return an error status and launch nothing; every
 * pointer must be aligned to its element type, else SSD_ERR_INVALID_ARG.
 * Outputs must not overlap inputs or one another unless it is said that they
 * may.  The same call gives the same bits each time, whatever runs beside it.
 */
#ifndef SSD_LAYER_H_
#define SSD_LAYER_H_

#include "ssd_mixer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bits OR-ed into *device_status by ssd_verify_drafts */
#define SSD_DEV_BAD_TOKEN 64   /* a drafted token outside [0, vocab)           */
#define SSD_DEV_BAD_PROBS 128  /* a row without a positive finite probability, */
                               /* or whose sum is no finite fp32 number        */

/* ------------------------------------------------------------------------
 * Residual addition and RMS norm.  For row t:
 *
 *   v = x + residual                       (fp32; x alone where residual is NULL)
 *   residual_out = v, rounded              (if not NULL)
 *   n = v / sqrt(mean(v^2) + eps) * weight
 *   out = n, rounded                       (if not NULL)
 *   out_codes, out_scale = n in 8 bits     (if not NULL)
 *
 * The norm is of v before it is rounded, the codes are of n before it is
 * rounded.  The codes of scale_group columns share one fp32 scale by the rule of
 * SSD_E4M3 and SSD_I8 (ssd_mixer.h), to nearest even.  Squares and their sum are in
 * fp32: where the sum is beyond it n is 0 (NaN where v is not finite), and with
 * eps = 0 a row of zeros has no norm (NaN).
 * Layouts, with row strides in elements:
 *   x, out        [rows, columns] io_dtype          weight [columns] or NULL
 *   residual, residual_out [rows, columns] residual_dtype
 *   out_codes     [rows, columns] one byte each
 *   out_scale     [rows, columns / scale_group] fp32, dense
 * residual_out may be residual, and out may be x (same pointer and stride); where
 * io_dtype is residual_dtype residual_out may be x too, if out is not.
 * columns up to 2^20 (SSD_ERR_UNSUPPORTED above).                           */
typedef struct {
    int64_t rows;
    int32_t columns;
    int32_t io_dtype;           /* SSD_F32 or SSD_BF16                        */
    int32_t residual_dtype;     /* SSD_F32 or SSD_BF16                        */
    int32_t code_dtype;         /* with out_codes: SSD_E4M3 or SSD_I8         */
    int32_t scale_group;        /* with out_codes: divides columns            */
    float eps;                  /* >= 0                                       */
    const void *x;
    int64_t x_stride;
    const void *residual;       /* may be NULL                                */
    int64_t residual_stride;
    const void *weight;         /* NULL = ones                                */
    void *residual_out;         /* may be NULL                                */
    int64_t residual_out_stride;
    void *out;                  /* at least one of out and out_codes          */
    int64_t out_stride;
    uint8_t *out_codes;
    int64_t codes_stride;
    float *out_scale;           /* with out_codes                             */
} ssd_residual_norm_params;

ssd_status ssd_residual_norm(const ssd_residual_norm_params *params, struct CUstream_st *stream);

/* ------------------------------------------------------------------------
 * Rows of x times a matrix of 4-bit weights:
 *
 *   out[r, o] = bias[o] + sum_k scale[o, k / group_size] (code[o, k] - zero[o, k / group_size]) x[r, k]
 *
 * Codes are 0 .. 15, zero is 8 where it is NULL.  Code k of row o is the low
 * (k even) or high (k odd) half of byte k / 2 of the row.  x is fp32 or bf16, or
 * 8-bit codes times x_scale[r, k / x_group] (what ssd_residual_norm leaves).
 * All arithmetic is in fp32, each output is rounded once; a group's columns may be
 * added before their scale is applied (15 |x| group_size has to be a fp32 number,
 * scales are below 2^121).  It is made for few rows: more of them are computed as
 * exactly, and read and unpack the weights again, which takes its time each time
 * (once for every 32 rows, 10 of fp32).
 * Layouts:
 *   x       [rows, in_features] x_dtype, row stride x_stride elements
 *   x_scale [rows, ceil(in_features / x_group)] fp32, dense (8-bit x alone)
 *   weight  [out_features, ceil(in_features / 2)] bytes, row stride weight_stride
 *   scale   [out_features, ceil(in_features / group_size)] scale_dtype, dense
 *   zero    the same, one byte each, dense (or NULL)
 *   bias    [out_features] out_dtype (or NULL)
 *   out     [rows, out_features] out_dtype, row stride out_stride elements
 * Any in_features, group_size and x_group are computed.  The tensor cores take rows
 * of up to 2^20 columns, even group sizes from 16 on (and x_group a multiple of 32 with group_size, or equal to
 * it, or a row); multiples of 32 without waste, and fastest rows of whole 16 bytes.
 * in_features and out_features up to 2^30 (SSD_ERR_UNSUPPORTED above), and rows
 * whose tiles a grid holds (500,000).                                       */
typedef struct {
    int32_t rows;
    int32_t in_features;
    int32_t out_features;
    int32_t group_size;         /* >= 1; in_features or more: one group a row */
    int32_t x_dtype;            /* SSD_F32, SSD_BF16, SSD_E4M3 or SSD_I8      */
    int32_t x_group;            /* 8-bit x: columns of a scale, >= 1          */
    int32_t scale_dtype;        /* SSD_F32, SSD_BF16 or SSD_F16               */
    int32_t out_dtype;          /* SSD_F32 or SSD_BF16                        */
    const void *x;
    int64_t x_stride;
    const float *x_scale;
    const uint8_t *weight;
    int64_t weight_stride;
    const void *scale;
    const uint8_t *zero;        /* may be NULL                                */
    const void *bias;           /* may be NULL                                */
    void *out;
    int64_t out_stride;
} ssd_matvec4_params;

ssd_status ssd_matvec4(const ssd_matvec4_params *params, struct CUstream_st *stream);

/* ------------------------------------------------------------------------
 * Verification of drafted tokens against the target's probabilities, from given
 * random numbers.  Window s holds the tokens cu_seqlens[s] .. cu_seqlens[s+1]-1:
 * the last token that stands, then its k drafts d_1 .. d_k (a window of one token
 * has none: plain sampling).  Row cu_seqlens[s] + i of target_probs is the
 * target's distribution p_i of the token that follows token i of the window; row
 * cu_seqlens[s] - s + i of draft_probs and entry cu_seqlens[s] - s + i of accept_u
 * belong to draft d_(i+1): the distribution q_i that it was drawn from and its
 * random number u_i.  Without draft_probs the drafts were given, not drawn (q_i is
 * 1 at d_(i+1) and 0 elsewhere).
 *
 *   n = the number of drafts before the first with u_(n) q_n(d_(n+1)) >= p_n(d_(n+1))
 *   w = max(p_n - q_n, 0), or p_n if n = k or no entry of max(p_n - q_n, 0) is positive
 *   new = the lowest token t whose w[0] + .. + w[t] > sample_u[s] (w[0] + .. + w[V-1])
 *
 * which leaves tokens distributed as the target's where the random numbers are
 * uniform in [0, 1) (values outside count as the nearest end, NaN as 0).  Products,
 * differences and comparisons are exact, the sums are kept to about 2^-44 of the
 * total.  Entries of w that are not positive and finite count as zero; where none
 * is left, or their sum is beyond fp32's largest number, new is -1 and
 * SSD_DEV_BAD_PROBS is set.  Rows need not sum to one.
 *
 *   out_tokens[cu_seqlens[s] + i] = d_(i+1) for i < n, new for i = n, -1 behind
 *   out_accepted[s] = n
 *   ring_count[s] += n + 1      (if not NULL: the inputs of the window that stand,
 *                                as ssd_replay_mtp's caller has to add them)
 *
 * Windows without tokens are padding, come last, and nothing of theirs is
 * written.  A window with bad cu_seqlens, whose draft rows are not within
 * [0, num_drafts), or in which a drafted token outside [0, vocab) is met, is
 * skipped: SSD_DEV_BAD_SEQLENS or SSD_DEV_BAD_TOKEN is set and nothing of it is
 * written.  (The window's first token and drafts behind a rejected one are not
 * looked at.  Where cu_seqlens decreases so that other windows overlap, each output
 * there is that of one of them.)
 * Layouts:
 *   target_probs [total_tokens, vocab] prob_dtype, row stride target_stride
 *   draft_probs  [num_drafts, vocab]   prob_dtype, row stride draft_stride, or NULL
 *   tokens [total_tokens], cu_seqlens [num_seqs + 1], accept_u [num_drafts],
 *   sample_u [num_seqs], out_tokens [total_tokens], out_accepted and ring_count
 *   [num_seqs], dense
 * vocab up to 2^30 (SSD_ERR_UNSUPPORTED above).                             */
typedef struct {
    int64_t total_tokens;       /* T                                          */
    int64_t num_drafts;         /* T - S where no window is empty             */
    int32_t num_seqs;           /* S                                          */
    int32_t vocab;              /* V                                          */
    int32_t prob_dtype;         /* SSD_F32 or SSD_BF16                        */
    int32_t reserved0;
    const void *target_probs;
    int64_t target_stride;
    const void *draft_probs;    /* may be NULL                                */
    int64_t draft_stride;
    const int32_t *tokens;
    const int32_t *cu_seqlens;
    const float *accept_u;      /* may be NULL where num_drafts is 0          */
    const float *sample_u;
    int32_t *out_tokens;
    int32_t *out_accepted;
    int32_t *ring_count;        /* may be NULL                                */
    int32_t *device_status;     /* may be NULL                                */
} ssd_verify_params;

ssd_status ssd_verify_drafts(const ssd_verify_params *params, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_LAYER_H_ */
