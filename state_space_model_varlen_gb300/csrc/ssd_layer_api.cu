// C ABI entry points of the layer operators: host-side argument checks and
// dispatch.  See include/ssd_layer.h for the contract.
#include "ssd_layer_internal.h"

namespace {

size_t size_of(int dtype) { return dtype == SSD_F32 ? 4 : dtype <= SSD_F16 ? 2 : 1; }
bool io_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }
bool code_ok(int dtype) { return dtype == SSD_E4M3 || dtype == SSD_I8; }

// a required or optional array of elements of `size` bytes
bool required(const void *p, size_t size) { return p != nullptr && ssd::aligned_to(p, size); }
bool optional(const void *p, size_t size) { return ssd::aligned_to(p, size); }

// a and b are one matrix, or two
bool same_or_apart(const void *a, int64_t a_stride, const void *b, int64_t b_stride, int64_t rows) {
    return a == nullptr || a != b || a_stride == b_stride || rows <= 1;
}

constexpr int kMost = 1 << 30;      // sizes below which the kernels' 32-bit indices along a row hold

ssd_status done(cudaError_t err) {
    if (err == cudaSuccess) return SSD_OK;
    return err == cudaErrorInvalidConfiguration ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

ssd_status check(const ssd_residual_norm_params *p) {
    if (p == nullptr || !io_ok(p->io_dtype) || !io_ok(p->residual_dtype)) return SSD_ERR_INVALID_ARG;
    if (p->rows < 0 || p->columns <= 0 || !(p->eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    if (p->out_codes != nullptr &&
        (!code_ok(p->code_dtype) || p->scale_group <= 0 || p->columns % p->scale_group != 0))
        return SSD_ERR_INVALID_ARG;
    if (p->columns > (1 << 20)) return SSD_ERR_UNSUPPORTED;
    if (p->rows == 0) return SSD_OK;
    const size_t io = size_of(p->io_dtype), res = size_of(p->residual_dtype);
    if (!required(p->x, io) || !optional(p->residual, res) || !optional(p->weight, io) || !optional(p->residual_out, res) ||
        !optional(p->out, io) || (p->out == nullptr && p->out_codes == nullptr))
        return SSD_ERR_INVALID_ARG;
    if (p->out_codes != nullptr && (!required(p->out_scale, 4) || p->codes_stride < p->columns)) return SSD_ERR_INVALID_ARG;
    if (p->x_stride < p->columns || (p->residual != nullptr && p->residual_stride < p->columns) ||
        (p->residual_out != nullptr && p->residual_out_stride < p->columns) ||
        (p->out != nullptr && p->out_stride < p->columns))
        return SSD_ERR_INVALID_ARG;
    if (!same_or_apart(p->out, p->out_stride, p->x, p->x_stride, p->rows) ||
        !same_or_apart(p->residual_out, p->residual_out_stride, p->residual, p->residual_stride, p->rows) ||
        !same_or_apart(p->residual_out, p->residual_out_stride, p->x, p->x_stride, p->rows))
        return SSD_ERR_INVALID_ARG;
    // outputs that would overwrite one another, or inputs of other elements
    if (p->out != nullptr && (p->out == p->residual_out || p->out == p->residual)) return SSD_ERR_INVALID_ARG;
    if (p->residual_out != nullptr && p->residual_out == p->x && p->io_dtype != p->residual_dtype) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status check(const ssd_matvec4_params *p) {
    if (p == nullptr || !io_ok(p->out_dtype)) return SSD_ERR_INVALID_ARG;
    if (!io_ok(p->x_dtype) && !code_ok(p->x_dtype)) return SSD_ERR_INVALID_ARG;
    if (p->scale_dtype < SSD_F32 || p->scale_dtype > SSD_F16) return SSD_ERR_INVALID_ARG;
    if (p->rows < 0 || p->in_features <= 0 || p->out_features < 0 || p->group_size <= 0) return SSD_ERR_INVALID_ARG;
    if (code_ok(p->x_dtype) && p->x_group <= 0) return SSD_ERR_INVALID_ARG;
    if (p->in_features > kMost || p->out_features > kMost) return SSD_ERR_UNSUPPORTED;
    if (p->rows == 0 || p->out_features == 0) return SSD_OK;
    const int64_t bytes = ((int64_t)p->in_features + 1) / 2;
    if (p->x_stride < p->in_features || p->weight_stride < bytes || p->out_stride < p->out_features)
        return SSD_ERR_INVALID_ARG;
    const size_t out = size_of(p->out_dtype);
    if (!required(p->x, size_of(p->x_dtype)) || p->weight == nullptr || !required(p->scale, size_of(p->scale_dtype)) ||
        !optional(p->bias, out) || !required(p->out, out))
        return SSD_ERR_INVALID_ARG;
    if (code_ok(p->x_dtype) && !required(p->x_scale, 4)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status check(const ssd_verify_params *p) {
    if (p == nullptr || !io_ok(p->prob_dtype)) return SSD_ERR_INVALID_ARG;
    if (p->total_tokens < 0 || p->num_drafts < 0 || p->num_seqs < 0 || p->vocab <= 0) return SSD_ERR_INVALID_ARG;
    if (p->vocab > kMost) return SSD_ERR_UNSUPPORTED;
    if (p->num_seqs == 0 || p->total_tokens == 0) return SSD_OK;
    const size_t io = size_of(p->prob_dtype);
    if (p->target_stride < p->vocab || (p->draft_probs != nullptr && p->draft_stride < p->vocab)) return SSD_ERR_INVALID_ARG;
    if (!required(p->target_probs, io) || !optional(p->draft_probs, io) || !required(p->tokens, 4) ||
        !required(p->cu_seqlens, 4) || !required(p->sample_u, 4) || !required(p->out_tokens, 4) ||
        !required(p->out_accepted, 4) || !optional(p->ring_count, 4) || !optional(p->device_status, 4))
        return SSD_ERR_INVALID_ARG;
    if (p->num_drafts > 0 ? !required(p->accept_u, 4) : !optional(p->accept_u, 4)) return SSD_ERR_INVALID_ARG;
    if (p->out_tokens == p->tokens) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_residual_norm(const ssd_residual_norm_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->rows == 0) return v;
    return done(params->io_dtype == SSD_F32 ? ssd::launch_residual_norm_f32(*params, stream)
                                            : ssd::launch_residual_norm_bf16(*params, stream));
}

ssd_status ssd_matvec4(const ssd_matvec4_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->rows == 0 || params->out_features == 0) return v;
    return done(ssd::launch_matvec4(*params, stream));
}

ssd_status ssd_verify_drafts(const ssd_verify_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->num_seqs == 0 || params->total_tokens == 0) return v;
    return done(ssd::launch_verify(*params, stream));
}

}  // extern "C"
