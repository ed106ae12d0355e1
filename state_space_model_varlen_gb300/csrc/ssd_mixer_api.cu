// C ABI entry points of the mixer operators: host-side argument checks and
// dispatch.  See include/ssd_mixer.h for the contract.
#include "ssd_mixer_internal.h"

namespace {

size_t io_size(int dtype) { return dtype == SSD_F32 ? 4 : 2; }
bool io_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }

// a required or optional array of elements of `size` bytes
bool required(const void *p, size_t size) { return p != nullptr && ssd::aligned_to(p, size); }
bool optional(const void *p, size_t size) { return ssd::aligned_to(p, size); }

ssd_status done(cudaError_t err) {
    if (err == cudaSuccess) return SSD_OK;
    return err == cudaErrorInvalidConfiguration ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

ssd_status check(const ssd_conv_params *p) {
    if (p == nullptr || !io_ok(p->io_dtype)) return SSD_ERR_INVALID_ARG;
    const size_t io = io_size(p->io_dtype);
    if (p->total_tokens < 0 || p->num_seqs < 0 || p->channels <= 0 || p->width < 1 || p->nheads < 0)
        return SSD_ERR_INVALID_ARG;
    if (p->width > SSD_CONV_MAX_WIDTH) return SSD_ERR_UNSUPPORTED;
    if (p->split0 < 0 || p->split1 < 0 || (int64_t)p->split0 + p->split1 > p->channels) return SSD_ERR_INVALID_ARG;
    if (p->num_seqs == 0 || p->total_tokens == 0) return SSD_OK;
    if (p->xbc_stride < p->channels || p->slot_idx_stride < 0) return SSD_ERR_INVALID_ARG;
    if (!required(p->xbc, io) || !required(p->weight, io) || !optional(p->bias, io) || !required(p->cu_seqlens, 4))
        return SSD_ERR_INVALID_ARG;
    const int rest = p->channels - p->split0 - p->split1;
    if ((p->split0 > 0 && !required(p->out0, io)) || (p->split1 > 0 && !required(p->out1, io)) ||
        (rest > 0 && !required(p->out2, io)))
        return SSD_ERR_INVALID_ARG;
    if (p->conv_cache != nullptr) {
        if (!required(p->conv_cache, io) || !required(p->slot_idx, 4) || p->num_slots <= 0 ||
            p->conv_rows < p->width)
            return SSD_ERR_INVALID_ARG;
    } else if (p->start_pos != nullptr) {
        return SSD_ERR_INVALID_ARG;
    }
    if (!optional(p->start_pos, 4) || !optional(p->device_status, 4)) return SSD_ERR_INVALID_ARG;
    if ((p->dt == nullptr) != (p->out_dt == nullptr)) return SSD_ERR_INVALID_ARG;
    if (p->dt != nullptr &&
        (p->nheads <= 0 || p->dt_stride < p->nheads || !required(p->dt, io) || !required(p->out_dt, 4)))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status check(const ssd_step_params *p) {
    if (p == nullptr || !io_ok(p->io_dtype)) return SSD_ERR_INVALID_ARG;
    const size_t io = io_size(p->io_dtype);
    if (p->state_dtype < SSD_F32 || p->state_dtype > SSD_I8) return SSD_ERR_INVALID_ARG;
    if (p->batch < 0 || p->nheads <= 0 || p->headdim <= 0 || p->dstate <= 0 || p->ngroups <= 0 || p->width < 1)
        return SSD_ERR_INVALID_ARG;
    if (p->nheads % p->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (p->width > SSD_CONV_MAX_WIDTH || p->dstate > 256) return SSD_ERR_UNSUPPORTED;
    const int64_t hp = (int64_t)p->nheads * p->headdim, channels = hp + 2LL * p->ngroups * p->dstate;
    if (hp * p->dstate > (1LL << 31) || channels > (1LL << 30)) return SSD_ERR_UNSUPPORTED;
    if (p->batch == 0) return SSD_OK;
    if (p->xbc_stride < channels || p->dt_stride < p->nheads || p->slot_idx_stride < 0) return SSD_ERR_INVALID_ARG;
    if (p->z != nullptr && p->z_stride < hp) return SSD_ERR_INVALID_ARG;
    if (p->num_slots <= 0 || p->conv_rows < p->width) return SSD_ERR_INVALID_ARG;
    if (!required(p->xbc, io) || !optional(p->z, io) || !required(p->dt, io) || !required(p->weight, io) ||
        !optional(p->bias, io) || !required(p->A, 4) || !optional(p->dt_bias, 4) || !optional(p->D, 4) ||
        !required(p->pos, 4) || !required(p->slot_idx, 4) || !required(p->conv_cache, io) ||
        !required(p->out_y, io) || !optional(p->sr_seed, 8) || !optional(p->device_status, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t st = p->state_dtype == SSD_F32 ? 4 : p->state_dtype <= SSD_F16 ? 2 : 1;
    if (!required(p->state_cache, st)) return SSD_ERR_INVALID_ARG;
    if (st == 1 && !required(p->state_scale, 4)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status check(const ssd_gated_norm_params *p) {
    if (p == nullptr || !io_ok(p->io_dtype)) return SSD_ERR_INVALID_ARG;
    const size_t io = io_size(p->io_dtype);
    if (p->rows < 0 || p->columns <= 0 || p->group_size <= 0 || p->columns % p->group_size != 0)
        return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    if (p->rows == 0) return SSD_OK;
    if (p->y_stride < p->columns || p->out_stride < p->columns || (p->z != nullptr && p->z_stride < p->columns))
        return SSD_ERR_INVALID_ARG;
    if (!required(p->y, io) || !optional(p->z, io) || !optional(p->weight, io) || !required(p->out, io))
        return SSD_ERR_INVALID_ARG;
    if (p->out == p->y && p->out_stride != p->y_stride && p->rows > 1) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status check(const ssd_state_params *p) {
    if (p == nullptr || !io_ok(p->dense_dtype)) return SSD_ERR_INVALID_ARG;
    if (p->state_dtype != SSD_E4M3 && p->state_dtype != SSD_I8) return SSD_ERR_INVALID_ARG;
    if (p->num_states < 0 || p->nheads <= 0 || p->headdim <= 0 || p->dstate <= 0) return SSD_ERR_INVALID_ARG;
    if (p->dstate > 256) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)p->nheads * p->headdim * p->dstate > (1LL << 31)) return SSD_ERR_UNSUPPORTED;
    if (p->num_states == 0) return SSD_OK;
    if (p->num_slots <= 0 || p->slot_idx_stride < 0) return SSD_ERR_INVALID_ARG;
    if (!required(p->states, io_size(p->dense_dtype)) || p->state_cache == nullptr ||
        !required(p->state_scale, 4) || !required(p->slot_idx, 4) || !optional(p->sr_seed, 8) ||
        !optional(p->device_status, 4))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_conv_varlen(const ssd_conv_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->num_seqs == 0 || params->total_tokens == 0) return v;
    return done(ssd::launch_conv(*params, stream));
}

ssd_status ssd_step(const ssd_step_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->batch == 0) return v;
    switch (params->state_dtype) {
        case SSD_F32: return done(ssd::launch_step_f32(*params, stream));
        case SSD_BF16: return done(ssd::launch_step_bf16(*params, stream));
        case SSD_F16: return done(ssd::launch_step_f16(*params, stream));
        case SSD_E4M3: return done(ssd::launch_step_e4m3(*params, stream));
    }
    return done(ssd::launch_step_i8(*params, stream));
}

ssd_status ssd_gated_norm(const ssd_gated_norm_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->rows == 0) return v;
    return done(ssd::launch_gated_norm(*params, stream));
}

ssd_status ssd_state_store(const ssd_state_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->num_states == 0) return v;
    return done(ssd::launch_state_store(*params, stream));
}

ssd_status ssd_state_load(const ssd_state_params *params, struct CUstream_st *stream) {
    const ssd_status v = check(params);
    if (v != SSD_OK || params->num_states == 0) return v;
    return done(ssd::launch_state_load(*params, stream));
}

}  // extern "C"
