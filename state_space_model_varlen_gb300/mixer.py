"""ctypes binding of the C ABI in ``include/ssd_mixer.h``: the operators of a
Mamba2 mixer around the scan (packed convolution, single-token step, gated
norm) and the 8-bit state cache.

Each operator has ``make_*_params`` (fills the argument block from torch
tensors, no copies, no device reads: a serving loop keeps it, and the block
keeps its tensors), ``call_*`` (one
call with such a block on a stream of its tensors' device, whatever device is
current; 0 is that device's default stream) and a function that does both and
allocates its outputs.  Marshalling only: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes

from . import binding
from .binding import SSD_BF16, SSD_F16, SSD_F32, SSD_OK, SSDError, _index_ptr, _ptr, _torch

SSD_E4M3, SSD_I8 = 3, 4
SSD_DEV_BAD_POS = 32
SSD_CONV_MAX_WIDTH = 8

# every entry point declared in include/ssd_mixer.h
EXPORTED = ("ssd_conv_varlen", "ssd_gated_norm", "ssd_state_load", "ssd_state_store", "ssd_step")


def _struct(name, fields):
    kinds = {"i32": ctypes.c_int32, "i64": ctypes.c_int64, "f32": ctypes.c_float, "p": ctypes.c_void_p}
    pairs = [(n, kinds[k]) for k, names in fields for n in names.split()]
    return type(name, (ctypes.Structure,), {"_fields_": pairs, "__doc__": "Mirror of the C struct of this operator.",
                                            "device": None})


ConvParams = _struct("ConvParams", [
    ("i64", "total_tokens"),
    ("i32", "num_seqs channels width io_dtype activation split0 split1 nheads num_slots conv_rows"),
    ("p", "xbc"), ("i64", "xbc_stride"), ("p", "weight bias cu_seqlens start_pos slot_idx"),
    ("i64", "slot_idx_stride"), ("p", "conv_cache out0 out1 out2 dt"), ("i64", "dt_stride"),
    ("p", "out_dt device_status")])
StepParams = _struct("StepParams", [
    ("i32", "batch nheads headdim dstate ngroups width io_dtype state_dtype activation dt_softplus num_slots conv_rows"),
    ("p", "xbc"), ("i64", "xbc_stride"), ("p", "z"), ("i64", "z_stride"), ("p", "dt"), ("i64", "dt_stride"),
    ("p", "weight bias A dt_bias D pos slot_idx"), ("i64", "slot_idx_stride"),
    ("p", "conv_cache state_cache state_scale sr_seed out_y device_status")])
GatedNormParams = _struct("GatedNormParams", [
    ("i64", "rows"), ("i32", "columns group_size io_dtype norm_before_gate"), ("f32", "eps"), ("i32", "reserved0"),
    ("p", "y"), ("i64", "y_stride"), ("p", "z"), ("i64", "z_stride"), ("p", "weight out"), ("i64", "out_stride")])
StateParams = _struct("StateParams", [
    ("i32", "num_states nheads headdim dstate dense_dtype state_dtype num_slots reserved0"),
    ("p", "states state_cache state_scale slot_idx"), ("i64", "slot_idx_stride"),
    ("p", "has_init sr_seed device_status")])

_STRUCTS = {"ssd_conv_varlen": ConvParams, "ssd_step": StepParams, "ssd_gated_norm": GatedNormParams,
            "ssd_state_store": StateParams, "ssd_state_load": StateParams}
_entries = {}


def _entry(name):
    """The C function of that name, loading (and if needed building) the library at its first use."""
    f = getattr(binding.load(), name)
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(_STRUCTS[name]), ctypes.c_void_p]
    _entries[name] = f
    return f


def _call(name, params, stream_ptr):
    entry = _entries.get(name) or _entry(name)
    rc = entry(params, stream_ptr or None) if params.device is None else binding.enqueue(entry, params, stream_ptr)
    if rc != SSD_OK:
        raise MixerError(name, rc)


class MixerError(SSDError):
    """An entry point of ``include/ssd_mixer.h`` refused its arguments."""

    def __init__(self, name: str, code: int):
        RuntimeError.__init__(self, "%s failed: %s (%d)" % (name, binding.status_string(code), code))
        self.code = code


def _stream(t, stream):
    if not t.is_cuda:
        raise ValueError("the mixer operators run on CUDA tensors")
    if stream is None:
        return _torch().cuda.current_stream(t.device).cuda_stream
    if stream.device != t.device:
        raise ValueError("the stream is of %s, the tensors are on %s" % (stream.device, t.device))
    return stream.cuda_stream


def _io(t):
    return binding._dtype_code(t, (SSD_F32, SSD_BF16))


def _state_code(t):
    torch = _torch()
    codes = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16, torch.float16: SSD_F16,
             torch.float8_e4m3fn: SSD_E4M3, torch.int8: SSD_I8}
    if t.dtype not in codes:
        raise TypeError("unsupported state cache dtype %s" % t.dtype)
    return codes[t.dtype]


def _rows(t, dtype=None, columns=None):
    """(pointer, row stride) of a 2-D tensor whose rows are dense; a 3-D one is taken as [rows, a * b]."""
    if t is None:
        return None, 0
    if t.dim() == 3:
        if t.shape[2] != 1 and t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError("the rows of a tensor passed to the mixer operators must be dense")
    elif t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("expected a 2-D tensor with dense rows")
    if dtype is not None and t.dtype != dtype:
        raise TypeError("expected %s, got %s" % (dtype, t.dtype))
    n = t.shape[1] * (t.shape[2] if t.dim() == 3 else 1)
    if columns is not None and n != columns:
        raise ValueError("expected rows of %d values, got %d" % (columns, n))
    return t.data_ptr(), int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), n)


def _shape(t, want, what):
    if t is not None and tuple(t.shape) != tuple(want):
        raise ValueError("%s must have the shape %s, not %s" % (what, tuple(want), tuple(t.shape)))


def _hold(params, *tensors):
    """The block's tensors, which live as long as it does, and their device (see ``binding.block_device``)."""
    where = {t.device for t in tensors if t is not None}
    if len(where) > 1:
        raise ValueError("the tensors of a call must be on one device, not on %s" % sorted(map(str, where)))
    params.device, params.tensors = binding.block_device(where.pop()), tensors


def _seed_ptr(t):
    torch = _torch()
    if t is None:
        return None
    if t.dtype not in (torch.int64, torch.uint64) or t.numel() != 1:
        raise TypeError("sr_seed must be one 64-bit integer in device memory")
    return t.data_ptr()


def _positions(t, n, what):
    if t is None:
        return None
    _shape(t, (n,), what)
    return _ptr(t, _torch().int32)


def _slots(p, t, n):
    if t is None:
        raise ValueError("slot_idx is missing")
    _shape(t, (n,), "slot_idx")
    p.slot_idx, p.slot_idx_stride = _index_ptr(t)
    if n > 1 and t.stride(0) <= 0:
        raise ValueError("slot_idx must have a positive stride")


# ---------------------------------------------------------------------------
# packed convolution
# ---------------------------------------------------------------------------
def make_conv_params(xbc, weight, cu_seqlens, out_x, out_B=None, out_C=None, *, bias=None, activation=True,
                     conv_cache=None, slot_idx=None, start_pos=None, dt=None, out_dt=None,
                     device_status=None) -> ConvParams:
    """Fill ``ssd_conv_params``.  ``xbc`` [T, channels] may be a column range of a wider tensor; the channels go to
    ``out_x``, ``out_B`` and ``out_C`` ([T, ...], dense) in that order."""
    torch = _torch()
    p = ConvParams()
    _hold(p, xbc, weight, cu_seqlens, out_x, out_B, out_C, bias, conv_cache, slot_idx, start_pos, dt, out_dt,
          device_status)
    T, C = xbc.shape
    S = cu_seqlens.shape[0] - 1
    p.total_tokens, p.num_seqs, p.channels, p.width = T, S, C, weight.shape[-1]
    p.io_dtype, p.activation = _io(xbc), int(bool(activation))
    p.xbc, p.xbc_stride = _rows(xbc)
    _shape(weight, (C, weight.shape[-1]), "weight")
    _shape(bias, (C,), "bias")
    p.weight, p.bias = _ptr(weight, xbc.dtype), _ptr(bias, xbc.dtype)
    p.cu_seqlens = _ptr(cu_seqlens, torch.int32)
    widths = []
    for o in (out_x, out_B, out_C):
        if o is not None and o.shape[0] != T:
            raise ValueError("the outputs must have one row per token")
        widths.append(0 if o is None else _row_numel(o))
    if sum(widths) != C:
        raise ValueError("the outputs have %d channels, xbc has %d" % (sum(widths), C))
    p.split0, p.split1 = widths[0], widths[1]
    p.out0, p.out1, p.out2 = (_ptr(o, xbc.dtype) for o in (out_x, out_B, out_C))
    if conv_cache is not None:
        _shape(conv_cache, (conv_cache.shape[0], conv_cache.shape[1], C), "conv_cache")
        p.conv_cache = _ptr(conv_cache, xbc.dtype)
        p.num_slots, p.conv_rows = conv_cache.shape[0], conv_cache.shape[1]
        _slots(p, slot_idx, S)
    p.start_pos = _positions(start_pos, S, "start_pos")
    if (dt is None) != (out_dt is None):
        raise ValueError("dt and out_dt go together")
    if dt is not None:
        p.nheads = dt.shape[1]
        _shape(dt, (T, p.nheads), "dt")
        _shape(out_dt, (T, p.nheads), "out_dt")
        p.dt, p.dt_stride = _rows(dt, xbc.dtype)
        p.out_dt = _ptr(out_dt, torch.float32)
    p.device_status = _ptr(device_status, torch.int32)
    return p


def _row_numel(t):
    n = 1
    for v in t.shape[1:]:
        n *= v
    return n


def call_conv(params: ConvParams, stream_ptr: int = 0) -> None:
    _call("ssd_conv_varlen", params, stream_ptr)


def conv_varlen(xbc, weight, cu_seqlens, *, nheads, headdim, ngroups, dstate, bias=None, activation=True,
                conv_cache=None, slot_idx=None, start_pos=None, dt=None, device_status=None, stream=None):
    """The short causal convolution of packed prompts; returns the scan's dense inputs (x, B, C, dt).  dt is None
    where none is given."""
    torch = _torch()

    def out(*shape, dtype=xbc.dtype):
        return binding.allocated(lambda: torch.empty(xbc.shape[0], *shape, dtype=dtype, device=xbc.device), xbc.device,
                                 stream)

    x, B, C = out(nheads, headdim), out(ngroups, dstate), out(ngroups, dstate)
    out_dt = None if dt is None else out(nheads, dtype=torch.float32)
    call_conv(make_conv_params(xbc, weight, cu_seqlens, x, B, C, bias=bias, activation=activation,
                               conv_cache=conv_cache, slot_idx=slot_idx, start_pos=start_pos, dt=dt, out_dt=out_dt,
                               device_status=device_status), _stream(xbc, stream))
    return x, B, C, out_dt


# ---------------------------------------------------------------------------
# single-token step
# ---------------------------------------------------------------------------
def make_step_params(xbc, dt, weight, A, conv_cache, state_cache, pos, slot_idx, out_y, *, ngroups, z=None,
                     conv_bias=None, dt_bias=None, D=None, state_scale=None, sr_seed=None, activation=True,
                     dt_softplus=True, device_status=None) -> StepParams:
    """Fill ``ssd_step_params``: one token for each row of ``xbc``.  ``xbc``, ``z`` and ``dt`` may be column ranges of
    one in-projection output; ``sr_seed`` is a one-element int64 device tensor."""
    torch = _torch()
    p = StepParams()
    _hold(p, xbc, dt, weight, A, conv_cache, state_cache, pos, slot_idx, out_y, z, conv_bias, dt_bias, D, state_scale,
          sr_seed, device_status)
    H, P, N = state_cache.shape[1:]
    B, C = xbc.shape
    if C != H * P + 2 * ngroups * N:
        raise ValueError("xbc has %d channels, %d heads of %d and %d groups of %d need %d"
                         % (C, H, P, ngroups, N, H * P + 2 * ngroups * N))
    p.batch, p.nheads, p.headdim, p.dstate, p.ngroups, p.width = B, H, P, N, ngroups, weight.shape[-1]
    p.io_dtype, p.state_dtype = _io(xbc), _state_code(state_cache)
    p.activation, p.dt_softplus = int(bool(activation)), int(bool(dt_softplus))
    _shape(conv_cache, (state_cache.shape[0], conv_cache.shape[1], C), "conv_cache")
    p.num_slots, p.conv_rows = conv_cache.shape[0], conv_cache.shape[1]
    p.xbc, p.xbc_stride = _rows(xbc)
    if z is not None and z.shape[0] != B or dt.shape[0] != B:
        raise ValueError("z and dt must have one row per request")
    p.z, p.z_stride = _rows(z, xbc.dtype, H * P)
    p.dt, p.dt_stride = _rows(dt, xbc.dtype, H)
    _shape(weight, (C, weight.shape[-1]), "weight")
    for t, n, what in ((conv_bias, C, "conv_bias"), (A, H, "A"), (dt_bias, H, "dt_bias"), (D, H, "D")):
        _shape(t, (n,), what)
    p.weight, p.bias = _ptr(weight, xbc.dtype), _ptr(conv_bias, xbc.dtype)
    p.A, p.dt_bias, p.D = (_ptr(t, torch.float32) for t in (A, dt_bias, D))
    p.pos = _positions(pos, B, "pos")
    _slots(p, slot_idx, B)
    p.conv_cache, p.state_cache = _ptr(conv_cache, xbc.dtype), _ptr(state_cache)
    _shape(state_scale, state_cache.shape[:3], "state_scale")
    p.state_scale = _ptr(state_scale, torch.float32)
    p.sr_seed = _seed_ptr(sr_seed)
    _shape(out_y, (B, H, P), "out_y")
    p.out_y = _ptr(out_y, xbc.dtype)
    p.device_status = _ptr(device_status, torch.int32)
    return p


def call_step(params: StepParams, stream_ptr: int = 0) -> None:
    _call("ssd_step", params, stream_ptr)


def step(xbc, dt, weight, A, conv_cache, state_cache, pos, slot_idx, *, ngroups, out_y=None, stream=None, **options):
    """One token per request: convolution, state update, read-out and (with ``z``) gate; returns ``out_y``
    [batch, H, P].  Both caches are updated in place.  ``options`` are those of ``make_step_params``."""
    if out_y is None:
        out_y = binding.allocated(lambda: _torch().empty(xbc.shape[0], *state_cache.shape[1:3], dtype=xbc.dtype,
                                                         device=xbc.device), xbc.device, stream)
    call_step(make_step_params(xbc, dt, weight, A, conv_cache, state_cache, pos, slot_idx, out_y, ngroups=ngroups,
                               **options), _stream(xbc, stream))
    return out_y


# ---------------------------------------------------------------------------
# gated norm
# ---------------------------------------------------------------------------
def make_norm_params(y, weight, out, *, z=None, group_size=None, eps=1e-5, norm_before_gate=False) -> GatedNormParams:
    """Fill ``ssd_gated_norm_params``.  ``y``, ``z`` and ``out`` are [rows, columns] or [rows, H, P]."""
    p = GatedNormParams()
    _hold(p, y, weight, out, z)
    columns = _row_numel(y)
    p.rows, p.columns = y.shape[0], columns
    p.group_size = columns if group_size is None else int(group_size)
    p.io_dtype, p.eps, p.norm_before_gate = _io(y), float(eps), int(bool(norm_before_gate))
    for t in (z, out):
        if t is not None and t.shape[0] != y.shape[0]:
            raise ValueError("y, z and out must have the same rows")
    p.y, p.y_stride = _rows(y)
    p.z, p.z_stride = _rows(z, y.dtype, columns)
    p.out, p.out_stride = _rows(out, y.dtype, columns)
    _shape(weight, (columns,), "weight")
    p.weight = _ptr(weight, y.dtype)
    return p


def call_norm(params: GatedNormParams, stream_ptr: int = 0) -> None:
    _call("ssd_gated_norm", params, stream_ptr)


def gated_rms_norm(y, weight=None, *, z=None, group_size=None, eps=1e-5, norm_before_gate=False, out=None,
                   stream=None):
    """RMS norm of ``y`` over groups of columns with the SiLU gate ``z``; returns ``out``."""
    if out is None:
        out = binding.allocated(lambda: _torch().empty(y.shape, dtype=y.dtype, device=y.device), y.device, stream)
    call_norm(make_norm_params(y, weight, out, z=z, group_size=group_size, eps=eps,
                               norm_before_gate=norm_before_gate), _stream(y, stream))
    return out


# ---------------------------------------------------------------------------
# 8-bit state cache
# ---------------------------------------------------------------------------
def make_state_params(states, state_cache, state_scale, slot_idx, *, has_init=None, sr_seed=None,
                      device_status=None) -> StateParams:
    """Fill ``ssd_state_params``: dense ``states`` [n, H, P, N] and the slots of an 8-bit cache."""
    torch = _torch()
    p = StateParams()
    _hold(p, states, state_cache, state_scale, slot_idx, has_init, sr_seed, device_status)
    n, H, P, N = states.shape
    p.num_states, p.nheads, p.headdim, p.dstate = n, H, P, N
    p.dense_dtype, p.state_dtype, p.num_slots = _io(states), _state_code(state_cache), state_cache.shape[0]
    _shape(state_cache, (state_cache.shape[0], H, P, N), "state_cache")
    _shape(state_scale, state_cache.shape[:3], "state_scale")
    p.states, p.state_cache, p.state_scale = _ptr(states), _ptr(state_cache), _ptr(state_scale, torch.float32)
    _slots(p, slot_idx, n)
    if has_init is not None and has_init.dtype == torch.bool:
        has_init = has_init.view(torch.uint8)
    _shape(has_init, (n,), "has_init")
    p.has_init = _ptr(has_init, torch.uint8)
    p.sr_seed = _seed_ptr(sr_seed)
    p.device_status = _ptr(device_status, torch.int32)
    return p


def call_state_store(params: StateParams, stream_ptr: int = 0) -> None:
    _call("ssd_state_store", params, stream_ptr)


def call_state_load(params: StateParams, stream_ptr: int = 0) -> None:
    _call("ssd_state_load", params, stream_ptr)


def state_store(states, state_cache, state_scale, slot_idx, *, sr_seed=None, device_status=None, stream=None) -> None:
    """Quantise ``states`` into the slots of an 8-bit cache."""
    call_state_store(make_state_params(states, state_cache, state_scale, slot_idx, sr_seed=sr_seed,
                                       device_status=device_status), _stream(states, stream))


def state_load(state_cache, state_scale, slot_idx, *, states=None, dtype=None, has_init=None, device_status=None,
               stream=None):
    """Read slots of an 8-bit cache back into dense states (fp32 unless ``dtype`` or ``states`` says otherwise)."""
    torch = _torch()
    if states is None:
        states = binding.allocated(lambda: torch.empty(slot_idx.shape[0], *state_cache.shape[1:],
                                                       dtype=dtype or torch.float32, device=state_cache.device),
                                   state_cache.device, stream)
    call_state_load(make_state_params(states, state_cache, state_scale, slot_idx, has_init=has_init,
                                      device_status=device_status), _stream(states, stream))
    return states
