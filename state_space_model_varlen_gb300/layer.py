"""ctypes binding of the C ABI in ``include/ssd_layer.h``: the operators at a
Mamba2 layer's edges (residual norm with an 8-bit output, products with 4-bit
weights) and of the decoding loop (verification of drafted tokens).

As in :mod:`.mixer`, each operator has ``make_*_params`` (the argument block, which
keeps its tensors), ``call_*`` (one call with such a block on a stream of its
tensors' device) and a function that does both and allocates its outputs.
Marshalling only: there is no fallback implementation.
"""
from __future__ import annotations

from . import binding, mixer
from .binding import SSD_BF16, SSD_F16, SSD_F32, _ptr, _torch
from .mixer import SSD_E4M3, SSD_I8, MixerError, _call, _hold, _io, _rows, _shape, _stream, _struct

SSD_DEV_BAD_TOKEN, SSD_DEV_BAD_PROBS = 64, 128

# every entry point declared in include/ssd_layer.h
EXPORTED = ("ssd_matvec4", "ssd_residual_norm", "ssd_verify_drafts")

ResidualNormParams = _struct("ResidualNormParams", [
    ("i64", "rows"), ("i32", "columns io_dtype residual_dtype code_dtype scale_group"), ("f32", "eps"),
    ("p", "x"), ("i64", "x_stride"), ("p", "residual"), ("i64", "residual_stride"), ("p", "weight residual_out"),
    ("i64", "residual_out_stride"), ("p", "out"), ("i64", "out_stride"), ("p", "out_codes"), ("i64", "codes_stride"),
    ("p", "out_scale")])
Matvec4Params = _struct("Matvec4Params", [
    ("i32", "rows in_features out_features group_size x_dtype x_group scale_dtype out_dtype"),
    ("p", "x"), ("i64", "x_stride"), ("p", "x_scale weight"), ("i64", "weight_stride"), ("p", "scale zero bias out"),
    ("i64", "out_stride")])
VerifyParams = _struct("VerifyParams", [
    ("i64", "total_tokens num_drafts"), ("i32", "num_seqs vocab prob_dtype reserved0"),
    ("p", "target_probs"), ("i64", "target_stride"), ("p", "draft_probs"), ("i64", "draft_stride"),
    ("p", "tokens cu_seqlens accept_u sample_u out_tokens out_accepted ring_count device_status")])

mixer._STRUCTS.update({"ssd_residual_norm": ResidualNormParams, "ssd_matvec4": Matvec4Params,
                       "ssd_verify_drafts": VerifyParams})
LayerError = MixerError     # what a refused call raises: the same error as the mixer operators'


def _code(t, what):
    torch = _torch()
    if t.dtype not in (torch.float8_e4m3fn, torch.int8):
        raise TypeError("%s must be float8_e4m3fn or int8, not %s" % (what, t.dtype))
    return SSD_E4M3 if t.dtype == torch.float8_e4m3fn else SSD_I8


def _row_count(n, **tensors):
    for what, t in tensors.items():
        if t is not None and t.shape[0] != n:
            raise ValueError("%s must have %d rows, not %d" % (what, n, t.shape[0]))


def _i32(*sizes):
    """Sizes for fields of 32 bits.  What these do not hold becomes the largest number that they do, which the library
    refuses: a wrapped one could pass its checks, and the call would then read and write by it."""
    return [min(n, 0x7fffffff) for n in sizes]


# ---------------------------------------------------------------------------
# residual norm
# ---------------------------------------------------------------------------
def make_residual_norm_params(x, weight=None, out=None, *, residual=None, residual_out=None, codes=None, scale=None,
                              eps=1e-5) -> ResidualNormParams:
    """Fill ``ssd_residual_norm_params``.  ``x``, ``out``, ``residual``, ``residual_out`` and ``codes`` are [rows, columns],
    ``scale`` [rows, groups]; ``codes`` is float8_e4m3fn or int8.  ``residual_out`` may be ``residual``, ``out`` may be
    ``x``."""
    torch = _torch()
    p = ResidualNormParams()
    _hold(p, x, weight, out, residual, residual_out, codes, scale)
    columns = mixer._row_numel(x)
    p.rows, (p.columns,) = x.shape[0], _i32(columns)
    _row_count(p.rows, out=out, residual=residual, residual_out=residual_out, codes=codes, scale=scale)
    p.io_dtype, p.eps = _io(x), float(eps)
    p.x, p.x_stride = _rows(x)
    stream = residual if residual is not None else residual_out
    p.residual_dtype = p.io_dtype if stream is None else _io(stream)
    p.residual, p.residual_stride = _rows(residual, None, columns)
    p.residual_out, p.residual_out_stride = _rows(residual_out, None if stream is None else stream.dtype, columns)
    _shape(weight, (columns,), "weight")
    p.weight = _ptr(weight, x.dtype)
    p.out, p.out_stride = _rows(out, x.dtype, columns)
    if (codes is None) != (scale is None):
        raise ValueError("codes and scale go together")
    if codes is not None:
        p.code_dtype = _code(codes, "codes")
        p.out_codes, p.codes_stride = _rows(codes, None, columns)
        p.out_scale = _ptr(scale, torch.float32)
        if scale.dim() != 2 or scale.shape[1] < 1 or columns % scale.shape[1]:
            raise ValueError("scale must be [rows, groups], groups a divisor of the %d columns" % columns)
        p.scale_group, = _i32(columns // scale.shape[1])
    return p


def call_residual_norm(params: ResidualNormParams, stream_ptr: int = 0) -> None:
    _call("ssd_residual_norm", params, stream_ptr)


def residual_rms_norm(x, weight=None, *, residual=None, residual_out=None, code_dtype=None, scale_group=None, eps=1e-5,
                      out=None, stream=None):
    """RMS norm of ``x + residual``, whose sum goes to ``residual_out`` (which may be ``residual``).  Returns ``out``, or
    with ``code_dtype`` (float8_e4m3fn or int8) the codes and their scales, one for ``scale_group`` columns (default: the
    row)."""
    torch = _torch()

    def empty(shape, dtype):
        return binding.allocated(lambda: torch.empty(shape, dtype=dtype, device=x.device), x.device, stream)

    codes = scale = None
    if code_dtype is not None:
        columns = mixer._row_numel(x)
        group = columns if scale_group is None else int(scale_group)
        if group < 1 or columns % group:
            raise ValueError("scale_group must divide the %d columns" % columns)
        codes, scale = empty(x.shape, code_dtype), empty((x.shape[0], columns // group), torch.float32)
    elif scale_group is not None:
        raise ValueError("scale_group goes with code_dtype")
    elif out is None:
        out = empty(x.shape, x.dtype)
    call_residual_norm(make_residual_norm_params(x, weight, out, residual=residual, residual_out=residual_out, codes=codes,
                                                 scale=scale, eps=eps), _stream(x, stream))
    return out if codes is None else (codes, scale)


# ---------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------
def make_matvec4_params(x, weight, scale, out, *, group_size, zero=None, bias=None, x_scale=None) -> Matvec4Params:
    """Fill ``ssd_matvec4_params``: ``x`` [rows, in] (fp32, bf16, or 8-bit codes with ``x_scale`` [rows, groups]),
    ``weight`` [out, ceil(in / 2)] uint8 (code k of a row: the low half of byte k / 2 for even k), ``scale`` and ``zero``
    [out, ceil(in / group_size)].  The columns of a row that share an ``x_scale`` are in / groups, which must be whole."""
    torch = _torch()
    p = Matvec4Params()
    _hold(p, x, weight, scale, out, zero, bias, x_scale)
    M, K = x.shape
    O = weight.shape[0]
    group_size = int(group_size)
    if group_size < 1:
        raise ValueError("group_size must be positive")
    p.rows, p.in_features, p.out_features = _i32(M, K, O)
    p.group_size = min(group_size, 1 << 30)     # the longest row's: one group
    if x.dtype in (torch.float8_e4m3fn, torch.int8):
        p.x_dtype = _code(x, "x")
        if x_scale is None:
            raise ValueError("x in 8 bits needs x_scale")
        if x_scale.dim() != 2 or x_scale.shape[0] != M or x_scale.shape[1] < 1 or K % x_scale.shape[1]:
            raise ValueError("x_scale must be [rows, groups], groups a divisor of the %d columns" % K)
        (p.x_group,), p.x_scale = _i32(K // x_scale.shape[1]), _ptr(x_scale, torch.float32)
    else:
        p.x_dtype = _io(x)
        if x_scale is not None:
            raise ValueError("x_scale goes with x in 8 bits")
    p.x, p.x_stride = _rows(x)
    _shape(weight, (O, (K + 1) // 2), "weight")
    p.weight, p.weight_stride = _rows(weight, torch.uint8)
    groups = -(-K // group_size)
    _shape(scale, (O, groups), "scale")
    _shape(zero, (O, groups), "zero")
    p.scale_dtype = binding._dtype_code(scale, (SSD_F32, SSD_BF16, SSD_F16))
    p.scale, p.zero = _ptr(scale), _ptr(zero, torch.uint8)
    p.out_dtype = _io(out)
    _shape(bias, (O,), "bias")
    p.bias = _ptr(bias, out.dtype)
    _shape(out, (M, O), "out")
    p.out, p.out_stride = _rows(out)
    return p


def call_matvec4(params: Matvec4Params, stream_ptr: int = 0) -> None:
    _call("ssd_matvec4", params, stream_ptr)


def matvec4(x, weight, scale, *, group_size, zero=None, bias=None, x_scale=None, out=None, out_dtype=None, stream=None):
    """Rows of ``x`` times 4-bit weights; returns ``out`` [rows, out] (of x's type, bf16 for 8-bit x, unless ``out_dtype``
    or ``out`` says otherwise)."""
    torch = _torch()
    if out is None:
        dtype = out_dtype or (x.dtype if x.dtype in (torch.float32, torch.bfloat16) else torch.bfloat16)
        out = binding.allocated(lambda: torch.empty(x.shape[0], weight.shape[0], dtype=dtype, device=x.device), x.device,
                                stream)
    call_matvec4(make_matvec4_params(x, weight, scale, out, group_size=group_size, zero=zero, bias=bias, x_scale=x_scale),
                 _stream(x, stream))
    return out


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------
def make_verify_params(target_probs, tokens, cu_seqlens, accept_u, sample_u, out_tokens, out_accepted, *,
                       draft_probs=None, ring_count=None, device_status=None) -> VerifyParams:
    """Fill ``ssd_verify_params``: windows packed by ``cu_seqlens``, ``target_probs`` [T, V], ``accept_u`` and
    ``draft_probs`` one entry or row for each drafted token in order ([T - S] where no window is empty)."""
    torch = _torch()
    p = VerifyParams()
    _hold(p, target_probs, tokens, cu_seqlens, accept_u, sample_u, out_tokens, out_accepted, draft_probs, ring_count,
          device_status)
    T, V = target_probs.shape
    S, n = cu_seqlens.shape[0] - 1, 0 if accept_u is None else accept_u.shape[0]
    p.total_tokens, p.num_drafts, (p.num_seqs, p.vocab) = T, n, _i32(S, V)
    p.prob_dtype = _io(target_probs)
    p.target_probs, p.target_stride = _rows(target_probs)
    if draft_probs is not None:
        _shape(draft_probs, (n, V), "draft_probs")
        p.draft_probs, p.draft_stride = _rows(draft_probs, target_probs.dtype)
    for what, t, shape in (("tokens", tokens, (T,)), ("accept_u", accept_u, (n,)), ("sample_u", sample_u, (S,)),
                           ("out_tokens", out_tokens, (T,)), ("out_accepted", out_accepted, (S,)),
                           ("ring_count", ring_count, (S,))):
        _shape(t, shape, what)
    i32, f32 = torch.int32, torch.float32
    p.tokens, p.cu_seqlens = _ptr(tokens, i32), _ptr(cu_seqlens, i32)
    p.accept_u, p.sample_u = _ptr(accept_u, f32), _ptr(sample_u, f32)
    p.out_tokens, p.out_accepted, p.ring_count = (_ptr(t, i32) for t in (out_tokens, out_accepted, ring_count))
    p.device_status = _ptr(device_status, i32)
    return p


def call_verify(params: VerifyParams, stream_ptr: int = 0) -> None:
    _call("ssd_verify_drafts", params, stream_ptr)


def verify_drafts(target_probs, tokens, cu_seqlens, accept_u, sample_u, *, draft_probs=None, ring_count=None,
                  device_status=None, out_tokens=None, out_accepted=None, stream=None):
    """Which drafts of each window stand, and the token after them; returns (tokens [T], accepted [S]).  ``ring_count`` is
    advanced in place by what stands of each window."""
    torch = _torch()

    def empty(n):
        return binding.allocated(lambda: torch.empty(n, dtype=torch.int32, device=target_probs.device), target_probs.device,
                                 stream)

    out_tokens = empty(target_probs.shape[0]) if out_tokens is None else out_tokens
    out_accepted = empty(cu_seqlens.shape[0] - 1) if out_accepted is None else out_accepted
    call_verify(make_verify_params(target_probs, tokens, cu_seqlens, accept_u, sample_u, out_tokens, out_accepted,
                                   draft_probs=draft_probs, ring_count=ring_count, device_status=device_status),
                _stream(target_probs, stream))
    return out_tokens, out_accepted
