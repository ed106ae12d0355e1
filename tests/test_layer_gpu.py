"""The layer operators on the GPU against their formulas in 64 bits."""
import numpy as np
import pytest

from state_space_model_varlen_gb300 import binding, layer
from tests import layer_reference as R
from tests import mixer_reference as M

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _t(name):
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
            "i8": torch.int8, "u8": torch.uint8, "i32": torch.int32}[name]


def _np(t):
    return None if t is None else t.detach().to(_torch().float64).cpu().numpy()


def _bits(t):
    return t.contiguous().view(_torch().uint8).cpu().numpy()


class Draw:
    def __init__(self, seed):
        self.g = _torch().Generator(device="cuda").manual_seed(seed)

    def randn(self, *shape, dtype="f32", scale=1.0):
        return (_torch().randn(*shape, generator=self.g, device="cuda") * scale).to(_t(dtype))

    def rand(self, *shape):
        return _torch().rand(*shape, generator=self.g, device="cuda")

    def ints(self, lo, hi, *shape, dtype="i32"):
        return _torch().randint(lo, hi, shape, generator=self.g, device="cuda").to(_t(dtype))

    def rows(self, rows, cols, dtype, pad=0, at=0, scale=1.0):
        """[rows, cols] as a column range of a wider tensor (row stride cols + pad, from column `at`)."""
        return self.randn(rows, cols + pad, dtype=dtype, scale=scale)[:, at:at + cols]


def _empty(rows, cols, dtype, pad=0):
    """Rows that are overwritten, with columns beside them that have to stay: (the rows, all of it)."""
    full = _torch().full((rows, cols + pad), 7.0, device="cuda").to(_t(dtype))
    return full[:, :cols], full


def _untouched(full, cols):
    assert (full[:, cols:].float() == 7.0).all()


# ---------------------------------------------------------------------------
# residual norm
# ---------------------------------------------------------------------------
def _norm_case(rows, cols, io="bf16", res="f32", code=None, group=None, out=True, weight=True, keep=True, pad=0, at=0, seed=0):
    torch = _torch()
    d = Draw(seed)
    x, w = d.rows(rows, cols, io, pad, at), d.randn(cols, dtype=io) if weight else None
    r = d.rows(rows, cols, res, pad, at, scale=3.0) if res else None
    o, o_full = _empty(rows, cols, io, pad) if out or not code else (None, None)
    s, s_full = _empty(rows, cols, res or io, pad) if keep else (None, None)
    c = c_full = scale = None
    if code:
        c, c_full = _empty(rows, cols, code, pad)
        scale = torch.full((rows, cols // (group or cols)), float("nan"), device="cuda")
    before = [_bits(t) for t in (x, w, r) if t is not None]
    layer.call_residual_norm(layer.make_residual_norm_params(x, w, o, residual=r, residual_out=s, codes=c, scale=scale,
                                                             eps=1e-5), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for b, t in zip(before, [t for t in (x, w, r) if t is not None]):
        assert np.array_equal(b, _bits(t))
    (v, ev), (n, en) = R.residual_norm(_np(x), _np(r), _np(w), 1e-5)
    if o is not None:
        M.check(_np(o), n, en, io, "norm")
        _untouched(o_full, cols)
    if s is not None:
        M.check(_np(s), v, ev, res or io, "sum")
        _untouched(s_full, cols)
    if c is not None:
        shape = (rows, -1, group or cols)
        M.check_codes(_np(c).reshape(shape), _np(scale), n.reshape(shape), en.reshape(shape), code, clear=0.8)
        _untouched(c_full, cols)
        if io == "f32" and o is not None:       # by the rule, from the fp32 values of the norm: bit for bit
            f = o.float().cpu().numpy().reshape(shape)
            m = np.abs(f).max(-1)
            lim = np.float32(R.LIM[code])
            assert np.array_equal(_np(scale), (m * (np.float32(1) / lim)).astype(np.float64))
            inv = (np.float32(1) / m) * lim
            assert np.array_equal(_np(c).reshape(shape), M.codes((f * inv[..., None]).astype(np.float64), code))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 33), (2, 64), (5, 100), (1, 512), (7, 1000), (2, 1001), (4, 2048),
                                       (1, 2560), (3, 4100), (2, 8191), (1, 8192), (2, 16384), (1, 33000), (1, 65536),
                                       (1, 70001), (1, 131072), (300, 256)])
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None)])
def test_norm(rows, cols, io, res):
    _norm_case(rows, cols, io, res, seed=rows * cols)


@pytest.mark.parametrize("cols,group", [(8, 8), (64, 32), (128, 128), (96, 3), (1000, 100), (1000, 125), (1001, 143),
                                        (2560, 128), (2560, 2560), (4096, 64), (4096, 16), (4096, 8), (4096, 4), (4096, 1),
                                        (8192, 1024), (16384, 16384), (65536, 128), (70000, 7000), (512, 512)])
@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("io,res,out", [("bf16", "f32", False), ("f32", "f32", True), ("bf16", "bf16", True)])
def test_norm_codes(cols, group, code, io, res, out):
    _norm_case(3, cols, io, res, code, group, out, seed=cols + group)


@pytest.mark.parametrize("pad,at", [(8, 0), (8, 8), (3, 1), (4, 4), (64, 2), (16, 16)])
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("code", [None, "e4m3"])
def test_norm_strides(pad, at, io, res, code):
    _norm_case(5, 512, io, res, code, 64, pad=pad, at=at)


@pytest.mark.parametrize("weight,keep,res", [(False, True, "f32"), (True, False, "bf16"), (False, False, None), (True, True, None)])
def test_norm_optional_parts(weight, keep, res):
    _norm_case(4, 768, "bf16", res, weight=weight, keep=keep)
    _norm_case(4, 768, "bf16", res, "i8", 96, weight=weight, keep=keep)


@pytest.mark.parametrize("cols", [40, 512, 4096, 100000])
@pytest.mark.parametrize("code", [None, "e4m3"])
def test_norm_in_place(cols, code):
    """The residual stream is advanced in place, and the norm may take x's place."""
    torch = _torch()
    d = Draw(cols)
    x, w, r = d.randn(6, cols, dtype="bf16"), d.randn(cols, dtype="bf16"), d.randn(6, cols)
    kw = dict(code_dtype=_t(code), scale_group=cols // 4) if code else {}
    total = torch.empty_like(r)
    want = layer.residual_rms_norm(x, w, residual=r, residual_out=total, **kw)
    x2, r2 = x.clone(), r.clone()
    got = layer.residual_rms_norm(x2, w, residual=r2, residual_out=r2, **kw, **({} if code else {"out": x2}))
    assert torch.equal(r2, total)
    for a, b in zip(got if code else [got], want if code else [want]):
        assert np.array_equal(_bits(a), _bits(b))
    x3 = x.clone()          # the sum over x itself
    layer.residual_rms_norm(x3, w, residual=x, residual_out=x3)
    assert torch.equal(x3, (x.float() * 2).bfloat16())


@pytest.mark.parametrize("cols", [1, 2, 3, 37, 255, 1001, 2009, 9999, 16387])
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("at", [0, 3])
def test_norm_rows_that_begin_anywhere(cols, io, res, at):
    """Odd dense rows, whose beginnings go through all alignments, also from an odd element on, out of place and in place."""
    torch = _torch()
    d = Draw(cols)
    rows = 9
    flat = lambda dtype: d.randn(rows * cols + at, dtype=dtype)[at:].view(rows, cols)      # noqa: E731
    x, r, w = flat(io), flat(res), d.randn(cols, dtype=io)
    out, total = torch.full_like(flat(io), 7.0), torch.full_like(flat(res), 7.0)
    layer.residual_rms_norm(x, w, residual=r, residual_out=total, out=out)
    (v, ev), (n, en) = R.residual_norm(_np(x), _np(r), _np(w), 1e-5)
    M.check(_np(out), n, en, io, "norm")
    M.check(_np(total), v, ev, res, "sum")
    kept, kept_r = flat(io), flat(res)
    x2, r2 = kept, kept_r
    x2.copy_(x)
    r2.copy_(r)
    layer.residual_rms_norm(x2, w, residual=r2, residual_out=r2, out=x2)
    M.check(_np(x2), n, en, io, "norm")
    M.check(_np(r2), v, ev, res, "sum")


@pytest.mark.parametrize("cols,group", [(64, 32), (4096, 128), (4096, 4096), (3100, 100), (70000, 100)])
@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_norm_special_values(cols, group, code):
    """Rows of zeros; a group that is all zero; groups and rows with an infinity or a NaN."""
    torch = _torch()
    x, w = torch.ones(5, cols, device="cuda"), torch.ones(cols, device="cuda")
    x[0] = 0.0
    w[:group] = 0.0
    x[2, group // 2] = float("nan")
    x[3, -1] = float("inf")
    w[-1] = 3e38
    o, s = torch.empty_like(x), torch.empty(5, cols // group, device="cuda")
    c = torch.empty(5, cols, dtype=_t(code), device="cuda")
    layer.call_residual_norm(layer.make_residual_norm_params(x, w, o, codes=c, scale=s), torch.cuda.current_stream().cuda_stream)
    assert (o[0] == 0).all() and (s[0] == 0).all() and (c[0].float() == 0).all()
    if group < cols:
        assert (s[:2, 0] == 0).all() and (c[:2, :group].float() == 0).all()
        assert torch.isfinite(s[1]).all() and (s[1, 1:] > 0).all()
    assert torch.isnan(o[2]).all() and torch.isnan(s[2]).all()
    assert torch.isnan(s[3, -1])            # inf / inf: the row's last group reads back as NaN
    assert torch.isfinite(o[1, :-1]).all() and torch.isfinite(o[4, :-1]).all()


@pytest.mark.parametrize("cols,group", [(8, 4), (16, 16), (32, 32), (32, 8), (40, 8), (64, 32), (96, 32), (128, 128), (128, 16),
                                        (256, 64), (24, 24), (36, 12), (894, 298), (30, 10)])
@pytest.mark.parametrize("rows", [1, 7, 33, 130])
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("f32", "bf16")])
def test_norm_short_rows(cols, group, rows, io, res):
    """Several rows of a warp, the last of them not there."""
    _norm_case(rows, cols, io, res, "e4m3", group, seed=rows)
    _norm_case(rows, cols, io, res, seed=rows)


@pytest.mark.parametrize("cols", [894, 2002, 12002, 13665, 16382, 20001])
@pytest.mark.parametrize("res", ["f32", "bf16"])
def test_norm_rows_of_two_and_long_odd_ones(cols, res):
    _norm_case(3, cols, "bf16", res)


def test_norm_many_rows():
    """More rows than one wave of CTAs, each the same as alone."""
    torch = _torch()
    d = Draw(3)
    x, r, w = d.randn(40000, 320, dtype="bf16"), d.randn(40000, 320), d.randn(320, dtype="bf16")
    c, s = layer.residual_rms_norm(x, w, residual=r, code_dtype=_t("e4m3"), scale_group=64)
    at = d.ints(0, 40000, 50).long()
    c1, s1 = layer.residual_rms_norm(x[at], w, residual=r[at], code_dtype=_t("e4m3"), scale_group=64)
    assert torch.equal(c.view(torch.uint8)[at], c1.view(torch.uint8)) and torch.equal(s[at], s1)


# ---------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------
def _mv_case(rows, K, O, group, x="bf16", scale="bf16", zero=False, bias=False, x_group=None, out=None, x_pad=0, w_pad=0, w_at=0,
             o_pad=0, seed=0):
    torch = _torch()
    d = Draw(seed + rows + K + O)
    out = out or ("f32" if x == "f32" else "bf16")
    groups = -(-K // group)
    w = d.ints(0, 256, O, (K + 1) // 2 + w_pad, dtype="u8")[:, w_at:w_at + (K + 1) // 2]
    s = (torch.exp(d.randn(O, groups, scale=0.5)) * K ** -0.5).to(_t(scale))
    z = d.ints(0, 16, O, groups, dtype="u8") if zero else None
    b = d.randn(O, dtype=out) if bias else None
    xs = None
    if x in R.LIM:
        xv = d.ints(-127, 128, rows, K + x_pad).to(_t("i8")) if x == "i8" else d.randn(rows, K + x_pad, scale=60.0).clamp(
            -448, 448).to(_t("e4m3"))
        x_group = x_group or K
        xs = torch.exp(d.randn(rows, K // x_group)) * 0.01
    else:
        xv = d.randn(rows, K + x_pad, dtype=x)
    xv = xv[:, :K]
    o, o_full = _empty(rows, O, out, o_pad)
    p = layer.make_matvec4_params(xv, w, s, o, group_size=group, zero=z, bias=b, x_scale=xs)
    layer.call_matvec4(p, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    want, err = R.matvec4(_np(xv), w.cpu().numpy(), _np(s), None if z is None else z.cpu().numpy(), _np(b), group, _np(xs),
                          x_group or 1)
    M.check(_np(o), want, err, out, "product")
    _untouched(o_full, O)
    first = o.clone()
    layer.call_matvec4(p, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(o, first)                # the same bits again


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 9, 16, 21, 33, 64, 65, 130])
@pytest.mark.parametrize("x", ["bf16", "f32", "e4m3", "i8"])
def test_matvec_rows(rows, x):
    _mv_case(rows, 512, 200, 64, x, zero=True, bias=True, x_group=128 if x in R.LIM else None)


@pytest.mark.parametrize("K", [1, 2, 7, 31, 32, 50, 64, 96, 100, 128, 160, 1000, 1023, 1024, 1056, 2080, 4096, 4128, 16384])
@pytest.mark.parametrize("group", [32, 128, 1 << 20])
def test_matvec_columns(K, group):
    _mv_case(2, K, 48, group, "bf16", zero=True)
    _mv_case(3, K, 17, group, "f32", scale="f32", bias=True)


@pytest.mark.parametrize("O", [1, 2, 15, 16, 17, 31, 33, 64, 100, 1000, 5000, 20000, 70001])
def test_matvec_outputs(O):
    _mv_case(1, 256, O, 32, zero=True)
    _mv_case(4, 640, O, 128, "e4m3", x_group=64, bias=True)


@pytest.mark.parametrize("group", [1, 2, 3, 8, 16, 24, 32, 50, 64, 96, 128, 160, 192, 256, 480, 960, 5000])
@pytest.mark.parametrize("scale", ["f32", "bf16", "f16"])
def test_matvec_groups(group, scale):
    _mv_case(3, 960, 70, group, "bf16", scale, zero=group % 2 == 0)
    _mv_case(2, 960, 70, group, "i8", scale, zero=group % 2 == 1, x_group=96)


@pytest.mark.parametrize("x_group", [1, 10, 32, 64, 96, 160, 480, 960])
@pytest.mark.parametrize("x", ["e4m3", "i8"])
def test_matvec_activation_groups(x_group, x):
    _mv_case(5, 960, 40, 64, x, x_group=x_group, zero=True)
    _mv_case(12, 960, 40, 96, x, x_group=x_group, out="f32")


@pytest.mark.parametrize("kw", [dict(x_pad=1), dict(x_pad=8), dict(w_pad=1), dict(w_pad=16), dict(w_pad=32, w_at=16),
                                dict(w_pad=20, w_at=4), dict(o_pad=1), dict(o_pad=8, x_pad=3, w_pad=16)])
@pytest.mark.parametrize("x", ["bf16", "f32", "e4m3"])
def test_matvec_strides(kw, x):
    _mv_case(3, 384, 50, 128, x, zero=True, **kw)


@pytest.mark.parametrize("rows,x,out", [(1, "bf16", "f32"), (17, "f32", "bf16"), (3, "i8", "f32")])
def test_matvec_output_types(rows, x, out):
    _mv_case(rows, 768, 90, 96, x, out=out, bias=True)


@pytest.mark.parametrize("rows,K,O", [(1, 8192, 4096), (3, 4096, 18560), (16, 2560, 10576), (64, 4096, 2048), (1, 32768, 512),
                                      (70, 16384, 64), (1, 128, 100000)])
def test_matvec_large(rows, K, O):
    _mv_case(rows, K, O, 128)
    _mv_case(rows, K, O, 32, "f32" if rows < 20 else "e4m3", zero=True)


@pytest.mark.parametrize("rows", [3, 12, 20, 70])
@pytest.mark.parametrize("group", [32, 64, 128, 1 << 20, 16, 48, 50])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("K", [800, 802])
def test_matvec_variants(rows, group, zero, K):
    """Each number of columns of a pass, of blocks that share scales, with zeros or not, for rows of whole 16 bytes or not."""
    _mv_case(rows, K, 300, group, "bf16", "f32", zero=zero)
    if K % group == 0 or group > K:
        _mv_case(rows, K, 300, group, "e4m3", "f16", zero=zero, x_group=min(group, K))


@pytest.mark.parametrize("rows,O,K", [(1, 64, 4096), (1, 300, 8192), (4, 130, 2176), (1, 5000, 512), (16, 64, 8192), (30, 40, 4224),
                                      (1, 40000, 640), (2, 9, 65536)])
def test_matvec_shares_of_columns(rows, O, K):
    """Columns shared by the warps of a CTA and by the CTAs of a cluster."""
    for group in (128, 32):
        _mv_case(rows, K, O, group, zero=True, bias=True)


def test_matvec_long_rows():
    """More columns than the tensor-core kernel counts."""
    _mv_case(2, (1 << 20) + 64, 3, 128, "bf16", zero=True)


def test_matvec_zeros_of_a_whole_byte():
    torch = _torch()
    d = Draw(6)
    w, s, z = d.ints(0, 256, 20, 128, dtype="u8"), d.rand(20, 2), d.ints(0, 256, 20, 2, dtype="u8")
    x = d.randn(3, 256, dtype="bf16")
    got = layer.matvec4(x, w, s, group_size=128, zero=z, out_dtype=torch.float32)
    want, err = R.matvec4(_np(x), w.cpu().numpy(), _np(s), z.cpu().numpy(), None, 128)
    M.check(_np(got), want, err, "f32", "product")


@pytest.mark.parametrize("group", [64, 25])
def test_matvec_ignores_a_scale_of_x_that_has_none(group):
    torch = _torch()
    d = Draw(7)
    x, w, s = d.randn(2, 256, dtype="bf16"), d.ints(0, 256, 20, 128, dtype="u8"), d.rand(20, -(-256 // group))
    want, out = layer.matvec4(x, w, s, group_size=group), torch.empty(2, 20, dtype=_t("bf16"), device="cuda")
    p = layer.make_matvec4_params(x, w, s, out, group_size=group)
    p.x_scale, p.x_group = s.data_ptr(), 0
    layer.call_matvec4(p, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, want)


def test_matvec_weights_at_large_offsets():
    """A matrix whose rows lie more than 2^32 bytes apart from the first."""
    torch = _torch()
    rows, stride, K = 5, 1 << 30, 256
    store = torch.empty(4 * stride + K // 2, dtype=torch.uint8, device="cuda")
    w = store.as_strided((rows, K // 2), (stride, 1))
    d = Draw(5)
    dense = d.ints(0, 256, rows, K // 2, dtype="u8")
    w.copy_(dense)
    x, s = d.randn(2, K, dtype="bf16"), d.randn(rows, 2)
    assert torch.equal(layer.matvec4(x, w, s, group_size=128), layer.matvec4(x, dense, s, group_size=128))


@pytest.mark.parametrize("K,group", [(256, 64), (250, 25)])
@pytest.mark.parametrize("rows", [2, 40])
def test_matvec_special_values(K, group, rows):
    """An infinity or a NaN in x reaches its own row alone, one in a scale its own output alone; large and small numbers of
    fp32 beside one another."""
    torch = _torch()
    d = Draw(1)
    w = d.ints(0, 256, 20, K // 2, dtype="u8")
    w[:, 3] = 0xFF                                              # codes 7 and 7 above the zero of 8
    s = torch.ones(20, K // group, device="cuda") * 2.0 ** -20
    for dtype in ("f32", "bf16"):
        x = d.randn(rows, K, dtype=dtype)
        clean = layer.matvec4(x, w, s, group_size=group, out_dtype=torch.float32)
        y = x.clone()
        y[0, 6], y[1, 7] = float("inf"), float("nan")
        got = layer.matvec4(y, w, s, group_size=group, out_dtype=torch.float32)
        assert torch.equal(got[2:], clean[2:])
        assert (got[0] == float("inf")).all() and torch.isnan(got[1]).all()
        t = s.clone()
        t[4, 1] = float("nan")
        got = layer.matvec4(x, w, t, group_size=group, out_dtype=torch.float32)
        assert torch.isnan(got[:, 4]).all() and torch.equal(got[:, :4], clean[:, :4]) and torch.equal(got[:, 5:], clean[:, 5:])
    x = torch.zeros(rows, K, device="cuda")
    x[:, 6], x[0, 7] = 3e34, 1e-30          # 15 x K is still an fp32 number
    got = layer.matvec4(x, w, s, group_size=group)
    want = 7.0 * 2.0 ** -20 * float(np.float32(3e34))
    assert np.all(np.abs(_np(got) - want) <= 2.0 ** -22 * want)


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------
def _probs(d, rows, V, dtype, pad=0, scale=2.0):
    torch = _torch()
    p = torch.softmax(d.randn(rows, V, scale=scale), 1).to(_t(dtype))
    full = torch.full((rows, V + pad), 7.0, device="cuda").to(_t(dtype))
    full[:, :V] = p
    return full[:, :V]


def _verify_check(target, draft, tokens, cu, au, su, ring=True):
    torch = _torch()
    T, S = target.shape[0], cu.shape[0] - 1
    out, acc = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (T, S))
    rc = torch.arange(S, dtype=torch.int32, device="cuda") if ring else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = R.verify(_np(target).astype(np.float32) if target.dtype == torch.float32 else _np(target),
                    None if draft is None else _np(draft), tokens.cpu().numpy(), cu.cpu().numpy(),
                    None if au is None else au.cpu().numpy(), su.cpu().numpy(), None if rc is None else rc.cpu().numpy(),
                    out.cpu().numpy(), acc.cpu().numpy())
    layer.call_verify(layer.make_verify_params(target, tokens, cu, au, su, out, acc, draft_probs=draft, ring_count=rc,
                                               device_status=st), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    got = (out.cpu().numpy(), acc.cpu().numpy(), None if rc is None else rc.cpu().numpy(), int(st))
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
    assert not ring or np.array_equal(got[2], want[2])
    assert got[3] == want[3]
    return got


def _windows(lens):
    return _torch().tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=_torch().int32, device="cuda")


def _verify_case(lens, V, dtype="f32", drafts=True, pad=0, seed=0, near=0.5, ring=True):
    torch = _torch()
    d = Draw(seed + V)
    T, S = sum(lens), len(lens)
    D = sum(max(n - 1, 0) for n in lens)
    target = _probs(d, max(T, 1), V, dtype, pad)[:T]
    cu = _windows(lens)
    behind = np.concatenate([[False] * (n > 0) + [True] * (n - 1) for n in lens]) if T else np.zeros(0, bool)
    behind = torch.from_numpy(np.nonzero(behind)[0]).cuda()
    tokens = d.ints(0, V, T)
    q = None
    if D:
        rows = (target[behind - 1].float().log() + d.randn(D, V, scale=near)).softmax(1).to(_t(dtype))
        tokens[behind] = torch.multinomial(rows.float(), 1, generator=d.g).view(-1).int()
        if drafts:
            q = torch.full((D, V + pad), 7.0, device="cuda").to(_t(dtype))[:, :V]
            q.copy_(rows)
    return _verify_check(target, q, tokens, cu, d.rand(D) if D else None, d.rand(S), ring)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 127, 1000, 1024, 4099, 32000, 50277, 131072, 262145])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drafts", [True, False])
def test_verify_vocabularies(V, dtype, drafts):
    acc = np.concatenate([_verify_case([3, 1, 4, 2, 9], V, dtype, drafts, seed=i)[1] for i in range(4)])
    assert V < 1000 or not drafts or 0 < acc.sum() < 4 * 14


@pytest.mark.parametrize("lens", [[1], [2], [3] * 128, [1] * 40, [40, 1, 33, 34, 2], [1100], [32, 33, 31], [5, 3, 0, 0], [300] * 3])
@pytest.mark.parametrize("near", [0.05, 1.0])
def test_verify_windows(lens, near):
    _verify_case(lens, 500, near=near, seed=len(lens))
    _verify_case(lens, 500, "bf16", drafts=False, seed=len(lens), ring=False)


@pytest.mark.parametrize("pad", [1, 4, 7, 8])
def test_verify_strides(pad):
    for dtype in ("f32", "bf16"):
        for V in (1000, 1003):
            _verify_case([3, 4, 1, 6], V, dtype, pad=pad)


def test_verify_many_random_numbers():
    """One window of one row sampled at many places of its distribution, and at the ends."""
    torch = _torch()
    d = Draw(9)
    S = 3000
    p = _probs(d, 1, 777, "f32").expand(S, 777).contiguous()
    u = torch.linspace(0, 1, S, device="cuda")
    u[0], u[-1], u[5], u[6], u[7] = 0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, float("nan")
    got = _verify_check(p, None, torch.zeros(S, dtype=torch.int32, device="cuda"), _windows([1] * S), None, u)
    assert got[0][0] == 0 and got[0][5] == 776 and got[0][6] == 776 and got[0][7] == 0


def test_verify_borders_are_exact():
    """Dyadic probabilities, so that products and sums are exact: a number on the border rejects the draft, and belongs to
    the next token."""
    torch = _torch()
    V, S = 2048, 512
    p = torch.full((2 * S, V), 2.0 ** -11, device="cuda")
    q = torch.full((S, V), 2.0 ** -11, device="cuda")
    p[0::2, 5], q[:, 5] = 2.0 ** -12, 2.0 ** -11
    p[0::2, 6], q[:, 6] = 2.0 ** -11 + 2.0 ** -12, 2.0 ** -12   # left over: 2^-11 at 6, and 2^-12 at 9
    p[0::2, 9], q[:, 9] = 2.0 ** -11 + 2.0 ** -13, 2.0 ** -11 - 2.0 ** -13
    tokens = torch.full((2 * S,), 5, dtype=torch.int32, device="cuda")
    au = torch.full((S,), 0.5, device="cuda")
    au[::2] = 0.5 - 2.0 ** -25                                  # the one just below stands
    su = torch.arange(S, device="cuda", dtype=torch.float32) / S
    two_thirds = 2.0 / 3.0
    su[1], su[3] = (float(np.nextafter(np.float32(two_thirds), np.float32(v))) for v in (0, 1))
    out, acc, _, _ = _verify_check(p, q, tokens, _windows([2] * S), au, su)
    assert (acc[::2] == 1).all() and (acc[1::2] == 0).all()
    assert (out[0::4] == 5).all() and (out[1::4] == (np.arange(0, S, 2) / S * V).astype(int)).all()
    assert out[2] == 6 and out[6] == 9 and set(out[2::4]) == {6, 9}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_rows_that_say_little(dtype):
    torch = _torch()
    V, nan, inf = 300, float("nan"), float("inf")
    base = torch.full((V,), 1.0 / 256, device="cuda")
    p = torch.stack([base] * 16).to(_t(dtype))
    q = torch.stack([base] * 8).to(_t(dtype))
    tokens = torch.full((16,), 7, dtype=torch.int32, device="cuda")
    p[0, 7] = 0.0                       # 0: rejected, and nothing left of p - q: the target's row
    p[2] = 0.0                          # 1: a target row of zeros
    p[4], p[4, 250] = nan, 0.25         # 2: one usable entry
    p[6], q[3, :] = nan, 0.0            # 3: none
    p[8, 3], p[8, 4], p[8, 7] = inf, -1.0, 0.0     # 4: an infinite and a negative entry
    q[4, 9] = 0.0
    q[5], q[5, 7], p[10, 7] = inf, inf, 0.0        # 5: nothing is left where q is infinite
    p[13] = 0.0                         # 6: stands; the row behind it is empty
    q[7, :] = nan                       # 7: a draft row of NaN rejects, and leaves nothing: the target's row
    su = torch.full((8,), 0.6, device="cuda")
    out, acc, _, status = _verify_check(p, q, tokens, _windows([2] * 8), torch.full((8,), 0.5, device="cuda"), su)
    assert status == 128 and out[4] == 250 and out[2] == -1 and out[6] == -1 and out[8] == 9
    assert acc[6] == 1 and out[12] == 7 and out[13] == -1


def test_verify_bad_metadata_skips_its_window_alone():
    torch = _torch()
    d = Draw(4)
    V, i32 = 64, torch.int32
    p, q = _probs(d, 12, V, "f32"), _probs(d, 8, V, "f32")
    au, su = torch.zeros(8, device="cuda"), d.rand(4)
    good = d.ints(0, V, 12)
    for at, value in ((1, -1), (4, V), (11, 1 << 30), (7, -(1 << 31))):
        tokens = good.clone()
        tokens[at] = value
        got = _verify_check(p, q, tokens, _windows([3, 3, 3, 3]), au, su)
        assert got[3] == 64 and (got[0] == -77).sum() == 3
    tokens = good.clone()               # behind a rejected draft and in front of the window nothing is looked at
    tokens[2], tokens[3] = -5, V + 9
    au2 = au.clone()
    au2[0] = 1.0
    p2 = p.clone()
    p2[0, int(tokens[1])] = 0.0
    assert _verify_check(p2, q, tokens, _windows([3, 3, 3, 3]), au2, su)[3] == 0
    for cu in ([3, 0, 3, 6, 9], [0, 3, 6, 9, 13], [-1, 3, 6, 9, 12], [0, 3, 6, 9, 1 << 30], [0, 0, 6, 9, 12]):
        got = _verify_check(p, q, good, torch.tensor(cu, dtype=i32, device="cuda"), au, su)
        assert got[3] == 2 and (got[1] == -77).any()
    assert _verify_check(p, q[:7], good, _windows([3, 3, 3, 3]), au[:7], su)[3] == 2    # a row too few


def test_verify_rows_at_large_offsets():
    """Rows whose elements lie behind 2^31."""
    torch = _torch()
    d = Draw(8)
    V, T, stride = 1000, 9, 1 << 28
    dense, q = _probs(d, T, V, "f32"), _probs(d, T - 3, V, "f32")
    far = torch.empty((T - 1) * stride + V, device="cuda").as_strided((T, V), (stride, 1))
    far.copy_(dense)
    args = (d.ints(0, V, T), _windows([3, 3, 3]), d.rand(T - 3) * 0.1, d.rand(3))
    a, b = layer.verify_drafts(far, *args, draft_probs=q), layer.verify_drafts(dense, *args, draft_probs=q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def _round(d):
    """What a decoding round is made of: a function that runs it, and its outputs."""
    torch = _torch()
    hidden, wide, V, S, L = 512, 1120, 3000, 5, 3
    T = S * L
    x, res, w = d.randn(T, hidden, dtype="bf16"), d.randn(T, hidden), d.randn(hidden, dtype="bf16")
    w1, s1 = d.ints(0, 256, wide, hidden // 2, dtype="u8"), d.rand(wide, hidden // 64) * 0.02
    w2, s2 = d.ints(0, 256, V, wide // 2, dtype="u8"), d.rand(V, wide // 32) * 0.02
    z2 = d.ints(6, 10, V, wide // 32, dtype="u8")
    q, tokens, cu = _probs(d, T - S, V, "f32", scale=0.3), d.ints(0, V, T), _windows([L] * S)
    au, su, ring = d.rand(T - S), d.rand(S), torch.zeros(S, dtype=torch.int32, device="cuda")

    def run(stream=None):
        kw = {} if stream is None else {"stream": stream}
        codes, scale = layer.residual_rms_norm(x, w, residual=res, code_dtype=_t("e4m3"), scale_group=64, **kw)
        h = layer.matvec4(codes, w1, s1, group_size=64, x_scale=scale, **kw)
        logits = layer.matvec4(h, w2, s2, group_size=32, zero=z2, out_dtype=torch.float32, **kw)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            p = torch.softmax(logits, 1)
        return (*layer.verify_drafts(p, tokens, cu, au, su, draft_probs=q, ring_count=ring, **kw), logits, codes, scale)

    return run, ring


def test_a_round_captured_replayed_and_on_another_stream():
    torch = _torch()
    run, ring = _round(Draw(12))
    want = [t.clone() for t in run()]
    moved = ring.clone()
    assert torch.equal(moved, want[1] + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.synchronize()
    assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(got, want)) and torch.equal(ring, 2 * moved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(3):
        for t in held:
            t.view(torch.uint8).fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(held, want)) and torch.equal(ring, (3 + i) * moved)


def test_two_rounds_at_once():
    """Two captured rounds and an eager one at the same time on three streams: nothing is shared between calls."""
    torch = _torch()
    rounds = [_round(Draw(20 + i))[0] for i in range(3)]
    want = [[t.clone() for t in run()] for run in rounds]
    graphs, held = [], []
    for run in rounds[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(run())
    streams = [torch.cuda.Stream() for _ in rounds]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            last = rounds[2]()
    torch.cuda.synchronize()
    for got, w in zip(held + [last], want):
        assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(got, w))


def test_refused_calls_raise_and_leave_the_context_usable():
    torch = _torch()
    x = torch.randn(3, 64, device="cuda")
    p = layer.make_residual_norm_params(x, None, torch.empty_like(x))
    p.eps = -1.0
    with pytest.raises(layer.LayerError) as e:
        layer.call_residual_norm(p)
    assert e.value.code == binding.SSD_ERR_INVALID_ARG
    assert torch.isfinite(layer.residual_rms_norm(x)).all()
