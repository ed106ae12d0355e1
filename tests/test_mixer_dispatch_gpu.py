"""Every kernel variant that the mixer operators' dispatch selects: widths,
vector lengths, row strides and mean lengths of the convolution, state sizes and
roundings of the step, long norm groups of odd sizes."""
import numpy as np
import pytest

from state_space_model_varlen_gb300 import mixer
from tests import mixer_reference as R
from tests.test_mixer_gpu import (KINDS, Draw, _conv_case, _conv_check, _conv_run, _np, _step_case, _step_check,
                                  _step_run, _t, _torch)

pytestmark = pytest.mark.gpu

BRIEF, LONG = [3, 70, 5, 1, 9, 2, 40], [300, 2, 200]    # mean lengths below and above 64


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [BRIEF, LONG])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("C0,C1", [(64, 16), (62, 14), (61, 7), (1024, 128)])     # multiples of 4, of 2, odd; several CTAs
@pytest.mark.parametrize("pad", [0, 2, 3, 4, 5, 8])     # row strides and bases of each alignment
def test_conv_of_every_width_stride_and_length(lens, W, C0, C1, pad, io):
    c = _conv_case(lens, C0, C1, W, io, seed=W + pad, pad=pad, start=lambda s: 5 * s)
    keep, st = _conv_run(c)
    assert st == 0
    _conv_check(c, keep, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_conv_infinity_shows_in_its_window(io):
    """An infinite input of a channel with positive weights makes the outputs of its window infinite, and no others."""
    c = _conv_case([50], 64, 16, 4, io, seed=8)
    c["xbc"][30, 70] = float("inf")
    c["w"][70] = c["w"][70].abs() + 0.125
    _conv_run(c)
    got = np.concatenate([_np(o) for o in c["out"]], 1)
    assert np.isposinf(got[30:34, 70]).all()
    got[30:34, 70] = 0.0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("channels", [64, 63])           # pairs and single values
def test_silu_keeps_its_stated_error(channels):
    """A convolution of width 1 with weight 1 is SiLU alone: relative error below 2^-20 + |v| 2^-23 down to -87, zero or
    as exact below, and the limits at the infinities' side."""
    torch = _torch()
    v = torch.cat([torch.linspace(-87, 87, 63 * 64 * 40), torch.linspace(-1e-3, 1e-3, 63 * 64)]).cuda().view(-1, channels)
    far = torch.tensor([-88.0, -100.0, -1e4, -3e38, 100.0, 3e38, 0.0, -0.0], device="cuda")[:, None].expand(8, channels)
    x = torch.cat([v, far])
    one = torch.ones(channels, 1, device="cuda")
    out = torch.full_like(x, float("nan"))
    cu = torch.tensor([0, x.shape[0]], dtype=torch.int32, device="cuda")
    mixer.call_conv(mixer.make_conv_params(x, one, cu, out), torch.cuda.current_stream().cuda_stream)
    got, a = _np(out), _np(x)
    want = a * R.sigmoid(a)
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -20 + np.abs(a) * 2.0 ** -23) + 2.0 ** -119)
    near = np.abs(a) <= 87
    assert np.all(np.abs(got - want)[near] <= (np.abs(want) * (2.0 ** -20 + np.abs(a) * 2.0 ** -23))[near])


@pytest.mark.parametrize("kind,sr", [(k, None) for k in KINDS] + [("f16", 5), ("e4m3", 5), ("i8", 5)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,P,N,G,W,pad", [
    (5, 4, 64, 128, 2, 2, 0), (5, 4, 64, 128, 2, 3, 0),         # four channels at a time, widths 2 and 3
    (6, 4, 20, 24, 2, 3, 8), (4, 2, 16, 32, 1, 4, 0), (4, 2, 9, 17, 1, 4, 1),   # 17 to 32 values a row
    (3, 2, 12, 64, 1, 2, 0), (3, 1, 33, 256, 1, 3, 2),
])
def test_step_of_every_width_and_state_size(B, H, P, N, G, W, pad, io, kind, sr):
    c = _step_case(B, H, P, N, G, W, io, kind, seed=13, pad=pad, sr=sr and 0x7654_3210_0FED_CBA9, gate=pad == 0)
    before, st = _step_run(c)
    assert st == 0
    _step_check(c, before)


@pytest.mark.parametrize("kind", ["f32", "e4m3"])
@pytest.mark.parametrize("field,value", [("slot", 99), ("slot", -2), ("pos", -1)])
def test_step_next_to_a_bad_request_is_right(kind, field, value):
    """The other requests of a batch with a faulty one have the reference's outputs and states."""
    c = _step_case(8, 4, 40, 64, 2, 4, "bf16", kind, seed=3, zero_pos=False)
    c[field][3] = value
    before, st = _step_run(c)
    assert st != 0 and bool(_torch().isnan(c["y"][3].float()).all())
    c["slot"][3], c["y"][3] = -1, 0.0                   # to the reference a padding row
    _step_check(c, before)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["before", "after", "none"])
@pytest.mark.parametrize("rows,cols,group", [
    (3, 1025, 1025), (2, 8193, 8193), (2, 10241, 10241), (2, 2051, 293),           # single elements
    (3, 5124, 5124), (2, 12300, 12300), (2, 20004, 20004), (3, 1608, 804), (2, 70000, 70000)])    # four at a time; long
def test_norm_of_long_groups(rows, cols, group, gate, io):
    d = Draw(rows + cols)
    y, w = d.columns(rows, cols, io, 8 if cols % 8 == 0 else 0), d.randn(cols, dtype=io)
    z = None if gate == "none" else d.columns(rows, cols, io, 16)
    out = _torch().full((rows, cols + 8), 7.0, dtype=_t(io), device="cuda")
    mixer.gated_rms_norm(y, w, z=z, group_size=group, eps=1e-5, norm_before_gate=gate == "after", out=out[:, :cols])
    want, err = R.norm(_np(y), None if z is None else _np(z), _np(w), group, 1e-5, gate == "after")
    R.check(_np(out[:, :cols]), want, err, io, "norm")
    assert bool((out[:, cols:] == 7.0).all())
