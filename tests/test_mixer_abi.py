"""The C ABI of include/ssd_mixer.h without a GPU: exports, struct layouts, and
refusals, which come back before anything is enqueued."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from state_space_model_varlen_gb300 import _build, binding, mixer
from tests import mixer_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssd_mixer.h")
BAD, UNSUPPORTED = binding.SSD_ERR_INVALID_ARG, binding.SSD_ERR_UNSUPPORTED


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(ssd_\w+)\s*\(", src)))
    assert sorted(mixer.EXPORTED) == declared
    binding.load()
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LIBPATH], capture_output=True, text=True,
                         check=True).stdout
    for name in declared:
        assert re.search(r"\bT %s$" % name, out, re.M), name


@pytest.mark.parametrize("cls,cname", [(mixer.ConvParams, "ssd_conv_params"), (mixer.StepParams, "ssd_step_params"),
                                       (mixer.GatedNormParams, "ssd_gated_norm_params"),
                                       (mixer.StateParams, "ssd_state_params")])
def test_struct_layout_matches_c(tmp_path, cls, cname):
    fields = [f[0] for f in cls._fields_]
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "%s"' % HEADER, "int main(void){",
            'printf("%%zu\\n", sizeof(%s));' % cname]
    prog += ['printf("%%zu\\n", offsetof(%s, %s));' % (cname, f) for f in fields] + ["return 0;}"]
    (tmp_path / "layout.c").write_text("\n".join(prog))
    subprocess.run(["gcc", str(tmp_path / "layout.c"), "-o", str(tmp_path / "layout")], check=True)
    vals = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                           check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(cls)
    for f, off in zip(fields, vals[1:]):
        assert getattr(cls, f).offset == off, f


def _conv(**kw):
    p = mixer.ConvParams(total_tokens=10, num_seqs=2, channels=96, width=4, io_dtype=1, activation=1, split0=64,
                         split1=16, nheads=4, num_slots=3, conv_rows=4, xbc_stride=100, dt_stride=4,
                         **{k: 0x1000 for k in "xbc weight bias cu_seqlens start_pos slot_idx conv_cache out0 out1 out2 "
                                               "dt out_dt device_status".split()})
    return _set(p, kw)


def _step(**kw):
    p = mixer.StepParams(batch=2, nheads=4, headdim=16, dstate=8, ngroups=2, width=4, io_dtype=1, state_dtype=3,
                         activation=1, dt_softplus=1, num_slots=3, conv_rows=4, xbc_stride=100, z_stride=64, dt_stride=4,
                         **{k: 0x1000 for k in "xbc z dt weight bias A dt_bias D pos slot_idx conv_cache state_cache "
                                               "state_scale sr_seed out_y device_status".split()})
    return _set(p, kw)


def _norm(**kw):
    return _set(mixer.GatedNormParams(rows=3, columns=64, group_size=32, io_dtype=0, eps=1e-5, y=0x1000, y_stride=64,
                                      z=0x2000, z_stride=64, weight=0x3000, out=0x4000, out_stride=64), kw)


def _state(**kw):
    return _set(mixer.StateParams(num_states=2, nheads=4, headdim=16, dstate=8, dense_dtype=0, state_dtype=4,
                                  num_slots=3, **{k: 0x1000 for k in "states state_cache state_scale slot_idx has_init "
                                                                     "sr_seed device_status".split()}), kw)


def _set(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("make,entry,field,value,code", [
    *[(_conv, "ssd_conv_varlen", f, v, BAD) for f, v in [
        ("channels", 0), ("width", 0), ("io_dtype", 2), ("split0", -1), ("split1", 64), ("total_tokens", -1),
        ("num_seqs", -1), ("xbc_stride", 95), ("xbc", None), ("weight", None), ("cu_seqlens", None), ("out0", None),
        ("out1", None), ("out2", None), ("conv_rows", 3), ("num_slots", 0), ("slot_idx", None), ("conv_cache", None),
        ("slot_idx_stride", -1), ("out_dt", None), ("dt_stride", 3), ("xbc", 0x1001), ("out_dt", 0x1002)]],
    (_conv, "ssd_conv_varlen", "width", 9, UNSUPPORTED),
    *[(_step, "ssd_step", f, v, BAD) for f, v in [
        ("batch", -1), ("ngroups", 3), ("headdim", 0), ("io_dtype", 2), ("state_dtype", 5), ("width", 0),
        ("xbc_stride", 95), ("z_stride", 63), ("dt_stride", 3), ("conv_rows", 3), ("num_slots", 0), ("A", None),
        ("pos", None), ("slot_idx", None), ("conv_cache", None), ("state_cache", None), ("state_scale", None),
        ("out_y", None), ("weight", None), ("state_scale", 0x1002), ("sr_seed", 0x1004), ("xbc", 0x1001)]],
    (_step, "ssd_step", "dstate", 257, UNSUPPORTED), (_step, "ssd_step", "width", 9, UNSUPPORTED),
    *[(_norm, "ssd_gated_norm", f, v, BAD) for f, v in [
        ("rows", -1), ("group_size", 33), ("group_size", 0), ("io_dtype", 2), ("eps", -1.0), ("eps", float("nan")),
        ("y", None), ("out", None), ("y_stride", 63), ("z_stride", 63), ("out_stride", 63), ("y", 0x1002)]],
    *[("%s" % n, n, f, v, BAD) for n in ("ssd_state_store", "ssd_state_load") for f, v in [
        ("num_states", -1), ("dense_dtype", 2), ("state_dtype", 1), ("state_dtype", 5), ("num_slots", 0),
        ("states", None), ("state_cache", None), ("state_scale", None), ("slot_idx", None), ("states", 0x1002)]],
    ("ssd_state_store", "ssd_state_store", "dstate", 257, UNSUPPORTED),
])
def test_refused_without_launch(make, entry, field, value, code):
    p = (make if callable(make) else _state)(**{field: value})
    with pytest.raises(mixer.MixerError) as e:
        mixer._call(entry, p, 0)
    assert e.value.code == code and entry in str(e.value)


def test_empty_batches_launch_nothing():
    mixer.call_conv(_conv(num_seqs=0))
    mixer.call_conv(_conv(total_tokens=0, xbc=None))
    mixer.call_step(_step(batch=0, xbc=None))
    mixer.call_norm(_norm(rows=0, y=None))
    mixer.call_state_store(_state(num_states=0, states=None))
    mixer.call_state_load(_state(num_states=0, states=None))


def test_null_params_refused():
    for name in mixer.EXPORTED:
        assert mixer._entry(name)(None, None) == BAD


def test_binding_refuses_wrong_tensors():
    import torch
    t = torch.zeros
    xbc, w, cu = t(5, 24), t(24, 4), t(2, dtype=torch.int32)
    x, B, C = t(5, 1, 8), t(5, 1, 8), t(5, 1, 8)
    mixer.make_conv_params(xbc, w, cu, x, B, C)
    with pytest.raises(ValueError):
        mixer.make_conv_params(xbc, w, cu, x, B)                        # 16 channels for 24
    with pytest.raises(ValueError):
        mixer.make_conv_params(xbc.t().contiguous().t(), w, cu, x, B, C)  # rows not dense
    with pytest.raises(TypeError):
        mixer.make_conv_params(xbc, w.bfloat16(), cu, x, B, C)
    with pytest.raises(TypeError):
        mixer.make_conv_params(xbc, w, cu.long(), x, B, C)
    with pytest.raises(ValueError):
        mixer.make_conv_params(xbc, w, cu, x, B, C, conv_cache=t(3, 4, 24))   # no slots
    with pytest.raises(ValueError):
        mixer.make_norm_params(t(3, 8), t(7), t(3, 8))
    with pytest.raises(TypeError):
        mixer.make_norm_params(t(3, 8), t(8), t(3, 8), z=t(3, 8).bfloat16())
    i32 = torch.int32
    good = dict(ngroups=1)
    args = [t(2, 24), t(2, 1), t(24, 4), t(1), t(3, 4, 24), t(3, 1, 8, 8), t(2, dtype=i32), t(2, dtype=i32), t(2, 1, 8)]
    mixer.make_step_params(*args, **good)
    for at, bad in ((0, t(2, 23)), (1, t(3, 1)), (3, t(2)), (4, t(2, 4, 24)), (6, t(3, dtype=i32)),
                    (8, t(2, 8, 1))):
        with pytest.raises(ValueError):
            mixer.make_step_params(*(args[:at] + [bad] + args[at + 1:]), **good)
    with pytest.raises(TypeError):
        mixer.make_step_params(*args, **good, sr_seed=t(1))
    with pytest.raises(TypeError):
        mixer.make_state_params(t(2, 1, 8, 8), t(3, 1, 8, 8, dtype=torch.int16), t(3, 1, 8), t(2, dtype=i32))


def test_binding_refuses_tensors_elsewhere():
    import torch
    t = torch.zeros
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        mixer.gated_rms_norm(t(3, 8))
    with pytest.raises(ValueError, match="one device"):
        mixer.make_norm_params(t(3, 8), t(8, device="meta"), t(3, 8))
    with pytest.raises(ValueError, match="one device"):
        mixer.make_state_params(t(2, 1, 8, 8), t(3, 1, 8, 8, dtype=torch.int8), t(3, 1, 8, device="meta"), t(2, dtype=i32))
    with pytest.raises(ValueError, match="slot_idx"):
        mixer.make_state_params(t(2, 1, 8, 8), t(3, 1, 8, 8, dtype=torch.int8), t(3, 1, 8), None)


# ---- the reference's own pieces --------------------------------------------
def test_reference_e4m3_grid_is_torchs():
    import torch
    v = np.linspace(-460, 460, 4001)
    v = np.concatenate([v, v * 2.0 ** -9, v * 2.0 ** -16])
    got = torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    want = R.codes(np.clip(v, -448, 448).astype(np.float32).astype(np.float64), "e4m3")
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_reference_stochastic_rounding_is_unbiased(kind):
    """Over all 256 bytes the mean code is the value, to the resolution of the bytes."""
    rng = np.random.default_rng(0)
    v = rng.uniform(-R.LIM[kind], R.LIM[kind], 300)
    v = np.concatenate([v, v * 2.0 ** -13])
    if kind == "e4m3":
        v = (v / 256).astype(np.float16).astype(np.float64) * 256
    c = np.stack([R.codes(v, kind, np.full(v.shape, r, np.uint32)) for r in range(256)])
    unit = 1.0 if kind == "i8" else np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    assert np.all(np.abs(c.mean(0) - v) <= unit / 256 + 1e-12)
    assert np.all(np.abs(c - v) <= unit * 1.0 + 1e-12)


def test_reference_conv_is_the_plain_sum():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((7, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    out, _, _ = R.conv(x, w, b, False, [0, 2, 7], None, None, None)
    for s, e in ((0, 2), (2, 7)):
        for t in range(s, e):
            for c in range(3):
                want = b[c] + sum(w[c, 3 - k] * x[t - k, c] for k in range(4) if t - k >= s)
                assert abs(out[t, c] - want) < 1e-12
