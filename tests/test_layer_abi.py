"""The C ABI of include/ssd_layer.h without a GPU: exports, struct layouts,
refusals, which come back before anything is enqueued, and the device and stream
of every call."""
import contextlib
import ctypes
import os
import re
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from state_space_model_varlen_gb300 import _build, binding, layer, mixer
from tests import layer_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssd_layer.h")
BAD, UNSUPPORTED = binding.SSD_ERR_INVALID_ARG, binding.SSD_ERR_UNSUPPORTED
BLOCKS = {"ssd_residual_norm": (layer.ResidualNormParams, "ssd_residual_norm_params", layer.call_residual_norm),
          "ssd_matvec4": (layer.Matvec4Params, "ssd_matvec4_params", layer.call_matvec4),
          "ssd_verify_drafts": (layer.VerifyParams, "ssd_verify_params", layer.call_verify)}
F32, BF16, F16, E4M3, I8 = 0, 1, 2, 3, 4


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(ssd_\w+)\s*\(", src)))
    assert sorted(layer.EXPORTED) == declared == sorted(BLOCKS)
    binding.load()
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LIBPATH], capture_output=True, text=True,
                         check=True).stdout
    for name in declared:
        assert re.search(r"\bT %s$" % name, out, re.M), name


@pytest.mark.parametrize("name", sorted(BLOCKS))
def test_struct_layout_matches_c(tmp_path, name):
    cls, cname, _ = BLOCKS[name]
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


def _set(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _norm(**kw):
    return _set(layer.ResidualNormParams(
        rows=3, columns=64, io_dtype=BF16, residual_dtype=F32, code_dtype=E4M3, scale_group=32, eps=1e-5, x=0x1000,
        x_stride=64, residual=0x2000, residual_stride=64, weight=0x3000, residual_out=0x4000, residual_out_stride=64,
        out=0x5000, out_stride=64, out_codes=0x6000, codes_stride=64, out_scale=0x7000), kw)


def _mv(**kw):
    return _set(layer.Matvec4Params(
        rows=2, in_features=64, out_features=16, group_size=32, x_dtype=E4M3, x_group=64, scale_dtype=BF16, out_dtype=BF16,
        x=0x1000, x_stride=64, x_scale=0x2000, weight=0x3000, weight_stride=32, scale=0x4000, zero=0x5000, bias=0x6000,
        out=0x7000, out_stride=16), kw)


def _verify(**kw):
    return _set(layer.VerifyParams(
        total_tokens=6, num_drafts=4, num_seqs=2, vocab=50, prob_dtype=F32, target_probs=0x1000, target_stride=50,
        draft_probs=0x2000, draft_stride=50, tokens=0x3000, cu_seqlens=0x4000, accept_u=0x5000, sample_u=0x6000,
        out_tokens=0x7000, out_accepted=0x8000, ring_count=0x9000, device_status=0xa000), kw)


@pytest.mark.parametrize("make,entry,change,code", [
    *[(_norm, "ssd_residual_norm", c, BAD) for c in [
        dict(rows=-1), dict(columns=0), dict(io_dtype=F16), dict(residual_dtype=F16), dict(code_dtype=F32),
        dict(code_dtype=5), dict(scale_group=0), dict(scale_group=33), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
        dict(x=0x1001), dict(x_stride=63), dict(residual=0x2002), dict(residual_stride=63), dict(weight=0x3001),
        dict(residual_out=0x4002), dict(residual_out_stride=63), dict(out=0x5001), dict(out_stride=63),
        dict(out=None, out_codes=None), dict(out_scale=None), dict(out_scale=0x7002), dict(codes_stride=63),
        dict(out=0x1000, out_stride=65), dict(residual_out=0x2000, residual_out_stride=65), dict(out=0x4000),
        dict(out=0x2000), dict(residual_out=0x1000),
        dict(residual_dtype=BF16, residual_out=0x1000, residual_out_stride=65)]],
    (_norm, "ssd_residual_norm", dict(columns=(1 << 20) + 32, x_stride=1 << 21), UNSUPPORTED),
    *[(_mv, "ssd_matvec4", c, BAD) for c in [
        dict(rows=-1), dict(in_features=0), dict(out_features=-1), dict(group_size=0), dict(x_dtype=F16), dict(x_dtype=5),
        dict(x_group=0), dict(scale_dtype=E4M3), dict(out_dtype=F16), dict(x=None), dict(x_stride=63), dict(x_scale=None),
        dict(x_scale=0x2002), dict(weight=None), dict(weight_stride=31), dict(scale=None), dict(scale=0x4001),
        dict(bias=0x6001), dict(out=None), dict(out=0x7001), dict(out_stride=15), dict(x_dtype=F32, x=0x1002)]],
    (_mv, "ssd_matvec4", dict(out_features=(1 << 30) + 1), UNSUPPORTED),
    (_mv, "ssd_matvec4", dict(in_features=(1 << 30) + 1), UNSUPPORTED),
    *[(_verify, "ssd_verify_drafts", c, BAD) for c in [
        dict(total_tokens=-1), dict(num_drafts=-1), dict(num_seqs=-1), dict(vocab=0), dict(prob_dtype=F16),
        dict(target_probs=None), dict(target_probs=0x1002), dict(target_stride=49), dict(draft_stride=49),
        dict(draft_probs=0x2002), dict(tokens=None), dict(cu_seqlens=None), dict(accept_u=None), dict(accept_u=0x5002),
        dict(sample_u=None), dict(out_tokens=None), dict(out_tokens=0x3000), dict(out_accepted=None),
        dict(ring_count=0x9002), dict(device_status=0xa002)]],
    (_verify, "ssd_verify_drafts", dict(vocab=(1 << 30) + 1), UNSUPPORTED),
])
def test_refused_without_launch(make, entry, change, code):
    with pytest.raises(layer.LayerError) as e:
        mixer._call(entry, make(**change), 0)
    assert e.value.code == code and entry in str(e.value)


def test_empty_calls_launch_nothing():
    layer.call_residual_norm(_norm(rows=0, x=None))
    layer.call_matvec4(_mv(rows=0, x=None))
    layer.call_matvec4(_mv(out_features=0, weight=None))
    layer.call_verify(_verify(num_seqs=0, tokens=None))
    layer.call_verify(_verify(total_tokens=0, tokens=None))


def test_null_params_refused():
    for name in layer.EXPORTED:
        assert mixer._entry(name)(None, None) == BAD


def _t(*shape, dtype=torch.float32, device="cpu"):
    return torch.zeros(*shape, dtype=dtype, device=device)


I32, U8, FP8, BF = torch.int32, torch.uint8, torch.float8_e4m3fn, torch.bfloat16


def test_norm_binding_refuses_wrong_tensors():
    x = _t(3, 8)
    layer.make_residual_norm_params(x, _t(8), x, residual=_t(3, 8, dtype=BF), residual_out=_t(3, 8, dtype=BF))
    good = dict(codes=_t(3, 8, dtype=FP8), scale=_t(3, 2))
    assert layer.make_residual_norm_params(x, **good).scale_group == 4
    for error, args, kw in [
            (ValueError, (x, _t(7), _t(3, 8)), {}), (TypeError, (x, _t(8, dtype=BF), _t(3, 8)), {}),
            (TypeError, (x, None, _t(3, 8, dtype=BF)), {}), (ValueError, (x, None, _t(2, 8)), {}),
            (ValueError, (x, None, _t(3, 8)), dict(residual=_t(2, 8))), (ValueError, (x, None, _t(3, 8)), dict(residual=_t(3, 7))),
            (TypeError, (x, None, _t(3, 8)), dict(residual=_t(3, 8, dtype=torch.float16))),
            (TypeError, (x, None, _t(3, 8)), dict(residual=_t(3, 8), residual_out=_t(3, 8, dtype=BF))),
            (ValueError, (x,), dict(codes=good["codes"])), (TypeError, (x,), dict(codes=_t(3, 8, dtype=U8), scale=_t(3, 2))),
            (ValueError, (x,), dict(codes=good["codes"], scale=_t(3, 3))),
            (ValueError, (x,), dict(codes=good["codes"], scale=_t(2, 2))),
            (TypeError, (x.half(), None, x.half()), {}), (ValueError, (x.t().contiguous().t(), None, _t(3, 8)), {})]:
        with pytest.raises(error):
            layer.make_residual_norm_params(*args, **kw)
    for kw in (dict(scale_group=4), dict(code_dtype=FP8, scale_group=3), dict(code_dtype=FP8, scale_group=0)):
        with pytest.raises(ValueError):
            layer.residual_rms_norm(x, **kw)


def test_matvec_binding_refuses_wrong_tensors():
    x, w, s, out = _t(3, 10), _t(4, 5, dtype=U8), _t(4, 3), _t(3, 4)
    layer.make_matvec4_params(x, w, s, out, group_size=4, zero=_t(4, 3, dtype=U8), bias=_t(4))
    p = layer.make_matvec4_params(x.to(FP8), w, s, out, group_size=4, x_scale=_t(3, 5))
    assert p.x_group == 2
    for error, args, kw in [
            (ValueError, (x, _t(4, 6, dtype=U8), s, out), {}), (TypeError, (x, _t(4, 5, dtype=torch.int8), s, out), {}),
            (ValueError, (x, w, _t(4, 2), out), {}), (TypeError, (x, w, _t(4, 3, dtype=torch.float64), out), {}),
            (ValueError, (x, w, s, _t(3, 5)), {}), (TypeError, (x, w, s, out.half()), {}),
            (TypeError, (x.half(), w, s, out), {}), (ValueError, (x, w, s, out), dict(zero=_t(4, 2, dtype=U8))),
            (TypeError, (x, w, s, out), dict(zero=_t(4, 3, dtype=I32))), (TypeError, (x, w, s, out), dict(bias=_t(4, dtype=BF))),
            (ValueError, (x, w, s, out), dict(bias=_t(5))), (ValueError, (x, w, s, out), dict(x_scale=_t(3, 5))),
            (ValueError, (x.to(FP8), w, s, out), {}), (ValueError, (x.to(FP8), w, s, out), dict(x_scale=_t(3, 4))),
            (ValueError, (x.to(FP8), w, s, out), dict(x_scale=_t(2, 5))), (ValueError, (x, w, s, out), dict(group_size=0))]:
        with pytest.raises(error):
            layer.make_matvec4_params(*args, **{"group_size": 4, **kw})


def test_verify_binding_refuses_wrong_tensors():
    args = [_t(5, 7), _t(5, dtype=I32), _t(3, dtype=I32), _t(3), _t(2), _t(5, dtype=I32), _t(2, dtype=I32)]
    p = layer.make_verify_params(*args, draft_probs=_t(3, 7), ring_count=_t(2, dtype=I32))
    assert (p.total_tokens, p.num_drafts, p.num_seqs, p.vocab) == (5, 3, 2, 7)
    layer.make_verify_params(*args[:3], None, *args[4:])
    for at, bad, error in [(0, _t(4, 7), ValueError), (0, _t(5, 7).double(), TypeError), (1, _t(5), TypeError),
                           (2, _t(3).long(), TypeError), (3, _t(3, dtype=I32), TypeError), (4, _t(3), ValueError),
                           (5, _t(4, dtype=I32), ValueError), (6, _t(2), TypeError)]:
        with pytest.raises(error):
            layer.make_verify_params(*(args[:at] + [bad] + args[at + 1:]))
    for kw, error in [(dict(draft_probs=_t(4, 7)), ValueError), (dict(draft_probs=_t(3, 7, dtype=BF)), TypeError),
                      (dict(ring_count=_t(3, dtype=I32)), ValueError), (dict(ring_count=_t(2)), TypeError)]:
        with pytest.raises(error):
            layer.make_verify_params(*args, **kw)


def _blocks(device):
    def t(*shape, dtype=torch.float32):
        return _t(*shape, dtype=dtype, device=device)
    return {"ssd_residual_norm": layer.make_residual_norm_params(t(3, 8), t(8), t(3, 8)),
            "ssd_matvec4": layer.make_matvec4_params(t(3, 8), t(4, 4, dtype=U8), t(4, 1), t(3, 4), group_size=8),
            "ssd_verify_drafts": layer.make_verify_params(t(5, 7), t(5, dtype=I32), t(3, dtype=I32), t(3), t(2),
                                                          t(5, dtype=I32), t(2, dtype=I32))}


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_tensors_that_are_not_on_a_gpu_are_refused(device):
    for name, p in _blocks(device).items():
        assert p.device == torch.device(device)
        with pytest.raises(ValueError, match="CUDA"):
            BLOCKS[name][2](p)
    with pytest.raises(ValueError, match="one device"):
        layer.make_residual_norm_params(_t(3, 8), _t(8, device="meta"), _t(3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        layer.matvec4(_t(3, 8), _t(4, 4, dtype=U8), _t(4, 1), group_size=8)
    with pytest.raises(ValueError, match="CUDA"):
        layer.residual_rms_norm(_t(3, 8), code_dtype=FP8, scale_group=4)
    with pytest.raises(ValueError, match="CUDA"):
        layer.verify_drafts(_t(5, 7), _t(5, dtype=I32), _t(3, dtype=I32), _t(3), _t(2))


@pytest.mark.parametrize("name", sorted(BLOCKS))
@pytest.mark.parametrize("stream", [0, 0x5000])
def test_call_launches_on_the_device_of_its_tensors(monkeypatch, name, stream):
    state = SimpleNamespace(current=0, launches=[])

    @contextlib.contextmanager
    def device(d):
        before, state.current = state.current, torch.device(d).index
        yield
        state.current = before

    def entry(params, at):
        state.launches.append((state.current, at))
        return binding.SSD_OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setitem(mixer._entries, name, entry)
    p = BLOCKS[name][0]()
    for index in (1, 0, 2):
        p.device = torch.device("cuda", index)
        BLOCKS[name][2](p, stream)
        assert state.launches[-1] == (index, stream or None) and state.current == 0


# ---- the reference's own pieces --------------------------------------------
def test_reference_codes_are_in_the_order_of_the_columns():
    w = np.array([[0x21, 0x43, 0x65]], dtype=np.uint8)
    np.testing.assert_array_equal(R.unpacked(w, 5), [[1, 2, 3, 4, 5]])
    out, _ = R.matvec4(np.ones((1, 5)), w, np.array([[2.0, 10.0, 100.0]]), np.array([[0, 1, 2]], dtype=np.uint8),
                       np.array([0.5]), 2)
    assert out[0, 0] == 0.5 + 2 * (1 + 2) + 10 * (2 + 3) + 100 * 3


def test_reference_verification_keeps_the_targets_distribution():
    """Over a fine grid of random numbers the first new token of a one-draft window is distributed as the target says."""
    p, q = np.array([0.1, 0.5, 0.25, 0.15]), np.array([0.4, 0.3, 0.25, 0.05])
    grid = (np.arange(100) + 0.5) / 100
    mass = np.zeros(4)
    for d in range(4):
        for u in grid:
            for v in grid:
                out, acc, _, status = R.verify(np.stack([p, p]), q[None], np.array([0, d]), [0, 2], [u], [v], None,
                                               np.zeros(2, int), np.zeros(1, int))
                assert status == 0
                mass[out[0]] += q[d] / len(grid) ** 2
    np.testing.assert_allclose(mass, p, atol=0.011)


# ---- sizes that a 32-bit field does not hold ---------------------------------
WIDE = 1 << 32


def test_a_group_longer_than_32_bits_is_one_group_of_the_row():
    """A wrapped size of 32 would read a scale for every 32 columns where there is one."""
    x, w, s, out = _t(3, 64), _t(4, 32, dtype=U8), _t(4, 1), _t(3, 4)
    for group in (WIDE + 32, WIDE, (1 << 31) + 32, 1 << 31, (1 << 31) - 1, 1 << 30, 64):
        p = layer.make_matvec4_params(x, w, s, out, group_size=group)
        assert p.in_features == 64 and p.group_size >= 64
    for group in (0, -1, -WIDE + 32):
        with pytest.raises(ValueError):
            layer.make_matvec4_params(x, w, s, out, group_size=group)


@pytest.mark.parametrize("more", [0, 64, 1 << 31, WIDE + 64])
def test_sizes_past_32_bits_do_not_wrap_into_small_ones(more):
    """They stay sizes that the library refuses."""
    def t(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")
    n = WIDE + more
    p = layer.make_residual_norm_params(t(1, n), t(n), t(1, n))
    assert p.columns > 1 << 20
    p = layer.make_residual_norm_params(t(1, n), t(n), None, codes=t(1, n, dtype=FP8), scale=t(1, 1))
    assert p.columns > 1 << 20
    p = layer.make_matvec4_params(t(1, n), t(4, n // 2, dtype=U8), t(4, 1), t(1, 4), group_size=n)
    assert p.in_features > 1 << 30
    p = layer.make_matvec4_params(t(1, 64), t(n, 32, dtype=U8), t(n, 1), t(1, n), group_size=64)
    assert p.out_features > 1 << 30
    p = layer.make_matvec4_params(t(n, 64), t(4, 32, dtype=U8), t(4, 1), t(n, 4), group_size=64)
    assert p.rows >= 1 << 30
    for x_dtype, parts in ((F32, 3), (BF16, 1), (E4M3, 1)):     # refused before anything is enqueued
        with pytest.raises(layer.LayerError) as e:
            mixer._call("ssd_matvec4", _mv(rows=p.rows, x_dtype=x_dtype), 0)
        assert e.value.code == UNSUPPORTED
    args = [t(5, n), t(5, dtype=I32), t(3, dtype=I32), t(3), t(2), t(5, dtype=I32), t(2, dtype=I32)]
    assert layer.make_verify_params(*args).vocab > 1 << 30
    args = [t(5, 7), t(5, dtype=I32), t(n + 1, dtype=I32), t(3), t(n), t(5, dtype=I32), t(n, dtype=I32)]
    p = layer.make_verify_params(*args)
    with pytest.raises(layer.LayerError) as e:
        mixer._call("ssd_verify_drafts", _verify(num_seqs=p.num_seqs), 0)
    assert e.value.code == UNSUPPORTED
