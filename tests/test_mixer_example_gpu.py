"""The mixer example: prompts, a continued prompt and decoded tokens on one set
of caches, against the same tokens as longer prompts."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mamba2_mixer.py")


def _example():
    spec = importlib.util.spec_from_file_location("mamba2_mixer_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("state,tol", [("f32", 0.02), ("bf16", 0.03), ("i8", 0.06), ("e4m3", 0.15)])
def test_example(state, tol):
    """tol: bf16 activations through four kernels and a norm (2^-8 each, and the norm's division by a small rms),
    and the stored type's rounding at each rewrite (bf16 2^-9, int8 0.4 %, e4m3 2.7 % of a row's rms), the rewrites'
    errors adding up over about ten steps of decay."""
    m = _example()
    assert m.run(state, tokens=12) <= tol
    assert m.run(state, tokens=4, nheads=6, headdim=32, dstate=64, ngroups=2, hidden=256, lens=(40, 3, 300)) <= tol
