"""What the mixer operators leave alone: tokens, requests and slots that are not
theirs, or whose metadata is faulty."""
import numpy as np
import pytest

from state_space_model_varlen_gb300 import binding, mixer
from tests import mixer_reference as R
from tests.test_mixer_gpu import _conv_case, _conv_run, _i32, _np, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [3, 130])
@pytest.mark.parametrize("lens", [[40, 40, 40], [3, 70, 5, 1, 9, 2], [1] * 90, [300, 2, 200], [0, 40, 0, 33, 0, 0, 25]])
@pytest.mark.parametrize("what", ["padding", "slot", "start", "end"])
def test_conv_writes_nothing_for_tokens_of_no_valid_sequence(lens, what, heads, io):
    """x, B, C and dt rows before and after the batch's sequences, and those of a faulty one, stay as they were."""
    torch = _torch()
    lead, tail, S = 5, 11, len(lens)
    bad = S // 2
    c = _conv_case([lead] + lens + [tail], 64, 16, 4, io, seed=S, heads=heads)
    c["cu"] = lead + np.concatenate([[0], np.cumsum(lens)])
    c["slot"], c["ring"] = c["slot"][:S].clone(), c["ring"][:S + 2]
    c["slot"].copy_(_i32(range(S)))
    c["start"] = _i32([9] * S)
    good = list(range(S)) if what == "padding" else [s for s in range(S) if s != bad]
    flag = 0
    if what == "slot":
        c["slot"][bad], flag = S + 2, binding.SSD_DEV_BAD_SLOT
    elif what == "start":
        c["start"][bad], flag = -1, mixer.SSD_DEV_BAD_POS
    elif what == "end":                                 # the last sequence runs past the batch
        good, flag = list(range(S - 1)), binding.SSD_DEV_BAD_SEQLENS
        c["cu"][S] = sum(lens) + lead + tail + 1
    keep, st = _conv_run(c)
    assert st == flag
    first = lead + np.concatenate([[0], np.cumsum(lens)])
    mine = np.zeros(lead + sum(lens) + tail, dtype=bool)
    for s in good:
        mine[first[s]:first[s + 1]] = True
    want, err, _ = R.conv(_np(c["xbc"]), _np(c["w"]), _np(c["bias"]), True, first, [9] * S, list(range(S)), _np(keep))
    got = _np(torch.cat(c["out"], 1))
    R.check(got[mine], want[mine], err[mine], io, "convolution")
    assert np.isnan(got[~mine]).all()
    dt = _np(c["out_dt"])
    np.testing.assert_array_equal(dt[mine], _np(c["dt"])[mine])
    assert np.isnan(dt[~mine]).all()
    for q in set(range(S + 2)) - set(good):
        assert torch.equal(c["ring"][q], keep[q])
