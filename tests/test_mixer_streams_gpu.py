"""Calls with ``stream=``: memory that the current stream still reads is not
handed to a kernel of another stream."""
import pytest

from state_space_model_varlen_gb300 import mixer

pytestmark = pytest.mark.gpu


def test_output_on_another_stream_leaves_memory_in_use_alone():
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    rows, cols = 4096, 8192
    busy = torch.randn(4096, 4096, generator=g, device="cuda")
    y = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    plain = mixer.gated_rms_norm(y)
    x, seen = y.clone(), torch.empty_like(y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        busy @ busy                                     # the current stream reads x only after these
    seen.copy_(x)
    del x
    out = mixer.gated_rms_norm(y, stream=side)          # the same size as x
    torch.cuda.synchronize()
    assert torch.equal(seen, y) and torch.equal(out, plain)


def test_output_of_another_stream_is_the_callers_to_read_and_free():
    import torch
    y = torch.randn(4096, 8192, device="cuda", dtype=torch.bfloat16)
    busy = torch.randn(4096, 4096, device="cuda")
    minus, want = -y, mixer.gated_rms_norm(y)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    out = mixer.gated_rms_norm(y, stream=side)
    here.wait_stream(side)
    for _ in range(20):
        busy @ busy
    seen = out + 0
    del out
    other = mixer.gated_rms_norm(minus, stream=side)    # may not take the place of what is still read
    torch.cuda.synchronize()
    assert torch.equal(seen, want) and torch.equal(other, -want)
