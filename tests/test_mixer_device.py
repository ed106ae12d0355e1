"""On which device and stream the calls of the binding and of the mixer operators
run, without a GPU: the library and torch's current device are stand-ins that record what they are
given."""
import contextlib
import weakref
from types import SimpleNamespace

import pytest
import torch

from state_space_model_varlen_gb300 import binding, mixer

ENTRIES = {"ssd_conv_varlen": (mixer.ConvParams, mixer.call_conv), "ssd_step": (mixer.StepParams, mixer.call_step),
           "ssd_gated_norm": (mixer.GatedNormParams, mixer.call_norm),
           "ssd_state_store": (mixer.StateParams, mixer.call_state_store),
           "ssd_state_load": (mixer.StateParams, mixer.call_state_load)}


class Fake:
    """A machine with several GPUs: the current one, and the (device, stream) of every launch."""

    def __init__(self, monkeypatch, code=binding.SSD_OK):
        self.current, self.launches, self.code = 0, [], code
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.device)

    @contextlib.contextmanager
    def device(self, device):
        before, self.current = self.current, torch.device(device).index
        try:
            yield
        finally:
            self.current = before

    def entry(self, params, stream):
        self.launches.append((self.current, stream))
        return self.code


@pytest.mark.parametrize("name", sorted(ENTRIES))
@pytest.mark.parametrize("stream", [0, 0x5000])
def test_call_launches_on_the_device_of_its_tensors(monkeypatch, name, stream):
    fake = Fake(monkeypatch)
    monkeypatch.setitem(mixer._entries, name, fake.entry)
    cls, call = ENTRIES[name]
    p = cls()
    for index in (1, 0, 2):
        p.device = torch.device("cuda", index)
        call(p, stream)
        assert fake.launches[-1] == (index, stream or None) and fake.current == 0


def test_device_is_put_back_after_a_refusal(monkeypatch):
    fake = Fake(monkeypatch, binding.SSD_ERR_INVALID_ARG)
    monkeypatch.setitem(mixer._entries, "ssd_gated_norm", fake.entry)
    p = mixer.GatedNormParams()
    p.device = torch.device("cuda", 1)
    with pytest.raises(mixer.MixerError):
        mixer.call_norm(p)
    assert fake.launches == [(1, None)] and fake.current == 0


def _blocks(device):
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)
    i32 = torch.int32
    states = (t(2, 1, 8, 8), t(3, 1, 8, 8, dtype=torch.int8), t(3, 1, 8), t(2, dtype=i32))
    return [
        (mixer.make_conv_params(t(5, 24), t(24, 4), t(2, dtype=i32), t(5, 1, 8), t(5, 1, 8), t(5, 1, 8)), mixer.call_conv),
        (mixer.make_step_params(t(2, 24), t(2, 1), t(24, 4), t(1), t(3, 4, 24), t(3, 1, 8, 8), t(2, dtype=i32),
                                t(2, dtype=i32), t(2, 1, 8), ngroups=1), mixer.call_step),
        (mixer.make_norm_params(t(3, 8), t(8), t(3, 8)), mixer.call_norm),
        (mixer.make_state_params(*states), mixer.call_state_store),
        (mixer.make_state_params(*states), mixer.call_state_load)]


def test_blocks_know_their_device_and_those_of_cpu_tensors_are_refused(monkeypatch):
    for device in ("cpu", "meta"):
        for p, call in _blocks(device):
            assert p.device == torch.device(device)
            with pytest.raises(ValueError, match="CUDA"):
                call(p)


def test_a_block_keeps_its_tensors():
    """The addresses in a kept block stay those of its tensors, also of ones that the caller has let go."""
    tensors = [torch.zeros(3, 8), torch.zeros(8), torch.zeros(3, 8), torch.zeros(3, 8)]
    p = mixer.make_norm_params(*tensors[:3], z=tensors[3])
    held = [weakref.ref(t) for t in tensors]
    del tensors
    assert [r().data_ptr() for r in held] == [p.y, p.weight, p.out, p.z]
    del p
    assert not any(r() for r in held)
    has = torch.ones(2, dtype=torch.bool)
    p = mixer.make_state_params(torch.zeros(2, 1, 8, 8), torch.zeros(3, 1, 8, 8, dtype=torch.int8), torch.zeros(3, 1, 8),
                                torch.zeros(2, dtype=torch.int32), has_init=has)
    has = weakref.ref(has)
    assert has().data_ptr() == p.has_init


def test_a_stream_of_another_device_is_refused():
    class Tensor:
        is_cuda, device = True, torch.device("cuda", 1)

    class Stream:
        cuda_stream = 0x7000

        def __init__(self, index):
            self.device = torch.device("cuda", index)

    assert mixer._stream(Tensor, Stream(1)) == 0x7000
    with pytest.raises(ValueError, match="stream"):
        mixer._stream(Tensor, Stream(0))


@pytest.mark.parametrize("name,call,cls", [("ssd_scan_varlen", binding.call, binding.ScanParams),
                                           ("ssd_scan_varlen_noalloc", binding.call_noalloc, binding.ScanParams),
                                           ("ssd_replay_mtp", binding.call_replay, binding.ReplayParams)])
@pytest.mark.parametrize("stream", [0, 0x5000])
def test_scan_launches_on_the_device_of_its_tensors(monkeypatch, name, call, cls, stream):
    fake = Fake(monkeypatch)

    class Library:
        pass

    setattr(Library, name, staticmethod(fake.entry))
    monkeypatch.setattr(binding, "load", lambda: Library)
    p = cls()
    for index in (1, 0, 2):
        p.device = torch.device("cuda", index)
        call(p, stream)
        assert fake.launches[-1] == (index, stream or None) and fake.current == 0


def test_scan_blocks_know_their_device():
    for device in ("cpu", "meta"):
        def t(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device=device)
        cu = t(2, dtype=torch.int32)
        p = binding.make_params(t(5, 1, 8), t(5, 1), t(1), t(5, 1, 8), t(5, 1, 8), cu, out_y=t(5, 1, 8))
        one = t(1, dtype=torch.int32)
        r = binding.make_replay_params(p, t(1, 4, 1, 8), t(1, 4, 1), t(1, 4, 1, 8), 4, one, one, one, one)
        for block, call in ((p, binding.call), (p, binding.call_noalloc), (r, binding.call_replay)):
            assert block.device == torch.device(device)
            with pytest.raises(ValueError, match="CUDA"):
                call(block)


class Memory:
    """Stand-ins for torch's streams and allocator: what is allocated, on which stream, and for whose use."""

    def __init__(self, monkeypatch):
        self.current, self.made = "here", []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stream("here"))
        monkeypatch.setattr(torch.cuda, "stream", self.switch)
        for name in ("empty", "empty_like"):
            monkeypatch.setattr(torch, name, self.make)
        for module, names in ((mixer, ("make_conv_params", "make_step_params", "make_norm_params", "make_state_params",
                                       "call_conv", "call_step", "call_norm", "call_state_load")),
                              (binding, ("make_params", "call"))):
            for name in names:
                monkeypatch.setattr(module, name, lambda *args, **options: SimpleNamespace())
        monkeypatch.setattr(binding, "workspace_size", lambda params: 256)

    def stream(self, name):
        return SimpleNamespace(name=name, cuda_stream=1, device=torch.device("cuda", 0))

    @contextlib.contextmanager
    def switch(self, stream):
        before, self.current = self.current, stream.name
        yield
        self.current = before

    def make(self, *args, **options):
        t = SimpleNamespace(stream=self.current, users=[self.current], data_ptr=lambda: 0x1000)
        t.record_stream = lambda stream: t.users.append(stream.name)
        self.made.append(t)
        return t


def test_outputs_belong_to_the_stream_that_writes_them(monkeypatch):
    """Memory of the current stream may still be read there when a kernel of another stream writes it: what a call
    with stream= allocates comes from that stream, and the current one may free it."""
    def tensor(*shape):
        return SimpleNamespace(shape=shape, dtype=torch.float32, device=torch.device("cuda", 0), is_cuda=True)

    memory = Memory(monkeypatch)
    x = tensor(5, 1, 8)
    for run, count in (
            (lambda **k: mixer.conv_varlen(tensor(5, 24), None, None, nheads=1, headdim=8, ngroups=1, dstate=8,
                                           dt=tensor(5, 1), **k), 4),
            (lambda **k: mixer.step(tensor(5, 24), None, None, None, None, tensor(3, 1, 8, 8), None, None, ngroups=1,
                                    **k), 1),
            (lambda **k: mixer.gated_rms_norm(tensor(5, 8), **k), 1),
            (lambda **k: mixer.state_load(tensor(3, 1, 8, 8), None, tensor(2), **k), 1),
            (lambda **k: binding.ssd_scan_varlen(x, None, None, None, None, None, **k), 2)):
        for name in ("side", "here"):
            memory.made.clear()
            monkeypatch.setattr(mixer, "_stream", lambda t, stream: 1)
            run(**({} if name == "here" else {"stream": memory.stream(name)}))
            assert [t.stream for t in memory.made] == [name] * count
            assert all("here" in t.users for t in memory.made)


@pytest.mark.parametrize("count,kept", [(1, None), (2, torch.device("cuda", 1))])
def test_blocks_look_at_the_current_device_only_where_there_are_others(monkeypatch, count, kept):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: count)
    assert binding.block_device(torch.device("cuda", 1)) == kept
    assert binding.block_device(torch.device("cpu")) == torch.device("cpu")
