"""The mixer operators on the GPU against their formulas in 64 bits."""
import numpy as np
import pytest

import oracle
from state_space_model_varlen_gb300 import binding, mixer
from tests import mixer_reference as R

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _t(name):
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
            "i8": torch.int8}[name]


def _np(t):
    torch = _torch()
    return t.detach().to(torch.float64).cpu().numpy() if t.dtype != torch.int8 else t.cpu().numpy().astype(np.float64)


def _bits(t):
    return t.contiguous().view(_torch().uint8).cpu().numpy()


class Draw:
    def __init__(self, seed):
        self.g = _torch().Generator(device="cuda").manual_seed(seed)

    def randn(self, *shape, dtype="f32", scale=1.0):
        return (_torch().randn(*shape, generator=self.g, device="cuda") * scale).to(_t(dtype))

    def columns(self, rows, cols, dtype, pad=0):
        """[rows, cols] as a column range of a wider tensor (row stride cols + pad)."""
        return self.randn(rows, cols + pad, dtype=dtype)[:, pad // 2:pad // 2 + cols]

    def slots(self, n, of):
        torch = _torch()
        return torch.randperm(of, generator=self.g, device="cuda")[:n].to(torch.int32)


def _i32(v):
    torch = _torch()
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _status():
    return _torch().zeros(1, dtype=_torch().int32, device="cuda")


# ---------------------------------------------------------------------------
# packed convolution
# ---------------------------------------------------------------------------
def _conv_case(lens, C0, C1, W, io, *, seed=0, pad=0, rows=None, act=True, bias=True, cache=True, start=None,
               slot_stride=1, heads=0):
    torch = _torch()
    d = Draw(seed)
    T, S, C = sum(lens), len(lens), C0 + 2 * C1
    R_ = rows or W
    cu = np.concatenate([[0], np.cumsum(lens)])
    c = dict(cu=cu, xbc=d.columns(T, C, io, pad), w=d.randn(C, W, dtype=io, scale=0.5),
             bias=d.randn(C, dtype=io) if bias else None, act=act)
    c["ring"] = d.randn(S + 2, R_, C, dtype=io) if cache else None
    slot = d.slots(S, S + 2)
    c["slot"] = slot
    if slot_stride > 1:
        table = torch.full((S, slot_stride), -9, dtype=torch.int32, device="cuda")
        table[:, 1] = slot
        c["slot"] = table[:, 1]
    c["start"] = None if start is None else _i32([start(s) for s in range(S)])
    c["dt"] = d.columns(T, heads, io, 3) if heads else None
    c["out"] = [torch.full((T, n), float("nan"), dtype=_t(io), device="cuda") for n in (C0, C1, C1)]
    c["out_dt"] = torch.full((T, heads), float("nan"), device="cuda") if heads else None
    return c


def _conv_run(c, stream=None):
    torch = _torch()
    st = _status()
    keep = None if c["ring"] is None else c["ring"].clone()
    p = mixer.make_conv_params(c["xbc"], c["w"], _i32(c["cu"]), *c["out"], bias=c["bias"], activation=c["act"],
                               conv_cache=c["ring"], slot_idx=c["slot"] if c["ring"] is not None else None,
                               start_pos=c["start"], dt=c["dt"], out_dt=c["out_dt"], device_status=st)
    torch.cuda.synchronize()
    mixer.call_conv(p, torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream)
    torch.cuda.synchronize()
    return keep, int(st.item())


def _conv_check(c, keep, io):
    want, err, ring = R.conv(_np(c["xbc"]), _np(c["w"]), 0.0 if c["bias"] is None else _np(c["bias"]), c["act"], c["cu"],
                             None if c["start"] is None else c["start"].cpu().numpy(), c["slot"].cpu().numpy(),
                             None if keep is None else _np(keep))
    R.check(np.concatenate([_np(o) for o in c["out"]], 1), want, err, io, "convolution")
    if keep is not None:
        np.testing.assert_array_equal(_np(c["ring"]), ring)
    if c["dt"] is not None:
        np.testing.assert_array_equal(_np(c["out_dt"]), _np(c["dt"]))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,C0,C1,W,kw", [
    ([1], 64, 16, 4, {}),
    ([1, 1, 1, 1, 1], 64, 16, 4, dict(start=lambda s: s)),                  # decode rows at positions 0..4
    ([2, 3, 4, 5], 64, 16, 4, dict(start=lambda s: 7 * s)),                 # around the width
    ([0, 1, 0, 0, 33, 0], 64, 16, 4, dict(start=lambda s: 3)),              # empty sequences
    ([31, 32, 33, 64, 1, 95], 1024, 128, 4, dict(pad=16)),                  # around the tile, aligned columns
    ([200], 128, 8, 4, dict(start=lambda s: 2, heads=3)),
    ([70, 5], 40, 8, 1, {}), ([70, 5], 40, 8, 2, {}), ([70, 5], 40, 8, 3, dict(rows=7)),
    ([70, 5, 1], 40, 8, 8, dict(rows=9, start=lambda s: 4)),
    ([37, 2], 25, 3, 4, dict(pad=5, start=lambda s: 100, heads=1)),         # odd channels, unaligned rows
    ([37, 2], 25, 3, 3, dict(pad=4)),
    ([300, 50], 64, 16, 4, dict(cache=False)), ([9, 40], 64, 16, 4, dict(bias=False, act=False)),
    ([40, 41], 64, 16, 4, dict(slot_stride=5, start=lambda s: 11 - s)),
    ([1] * 150 + [130], 72, 8, 4, dict(start=lambda s: s % 6, heads=7)),    # a mixed batch
    ([3] * 700, 16, 8, 4, dict(start=lambda s: s % 5)),                     # more sequences than threads
])
def test_conv(lens, C0, C1, W, kw, io):
    c = _conv_case(lens, C0, C1, W, io, **kw)
    keep, st = _conv_run(c)
    assert st == 0
    _conv_check(c, keep, io)


@pytest.mark.parametrize("cuts", [[64], [1, 2, 63], [30, 31, 32, 33, 61], list(range(1, 70))])
def test_conv_in_pieces_is_the_whole(cuts):
    """A prompt cut into calls that carry the ring gives the same bits and leaves the same last inputs."""
    torch = _torch()
    whole = _conv_case([70], 64, 16, 4, "bf16", seed=3, start=lambda s: 5)
    ring0 = whole["ring"].clone()
    _conv_run(whole)
    ring, got = ring0.clone(), []
    edges = [0] + cuts + [70]
    for a, b in zip(edges, edges[1:]):
        part = dict(whole, cu=np.array([0, b - a]), xbc=whole["xbc"][a:b], start=_i32([5 + a]), ring=ring,
                    out=[torch.empty_like(o[a:b]) for o in whole["out"]])
        _conv_run(part)
        got.append(torch.cat(part["out"], 1))
    assert torch.equal(torch.cat(got), torch.cat(whole["out"], 1))
    q, last = int(whole["slot"][0]), [(5 + 70 - k) % 4 for k in (1, 2, 3)]     # the rows that the call defines
    assert torch.equal(ring[q][last], whole["ring"][q][last])


@pytest.mark.parametrize("W", [4, 7])
def test_conv_ring_in_place_where_sequences_begin_at_a_tiles_end(W):
    """Sequences of 12 tokens with W or 12 ring rows, so that the rows a sequence writes last are among those its first
    tokens read, beginning at every distance (mod 4) from a tile's end, in more CTAs than run at a time."""
    lens, C = [7] + [12] * 900, 10_240
    c = _conv_case(lens, C - 512, 256, W, "bf16", seed=W, start=lambda s: 5 + s, rows=12 if W == 7 else 4)
    keep, st = _conv_run(c)
    assert st == 0
    at = np.unique(np.concatenate([np.arange(3, C, 128), np.arange(C - 3, C)]))
    want, err, ring = R.conv(_np(c["xbc"])[:, at], _np(c["w"])[at], _np(c["bias"])[at], True, c["cu"],
                             c["start"].cpu().numpy(), c["slot"].cpu().numpy(), _np(keep)[:, :, at])
    R.check(_np(_torch().cat(c["out"], 1))[:, at], want, err, "bf16", "convolution")
    np.testing.assert_array_equal(_np(c["ring"])[:, :, at], ring)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 23, 24, 25, 40, 56, 63, 64, 65])
def test_conv_sequences_across_tile_ends(n):
    """A sequence that begins n tokens into the batch, whatever the tile, and others of one to five tokens after it."""
    c = _conv_case([n, 9, 1, 2, 3, 4, 5, 30], 64, 16, 4, "bf16", seed=n, start=lambda s: 3 * s)
    keep, st = _conv_run(c)
    assert st == 0
    _conv_check(c, keep, "bf16")


def test_conv_fresh_sequences_do_not_read_the_ring():
    c = _conv_case([1, 3, 40, 2], 64, 16, 4, "bf16", start=lambda s: 0)
    c["ring"].fill_(float("nan"))
    keep, st = _conv_run(c)
    got = np.concatenate([_np(o) for o in c["out"]], 1)
    want, err, _ = R.conv(_np(c["xbc"]), _np(c["w"]), _np(c["bias"]), True, c["cu"], None, None, None)
    assert st == 0
    R.check(got, want, err, "bf16", "convolution")


def test_conv_bad_metadata_is_reported_and_skipped():
    torch = _torch()
    for what, flag in (("cu", binding.SSD_DEV_BAD_SEQLENS), ("slot", binding.SSD_DEV_BAD_SLOT),
                       ("start", mixer.SSD_DEV_BAD_POS)):
        c = _conv_case([40, 40, 40], 64, 16, 4, "bf16", start=lambda s: 9)
        ok = dict(c)
        if what == "cu":
            c["cu"] = np.array([0, 40, 200, 120])       # sequence 1 runs past T, sequence 2 backwards
        elif what == "slot":
            c["slot"] = c["slot"].clone()
            c["slot"][1] = 99
        else:
            c["start"] = _i32([9, -1, 9])
        keep, st = _conv_run(c)
        assert st == flag, what
        good = [0] if what == "cu" else [0, 2]
        want, err, ring = R.conv(_np(ok["xbc"]), _np(ok["w"]), _np(ok["bias"]), True, [0, 40, 80, 120], [9, 9, 9],
                                 [int(v) if 0 <= int(v) < 5 else 0 for v in c["slot"]], _np(keep))
        got = np.concatenate([_np(o) for o in c["out"]], 1)
        for s in range(3):
            rows = slice(40 * s, 40 * s + 40)
            if s in good:
                R.check(got[rows], want[rows], err[rows], "bf16", "convolution")
            else:
                assert np.all(np.isnan(got[rows]))
        named = [int(c["slot"][s]) for s in good]
        for q in range(5):
            if q not in named:
                assert torch.equal(c["ring"][q], keep[q])


def test_conv_non_finite_inputs_stay_with_their_channel_and_window():
    c = _conv_case([50], 64, 16, 4, "bf16", seed=8)
    c["xbc"][10, 3] = float("nan")
    c["xbc"][30, 70] = float("inf")
    _conv_run(c)
    got = np.concatenate([_np(o) for o in c["out"]], 1)
    bad = ~np.isfinite(got)
    want = np.zeros_like(bad)
    want[10:14, 3] = True
    assert np.array_equal(bad[:, :70], want[:, :70]) and not bad[:, 71:].any()
    assert not bad[:30, 70].any() and not bad[34:, 70].any()


def test_conv_offsets_past_32_bits():
    """225,000 tokens of 10,240 channels: element offsets pass 2^31 (inputs and outputs)."""
    torch = _torch()
    d = Draw(5)
    T, C, W = 225_000, 10_240, 4
    xbc = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    xbc[-600:] = d.randn(600, C, dtype="bf16")
    w, bias = d.randn(C, W, dtype="bf16"), d.randn(C, dtype="bf16")
    out = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    mixer.call_conv(mixer.make_conv_params(xbc, w, _i32([0, T]), out, bias=bias),
                    torch.cuda.current_stream().cuda_stream)
    want, err, _ = R.conv(_np(xbc[-600:, ::64]), _np(w[::64]), _np(bias[::64]), True, [0, 600], None, None, None)
    R.check(_np(out[-600:, ::64])[3:], want[3:], err[3:], "bf16", "convolution")


# ---------------------------------------------------------------------------
# single-token step
# ---------------------------------------------------------------------------
def _stored(h, kind):
    """fp32 states [..., N] as a cache of that type, and its scales."""
    torch = _torch()
    if kind not in R.LIM:
        return h.to(_t(kind)), None
    m = h.abs().amax(-1)
    v = h * torch.where(m > 0, R.LIM[kind] / m, torch.zeros_like(m))[..., None]
    code = v.clamp(-448, 448).to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(v).to(torch.int8)
    return code, m / R.LIM[kind]


def _step_case(B, H, P, N, G, W, io, kind, *, seed=0, pad=0, rows=None, gate=False, bias=True, slots=None, sr=None,
               act=True, softplus=True, slot_stride=1, zero_pos=True):
    torch = _torch()
    d = Draw(seed)
    C = H * P + 2 * G * N
    n = slots or B + 2
    c = dict(H=H, P=P, N=N, G=G, io=io, kind=kind, act=act, softplus=softplus)
    c["xbc"], c["dt"] = d.columns(B, C, io, pad), d.columns(B, H, io, pad)
    c["z"] = d.columns(B, H * P, io, pad) if gate else None
    c["w"], c["bias"] = d.randn(C, W, dtype=io, scale=0.5), d.randn(C, dtype=io) if bias else None
    c["A"] = -torch.exp(torch.rand(H, generator=d.g, device="cuda") * 2.7)
    c["dt_bias"], c["D"] = (d.randn(H, scale=0.5) - 2.0, d.randn(H)) if bias else (None, None)
    c["ring"] = d.randn(n, rows or W, C, dtype=io)
    c["state"], c["scale"] = _stored(d.randn(n, H, P, N), kind)
    c["pos"] = _i32([(0 if zero_pos and b % 5 == 1 else b % 3 if b % 5 == 2 else 1000 + 17 * b) for b in range(B)])
    slot = d.slots(B, n)
    if slot_stride > 1:
        table = torch.full((B, slot_stride), -9, dtype=torch.int32, device="cuda")
        table[:, 1] = slot
        slot = table[:, 1]
    c["slot"] = slot
    c["seed"] = None if sr is None else torch.tensor([sr], dtype=torch.int64, device="cuda")
    c["y"] = torch.full((B, H, P), float("nan"), dtype=_t(io), device="cuda")
    return c


def _step_params(c, st=None):
    return mixer.make_step_params(c["xbc"], c["dt"], c["w"], c["A"], c["ring"], c["state"], c["pos"], c["slot"], c["y"],
                                  ngroups=c["G"], z=c["z"], conv_bias=c["bias"], dt_bias=c["dt_bias"], D=c["D"],
                                  state_scale=c["scale"], sr_seed=c["seed"], activation=c["act"],
                                  dt_softplus=c["softplus"], device_status=st)


def _step_run(c):
    torch = _torch()
    st = _status()
    before = {k: None if c[k] is None else c[k].clone() for k in ("ring", "state", "scale")}
    mixer.call_step(_step_params(c, st), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return before, int(st.item())


def _step_check(c, before, clear=0.9):
    torch = _torch()
    slot = c["slot"].cpu().numpy()
    H, P, N, kind = c["H"], c["P"], c["N"], c["kind"]
    live = [b for b in range(len(slot)) if 0 <= slot[b] < c["state"].shape[0]]
    state = _np(before["state"])
    if before["scale"] is not None:
        state = state * _np(before["scale"])[..., None]
    zero = np.zeros(H)
    y, ey, h, eh, ring = R.step(
        _np(c["xbc"]), _np(c["dt"]), _np(c["w"]), 0.0 if c["bias"] is None else _np(c["bias"]), _np(c["A"]),
        zero if c["dt_bias"] is None else _np(c["dt_bias"]), None if c["D"] is None else _np(c["D"]),
        c["pos"].cpu().numpy(), slot, _np(before["ring"]), state, None if c["z"] is None else _np(c["z"]), c["G"],
        c["act"], c["softplus"])
    R.check(_np(c["y"]), y, ey, c["io"], "y")
    np.testing.assert_array_equal(_np(c["ring"]), ring)
    for b in live:
        q = int(slot[b])
        got = _np(c["state"][q])
        if kind in R.LIM or (kind == "f16" and c["seed"] is not None):
            e = (np.arange(H * P * N, dtype=np.uint64) + np.uint64(q * H * P * N)).reshape(H, P, N)
            seed = None if c["seed"] is None else int(c["seed"].item())
        if kind in R.LIM:
            rnd = None if seed is None else R.random_bytes(seed, e)
            R.check_codes(got, _np(c["scale"][q]), h[b], eh[b], kind, rnd, clear)
        elif kind == "f16" and c["seed"] is not None:
            words = oracle.sr_words(seed, q, (0, H), H, P, N)
            lo, hi = (oracle.sr_round_f16((h[b] + s * eh[b]).astype(np.float32), words).astype(np.float64)
                      for s in (-1.001, 1.001))
            assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))
            assert np.mean(lo == hi) >= clear
        else:
            R.check(got, h[b], eh[b], kind, "state")
    named = {int(slot[b]) for b in live}
    for q in set(range(c["state"].shape[0])) - named:
        assert np.array_equal(_bits(c["state"][q]), _bits(before["state"][q]))
        if c["scale"] is not None:
            assert torch.equal(c["scale"][q], before["scale"][q])


KINDS = ["f32", "bf16", "f16", "e4m3", "i8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,P,N,G,W,kw", [
    (1, 8, 64, 128, 2, 4, dict(zero_pos=False)),
    (7, 4, 64, 128, 1, 4, dict(gate=True)),
    (6, 4, 64, 64, 4, 4, dict(pad=6, slot_stride=3)),
    (5, 2, 128, 256, 1, 4, {}),
    (6, 3, 16, 16, 3, 2, dict(gate=True, pad=3)),
    (4, 2, 50, 100, 1, 4, dict(rows=6)),
    (6, 2, 33, 40, 2, 3, {}),
    (6, 1, 130, 37, 1, 4, {}),                          # odd state size: rows of no vector alignment
    (3, 2, 3, 1, 1, 1, {}), (4, 2, 5, 200, 2, 8, dict(rows=8)),
    (5, 4, 20, 128, 2, 4, dict(bias=False, act=False, softplus=False)),
])
def test_step(B, H, P, N, G, W, kw, io, kind):
    c = _step_case(B, H, P, N, G, W, io, kind, **kw)
    if not c["softplus"]:
        c["dt"].abs_()
    before, st = _step_run(c)
    assert st == 0
    _step_check(c, before)


@pytest.mark.parametrize("kind", ["f16", "e4m3", "i8"])
@pytest.mark.parametrize("H,P,N", [(4, 64, 128), (4, 16, 64), (2, 20, 256), (2, 50, 100), (3, 7, 37), (1, 5, 8)])
def test_step_stochastic_rounding(H, P, N, kind):
    c = _step_case(5, H, P, N, 1, 4, "bf16", kind, sr=0x1234_5678_9ABC_DEF0, seed=11)
    before, st = _step_run(c)
    assert st == 0
    _step_check(c, before)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "i8"])
@pytest.mark.parametrize("B,H,P,N,G,W", [(6, 4, 64, 128, 2, 4), (5, 3, 50, 100, 1, 2), (4, 2, 7, 37, 1, 4)])
def test_step_fp32_activations_store_the_bits_of_a_plain_program(B, H, P, N, G, W, kind):
    """fp32 activations, a narrower cache: every operation rounds by itself, so elementwise torch operations in the
    formula's order (taps summed from the oldest, bias last) give the stored states bit for bit, step after step."""
    torch = _torch()
    c = _step_case(B, H, P, N, G, W, "f32", kind, seed=21)
    c["A"] = -torch.rand(H, device="cuda") - 0.5
    lim = R.LIM.get(kind)
    for _ in range(3):
        q, pos = c["slot"].long(), c["pos"].long()
        u = torch.zeros_like(c["xbc"])
        for k in range(W - 1, -1, -1):
            x = c["xbc"] if k == 0 else c["ring"][q, (pos - k) % W] * (pos >= k)[:, None]
            u = u + c["w"][:, W - 1 - k] * x
        u = u + c["bias"]
        u = u / (1.0 + torch.exp(-u))
        x = u[:, :H * P].view(B, H, P)
        Bm = u[:, H * P:H * P + G * N].view(B, G, N).repeat_interleave(H // G, 1)
        dt = c["dt"] + c["dt_bias"]
        dt = dt.clamp(min=0) + torch.log1p(torch.exp(-dt.abs()))
        h = c["state"].view(torch.uint8)[q].view(_t(kind)).float()
        if lim:
            h = h * c["scale"][q][..., None]
        h = torch.where((pos > 0)[:, None, None, None], h, 0.0)
        h = torch.exp(dt * c["A"])[..., None, None] * h + (dt[..., None] * x)[..., None] * Bm[:, :, None]
        if lim:
            m = h.abs().amax(-1)
            v = h * (torch.reciprocal(m) * lim)[..., None]
            want = v.to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(v).to(torch.int8)
        else:
            want = h.to(_t(kind))
        _step_run(c)
        got = c["state"].view(torch.uint8)[q].view(_t(kind))
        assert np.array_equal(_bits(got), _bits(want))
        c["pos"] += 1


def test_step_padding_and_bad_requests():
    torch = _torch()
    for kind in ("f32", "e4m3"):
        c = _step_case(8, 4, 40, 64, 2, 4, "bf16", kind, zero_pos=False)
        slots = c["slot"].clone()
        c["slot"][1] = c["slot"][4] = -1
        before, st = _step_run(c)
        assert st == 0
        assert float(c["y"][[1, 4]].float().abs().max()) == 0.0
        _step_check(c, before)
        for field, value, flag in (("slot", 99, binding.SSD_DEV_BAD_SLOT), ("slot", -2, binding.SSD_DEV_BAD_SLOT),
                                   ("pos", -1, mixer.SSD_DEV_BAD_POS)):
            c = _step_case(8, 4, 40, 64, 2, 4, "bf16", kind, zero_pos=False)
            q = int(c["slot"][3])
            c[field][3] = value
            before, st = _step_run(c)
            assert st == flag
            assert torch.isnan(c["y"][3].float()).all()
            assert np.array_equal(_bits(c["state"][q]), _bits(before["state"][q]))
            assert torch.equal(c["ring"][q], before["ring"][q])
            assert torch.isfinite(c["y"][[0, 1, 2, 4, 5, 6, 7]].float()).all()
        assert slots.shape[0] == 8


def test_step_fresh_slots_need_no_clearing():
    """Position 0 reads neither cache, whatever a slot's last owner left there."""
    torch = _torch()
    for kind in KINDS:
        c = _step_case(3, 2, 16, 64, 1, 4, "bf16", kind, seed=2)
        c["pos"].zero_()
        clean = _step_case(3, 2, 16, 64, 1, 4, "bf16", kind, seed=2)
        clean["pos"].zero_()
        c["ring"].fill_(float("nan"))
        if kind in R.LIM:
            c["scale"].fill_(float("nan"))
        else:
            c["state"].fill_(float("nan"))
        _step_run(c)
        _step_run(clean)
        assert torch.equal(c["y"], clean["y"])
        q = clean["slot"].long()
        assert np.array_equal(_bits(c["state"].view(torch.uint8)[q]), _bits(clean["state"].view(torch.uint8)[q]))


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_step_non_finite_rows_and_zero_rows(kind, poison):
    """A row with a non-finite value gets the scale NaN and stays poisoned; its neighbours and zero rows do not."""
    torch = _torch()
    c = _step_case(2, 2, 16, 64, 1, 4, "f32", kind, zero_pos=False, bias=False)
    c["xbc"][0, 5] = poison                              # x of row (head 0, p 5)
    c["xbc"][1] = 0.0                                    # the second request: zero inputs and states
    c["ring"][int(c["slot"][1])] = 0.0
    c["scale"][int(c["slot"][1])] = 0.0
    _step_run(c)
    s = c["scale"][int(c["slot"][0])]
    assert torch.isnan(s[0, 5]) and int(torch.isnan(s).sum()) == 1
    q = int(c["slot"][1])
    assert float(c["scale"][q].abs().max()) == 0.0 and float(c["y"][1].abs().max()) == 0.0
    assert float(c["state"][q].float().abs().max()) == 0.0


def test_step_offsets_past_32_bits():
    """2,100 slots of 2^20 codes: the last slot's offset passes 2^31."""
    torch = _torch()
    c = _step_case(1, 2, 64, 128, 1, 4, "bf16", "e4m3", zero_pos=False)
    H, P, N, n = 128, 64, 128, 2100
    d = Draw(4)
    C = H * P + 2 * N
    c.update(H=H, xbc=d.randn(1, C, dtype="bf16"), dt=d.randn(1, H, dtype="bf16"), w=d.randn(C, 4, dtype="bf16"),
             bias=None, A=-torch.rand(H, device="cuda", generator=d.g), dt_bias=None, D=None,
             ring=torch.zeros(n, 4, C, dtype=torch.bfloat16, device="cuda"),
             y=torch.zeros(1, H, P, dtype=torch.bfloat16, device="cuda"), slot=_i32([n - 1]))
    c["state"] = torch.zeros(n, H, P, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    c["scale"] = torch.zeros(n, H, P, device="cuda")
    code, scale = _stored(d.randn(H, P, N), "e4m3")
    c["state"].view(torch.uint8)[n - 1] = code.view(torch.uint8)
    c["scale"][n - 1] = scale
    small = dict(c, ring=c["ring"][n - 1:].clone(), state=c["state"][n - 1:].clone(), scale=c["scale"][n - 1:].clone(),
                 slot=_i32([0]), y=c["y"].clone())
    _step_run(small)
    mixer.call_step(_step_params(c), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(c["y"], small["y"])
    assert np.array_equal(_bits(c["state"][n - 1]), _bits(small["state"][0]))
    assert torch.equal(c["scale"][n - 1], small["scale"][0]) and float(c["scale"][:n - 1].abs().max()) == 0.0


def test_step_on_another_stream_and_in_a_graph():
    torch = _torch()
    a, b = (_step_case(9, 4, 64, 128, 2, 4, "bf16", "e4m3", seed=6, sr=77) for _ in range(2))
    for _ in range(3):
        _step_run(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = _step_params(b)
    with torch.cuda.stream(side):
        mixer.call_step(p, side.cuda_stream)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mixer.call_step(p, side.cuda_stream)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["y"], b["y"]) and np.array_equal(_bits(a["state"]), _bits(b["state"]))


@pytest.mark.parametrize("captured", [False, True])
def test_order_with_copies_other_streams_and_plain_kernels(captured):
    """Each operator is set up while the work before it drains: it must still see all of it, whatever that is (a copy,
    a fill, a kernel of another stream joined by an event, one of these operators), and what follows must see its own."""
    torch = _torch()
    T, H, P = 20_000, 4, 64
    d = Draw(3)
    src, big = d.randn(T, H * P, dtype="bf16"), d.randn(1500, 1500)
    y, z = torch.zeros_like(src), torch.zeros_like(src)
    a, b, e = (torch.zeros_like(src) for _ in range(3))
    states, back = d.randn(40, H, P, 128), torch.zeros(40, H, P, 128, device="cuda")
    cache = torch.zeros(40, H, P, 128, dtype=torch.int8, device="cuda")
    scale, slot = torch.zeros(40, H, P, device="cuda"), _i32(range(40))
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def body():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for _ in range(6):
                big @ big                                   # keeps the side stream busy before it writes z
            z.copy_(src)
        y.fill_(3.0)
        y.copy_(src)
        here.wait_stream(side)
        mixer.gated_rms_norm(y, z=z, group_size=P, out=a)   # after the join
        mixer.gated_rms_norm(a, z=z, group_size=P, out=b)   # after one of its own kind
        back.zero_()
        mixer.state_store(states, cache, scale, slot)
        mixer.state_load(cache, scale, slot, states=back)
        e.copy_(b)                                          # a copy after it
        e.mul_(2.0)
        y.zero_()                                           # overwrites what the norm read

    with torch.cuda.stream(main):
        body()
        torch.cuda.synchronize()
        want = [t.clone() for t in (a, b, e, back)]
        for t in (a, b, e, back, scale):
            t.zero_()
        torch.cuda.synchronize()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=main):
                body()
            for _ in range(5):
                g.replay()
        else:
            for _ in range(5):
                body()
        torch.cuda.synchronize()
    for t, w in zip((a, b, e, back), want):
        assert torch.equal(t, w)
    ref, err = R.norm(_np(src[:50]), _np(src[:50]), None, P, 1e-5, False)
    R.check(_np(a[:50]), ref, err, "bf16", "norm")
    assert torch.equal(e, b * 2.0) and torch.equal(back, cache.float() * scale[..., None])


# ---------------------------------------------------------------------------
# gated norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,group", [
    (1, 8192, 1024), (3, 5120, 5120), (5, 64, 64), (700, 256, 32), (2, 16384, 16384), (4, 30000, 30000),
    (7, 121, 121), (6, 242, 121), (3, 52, 52), (2, 9, 1), (1, 1, 1), (33, 1000, 200), (2, 40000, 40000)])
@pytest.mark.parametrize("gate", ["before", "after", "none"])
def test_norm(rows, cols, group, gate, io):
    torch = _torch()
    d = Draw(rows + cols)
    y, w = d.columns(rows, cols, io, 8 if cols % 8 == 0 else 0), d.randn(cols, dtype=io)
    z = None if gate == "none" else d.columns(rows, cols, io, 16)
    out = torch.full((rows, cols + 8), 7.0, dtype=_t(io), device="cuda")
    mixer.gated_rms_norm(y, w, z=z, group_size=group, eps=1e-5, norm_before_gate=gate == "after", out=out[:, :cols])
    want, err = R.norm(_np(y), None if z is None else _np(z), _np(w), group, 1e-5, gate == "after")
    R.check(_np(out[:, :cols]), want, err, io, "norm")
    assert bool((out[:, cols:] == 7.0).all())


def test_norm_in_place_without_weight_and_zero_rows():
    torch = _torch()
    d = Draw(1)
    y = d.randn(6, 4, 64, dtype="bf16")
    y[2] = 0
    want, err = R.norm(_np(y).reshape(6, 256), None, None, 64, 1e-5, False)
    out = mixer.gated_rms_norm(y, group_size=64, out=y)
    assert out is y
    R.check(_np(y).reshape(6, 256), want, err, "bf16", "norm")
    assert float(y[2].float().abs().max()) == 0.0
    y[1, 0, 0] = float("nan")
    got = mixer.gated_rms_norm(y, group_size=64)
    assert bool(torch.isnan(got[1, 0].float()).all()) and bool(torch.isfinite(got[1, 1:].float()).all())


# ---------------------------------------------------------------------------
# 8-bit cache
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("dense", ["f32", "bf16"])
@pytest.mark.parametrize("sr", [None, 987654321987])
@pytest.mark.parametrize("S,H,P,N", [(3, 4, 64, 128), (5, 2, 50, 100), (2, 3, 7, 37), (4, 2, 16, 256), (1, 1, 1, 1),
                                     (6, 2, 33, 16), (2, 2, 9, 64)])
def test_state_store_and_load(S, H, P, N, sr, dense, kind):
    torch = _torch()
    d = Draw(S + N)
    n = S + 2
    h = (d.randn(S, H, P, N) * torch.exp(3 * d.randn(S, H, P, 1))).to(_t(dense))
    h[0, 0, 0] = 0.0
    cache = torch.zeros(n, H, P, N, dtype=torch.uint8, device="cuda").view(_t(kind))
    scale = torch.full((n, H, P), -1.0, device="cuda")
    slot = d.slots(S, n)
    seed = None if sr is None else torch.tensor([sr], dtype=torch.int64, device="cuda")
    mixer.state_store(h, cache, scale, slot, sr_seed=seed)
    exact = _np(h)
    for i, q in enumerate(slot.tolist()):
        e = (np.arange(H * P * N, dtype=np.uint64) + np.uint64(q * H * P * N)).reshape(H, P, N)
        R.check_codes(_np(cache[q]), _np(scale[q]), exact[i], np.zeros_like(exact[i]), kind,
                      None if sr is None else R.random_bytes(sr, e), clear=0.98)
    named = set(slot.tolist())
    for q in set(range(n)) - named:
        assert float(scale[q].max()) == -1.0 and int(_bits(cache[q]).max()) == 0
    has = _i32([i % 3 != 1 for i in range(S)]).bool()
    back = mixer.state_load(cache, scale, slot, dtype=_t(dense), has_init=has)
    code = cache.view(torch.uint8)[slot.long()].view(_t(kind)).float()
    want = (code * scale[slot.long()][..., None]).to(_t(dense)) * has[:, None, None, None]
    assert torch.equal(back, want)


def test_state_store_and_load_special_rows_and_bad_slots():
    torch = _torch()
    for kind in ("e4m3", "i8"):
        h = torch.randn(4, 1, 6, 32, device="cuda")
        h[0, 0, 0, 3] = float("nan")
        h[0, 0, 1, 3] = float("-inf")
        h[0, 0, 2] = 0.0
        h[0, 0, 3] *= 1e-35                              # below 2^-100: held as zeros
        h[0, 0, 4] *= 1e37
        cache = torch.zeros(5, 1, 6, 32, dtype=torch.uint8, device="cuda").view(_t(kind))
        scale = torch.zeros(5, 1, 6, device="cuda")
        st = _status()
        mixer.state_store(h, cache, scale, _i32([2, 9, -1, 0]), device_status=st)
        assert int(st.item()) == binding.SSD_DEV_BAD_SLOT
        back = mixer.state_load(cache, scale, _i32([2, 0]))
        assert bool(torch.isnan(back[0, 0, :2]).all()) and float(back[0, 0, 2:4].abs().max()) == 0.0
        tol = 0.07 if kind == "e4m3" else 0.02           # half a step of the coarsest code, relative to the row's largest
        for i, s in ((0, 0), (1, 3)):
            rows = slice(4, 6) if i == 0 else slice(0, 6)
            m = h[s, 0, rows].abs().amax(-1, keepdim=True)
            assert bool(((back[i, 0, rows] - h[s, 0, rows]).abs() <= tol * m).all())
        st.zero_()
        dst = torch.full((2, 1, 6, 32), 5.0, device="cuda")
        mixer.state_load(cache, scale, _i32([5, 7]), states=dst, has_init=_i32([1, 0]).bool(), device_status=st)
        assert int(st.item()) == binding.SSD_DEV_BAD_SLOT            # slot 5 skipped, slot 7 not looked at
        assert float(dst[0].min()) == 5.0 and float(dst[1].abs().max()) == 0.0


# ---------------------------------------------------------------------------
# together with the scan
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind,tol", [("f32", 0.02), ("i8", 0.05), ("e4m3", 0.12)])
def test_prompt_then_steps_equals_longer_prompt(kind, tol):
    """Convolution and scan over a prompt, then single-token steps, against the same tokens as one longer prompt.
    tol: bf16 y (2^-7 of its rms twice over) and, for 8-bit caches, the rounding of ten rewrites of the state
    (about 0.4 % each of a row's rms for int8 and 2.7 % for e4m3, decaying)."""
    torch = _torch()
    H, P, N, G, W, S, extra = 4, 64, 128, 1, 4, 3, 10
    lens = [150, 31, 260]
    d = Draw(9)
    C = H * P + 2 * G * N
    w, bias = d.randn(C, W, dtype="bf16", scale=0.5), d.randn(C, dtype="bf16", scale=0.1)
    A = -torch.exp(torch.rand(H, device="cuda", generator=d.g) * 2)
    dt_bias, D = torch.full((H,), -3.0, device="cuda"), d.randn(H)
    tok = [d.randn(n + extra, C + H, dtype="bf16") for n in lens]
    slots = _i32([4, 0, 2])

    def prompt(parts, states, ring):
        xbc = torch.cat(parts)
        cu = _i32(np.concatenate([[0], np.cumsum([p.shape[0] for p in parts])]))
        x, B, Cm, dt = mixer.conv_varlen(xbc[:, :C], w, cu, nheads=H, headdim=P, ngroups=G, dstate=N, bias=bias,
                                         conv_cache=ring, slot_idx=slots, dt=xbc[:, C:])
        y = binding.ssd_scan_varlen(x, dt, A, B, Cm, cu, dt_bias=dt_bias, D=D, state_cache=states, slot_idx=slots)
        return y, cu

    ring = torch.zeros(5, W, C, dtype=torch.bfloat16, device="cuda")
    full, cu = prompt(tok, torch.zeros(5, H, P, N, device="cuda"), ring.clone())
    states = torch.zeros(5, H, P, N, device="cuda")
    prompt([t[:n] for t, n in zip(tok, lens)], states, ring)
    cache, scale = states, None
    if kind in R.LIM:
        cache = torch.zeros(5, H, P, N, dtype=torch.uint8, device="cuda").view(_t(kind))
        scale = torch.zeros(5, H, P, device="cuda")
        mixer.state_store(states[slots.long()].contiguous(), cache, scale, slots)
    pos = _i32(lens)
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    for i in range(extra):
        now = torch.stack([t[n + i] for t, n in zip(tok, lens)])
        y = mixer.step(now[:, :C], now[:, C:], w, A, ring, cache, pos, slots, ngroups=G, conv_bias=bias,
                       dt_bias=dt_bias, D=D, state_scale=scale, sr_seed=seed if kind in R.LIM else None)
        want = torch.stack([full[int(cu[s]) + lens[s] + i] for s in range(S)]).float()
        off = (y.float() - want).norm() / want.norm()
        assert float(off) <= tol, "step %d is %.3g off" % (i, float(off))
        pos += 1
        seed += 1
