"""The single-token step against a plain fp32 program, bit for bit and step
after step: what a narrow cache stores is rounded to a few bits, so a state that
is off by one fp32 rounding can be off by a whole code, and a code that differs
in a row's largest value moves the whole row's scale."""
import numpy as np
import pytest

import oracle
from tests import mixer_reference as R
from tests.test_mixer_gpu import _bits, _step_case, _step_run, _t, _torch

pytestmark = pytest.mark.gpu

M32 = 0xFFFFFFFF


def _philox(q, stream, seed):
    """The four words of Philox4x32-10 with counters (q, q >> 32, stream, 0), [len(q), 4], in 64-bit integers."""
    torch = _torch()

    def product(a, b):          # high and low words of a 32 x 32-bit product, in steps that stay below 2^63
        part = (b & 0xFFFF) * a
        high = (b >> 16) * a + (part >> 16)
        return high >> 16, ((high & 0xFFFF) << 16) | (part & 0xFFFF)

    c = [q & M32, q >> 32, torch.full_like(q, stream), torch.zeros_like(q)]
    key = [seed & M32, seed >> 32 & M32]
    for _ in range(10):
        (h0, l0), (h1, l1) = product(0xD2511F53, c[0]), product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
    return torch.stack(c, 1)


def _words(shape, seed):
    """The random word of every element of an fp16 cache."""
    torch = _torch()
    n = int(np.prod(shape))
    return _philox(torch.arange((n + 3) // 4, device="cuda"), 0, seed).reshape(-1)[:n].view(shape)


def _bytes(shape, seed):
    """The random byte of every element of an 8-bit cache."""
    torch = _torch()
    n = int(np.prod(shape))
    w = _philox(torch.arange((n + 15) // 16, device="cuda"), 2, seed)
    return torch.stack([w >> 8 * i & 0xFF for i in range(4)], 2).reshape(-1)[:n].view(shape)


def test_random_numbers_are_the_oracles():
    torch = _torch()
    q, seed = [0, 1, 77, 2 ** 32 - 1, 2 ** 32 + 5], 0x1234_5678_9ABC_DEF0
    got = _philox(torch.tensor(q, device="cuda"), 2, seed).cpu().numpy()
    at = np.array(q, dtype=np.uint64)
    want = oracle.philox4x32_10([at & np.uint64(M32), at >> np.uint64(32), np.full(at.shape, 2, np.uint64),
                                 np.zeros(at.shape, np.uint64)], (seed & M32, seed >> 32))
    np.testing.assert_array_equal(got, np.stack([np.asarray(w, dtype=np.int64) for w in want], 1))
    e = np.arange(100, dtype=np.uint64)
    np.testing.assert_array_equal(_bytes((100,), seed).cpu().numpy(), R.random_bytes(seed, e).astype(np.int64))
    np.testing.assert_array_equal(_words((2, 1, 2, 8), seed)[1].cpu().numpy(),
                                  oracle.sr_words(seed, 1, (0, 1), 1, 2, 8).astype(np.int64))


def plain_step(c):
    """The stored states and scales that elementwise fp32 torch operations in the order of the formulas give (taps
    summed from the oldest, the bias last)."""
    torch = _torch()
    H, P, N, G, kind = c["H"], c["P"], c["N"], c["G"], c["kind"]
    B, W, rows = c["xbc"].shape[0], c["w"].shape[1], c["ring"].shape[1]
    q, pos, lim = c["slot"].long(), c["pos"].long(), R.LIM.get(kind)
    u = torch.zeros_like(c["xbc"], dtype=torch.float32)
    for k in range(W - 1, -1, -1):
        x = c["xbc"].float() if k == 0 else c["ring"][q, (pos - k) % rows].float() * (pos >= k)[:, None]
        u = u + c["w"][:, W - 1 - k].float() * x
    u = u + c["bias"].float()
    u = u / (1.0 + torch.exp(-u))
    x = u[:, :H * P].view(B, H, P)
    Bm = u[:, H * P:H * P + G * N].view(B, G, N).repeat_interleave(H // G, 1)
    dt = c["dt"].float() + c["dt_bias"]
    dt = dt.clamp(min=0) + torch.log1p(torch.exp(-dt.abs()))
    h = c["state"].view(torch.uint8)[q].view(_t(kind)).float()
    if lim:
        h = h * c["scale"][q][..., None]
    h = torch.where((pos > 0)[:, None, None, None], h, 0.0)
    h = torch.exp(dt * c["A"])[..., None, None] * h + (dt[..., None] * x)[..., None] * Bm[:, :, None]
    seed = None if c["seed"] is None else int(c["seed"].item())
    shape = tuple(c["state"].shape)
    if not lim:
        return (h.to(_t(kind)) if seed is None else _sr_f16(h, _words(shape, seed)[q])), None
    m = h.abs().amax(-1)
    v = h * (torch.reciprocal(m) * lim)[..., None]
    scale = m * float(np.float32(1.0) / np.float32(lim))
    if seed is None:
        return (v.to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(v).to(torch.int8)), scale
    r = _bytes(shape, seed)[q]
    if kind == "i8":
        return torch.floor(v + (r.float() + 0.5) / 256.0).to(torch.int8), scale
    half = (v * 2.0 ** -8).to(torch.float16).view(torch.int16)
    code = ((half & 0x7FFF) + (r & 0x7F).to(torch.int16)) >> 7
    return (code | ((half < 0).to(torch.int16) << 7)).to(torch.uint8).view(torch.float8_e4m3fn), scale


def _sr_f16(h, words):
    torch = _torch()
    a = h.abs()
    lo = a.to(torch.float16)
    lo = torch.where(lo.float() > a, (lo.view(torch.int16) - 1).view(torch.float16), lo)
    hi = (lo.view(torch.int16) + 1).view(torch.float16)
    part = (a.double() - lo.double()) / (hi.double() - lo.double())
    return torch.copysign(torch.where(part * 2.0 ** 32 > words.double(), hi, lo).float(), h).to(torch.float16)


@pytest.mark.parametrize("kind,sr", [("e4m3", None), ("i8", None), ("e4m3", 1), ("i8", 1), ("f16", 1)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,P,N,G,W,kw", [
    (48, 32, 64, 128, 4, 4, {}),                        # 12.6 million values: enough for codes that a rounding tips
    (5, 3, 50, 100, 1, 2, dict(pad=3)),                 # vectors of four values, single channels
    (4, 2, 7, 37, 1, 3, {}),                            # single values
    (6, 4, 20, 24, 2, 3, dict(pad=8)),                  # rows of 17 to 32 values
    (3, 2, 64, 256, 1, 4, {}), (3, 2, 16, 16, 1, 8, dict(rows=9)),
])
def test_step_stores_the_bits_of_a_plain_program(B, H, P, N, G, W, kw, io, kind, sr):
    """The codes and scales of ten steps, each from the last one's, with a new seed a step."""
    torch = _torch()
    c = _step_case(B, H, P, N, G, W, io, kind, seed=31, sr=sr and 0x0F1E_2D3C_4B5A_6978, **kw)
    c["A"] = -torch.rand(H, device="cuda") - 0.5
    q = c["slot"].long()
    for step in range(10):
        want, scale = plain_step(c)
        _, st = _step_run(c)
        assert st == 0
        got = c["state"].view(torch.uint8)[q].view(_t(kind))
        off = int((got.view(torch.uint8) != want.view(torch.uint8)).sum())
        assert off == 0, "step %d: %d bytes differ" % (step, off)
        if scale is not None:
            assert torch.equal(c["scale"][q], scale), "step %d" % step
        c["pos"] += 1
        c["xbc"].copy_(torch.roll(c["xbc"].clone(), 1, 1))
        if sr:
            c["seed"] += 1
    assert np.array_equal(_bits(got), _bits(want))
