"""The mixer operators in 64 bits (numpy), each with a bound of what fp32
arithmetic may add to it.

The bounds follow the formulas: u24 = 2^-24 is fp32's rounding.
  * a sum of k products: (k + 1) u24 times the sum of their magnitudes;
  * SiLU through ex2 and a reciprocal approximation: relative 2^-20 plus
    |v| 2^-23 from the exponent's own rounding; its slope is at most 1.1;
  * softplus and exp: relative 2^-21, plus what their argument's error makes;
  * the state: its two terms' bounds plus three roundings; the read-out: a sum
    of N products of values that have bounds of their own.
Storing adds half a unit of the stored type.
"""
import numpy as np

import oracle

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # unit roundoff: 24, 8, 11 significant bits
LIM = {"e4m3": 448.0, "i8": 127.0}


def sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def silu(v, err=0.0):
    u = v * sigmoid(v)
    return u, 1.1 * err + np.abs(u) * (2.0 ** -20 + np.abs(v) * 2.0 ** -23)


def conv_window(win, w, bias, act):
    """win [..., W, C] (newest last), w [C, W]: the convolved value and its bound."""
    W = w.shape[1]
    terms = win * w.T
    v = terms.sum(-2) + bias
    err = (W + 2) * U * (np.abs(terms).sum(-2) + np.abs(bias))
    return silu(v, err) if act else (v, err)


def conv(xbc, w, bias, act, cu, start, slot, ring):
    """Packed prompts: outputs, their bounds and the updated ring ([slots, R, C] or None)."""
    out, err = np.zeros_like(xbc), np.zeros_like(xbc)
    W = w.shape[1]
    after = None if ring is None else ring.copy()
    for s in range(len(cu) - 1):
        a, b, p0 = cu[s], cu[s + 1], 0 if start is None else int(start[s])
        past = np.zeros((W - 1, xbc.shape[1]))
        for j in range(W - 1):
            p = p0 - (W - 1) + j
            if p >= 0 and ring is not None:
                past[j] = ring[slot[s], p % ring.shape[1]]
        full = np.concatenate([past, xbc[a:b]])
        for t in range(a, b):
            out[t], err[t] = conv_window(full[t - a:t - a + W], w, bias, act)
        if ring is not None:
            for t in range(max(a, b - (W - 1)), b):
                after[slot[s], (p0 + t - a) % ring.shape[1]] = xbc[t]
    return out, err, after


def step(xbc, dt, w, bias, A, dt_bias, D, pos, slot, ring, state, z, G, act=True, softplus=True):
    """One token per request.  state [slots, H, P, N] in 64 bits (scales applied).  Returns y and its bound, the new
    states [batch, H, P, N] and theirs, and the updated ring.  Requests of slot -1 give y = 0."""
    B = xbc.shape[0]
    _, H, P, N = state.shape
    W, R = w.shape[1], ring.shape[1]
    y, ey = np.zeros((B, H, P)), np.zeros((B, H, P))
    hs, eh = np.zeros((B, H, P, N)), np.zeros((B, H, P, N))
    ring = ring.copy()
    before = ring.copy()
    for b in range(B):
        q, t = int(slot[b]), int(pos[b])
        if q < 0:
            continue
        win = np.stack([before[q, (t - k) % R] if t - k >= 0 else np.zeros(xbc.shape[1])
                        for k in range(W - 1, 0, -1)] + [xbc[b]])
        u, eu = conv_window(win, w, bias, act)
        ring[q, t % R] = xbc[b]
        d = H * P
        x, ex = u[:d].reshape(H, P), eu[:d].reshape(H, P)
        rep = lambda v: np.repeat(v.reshape(G, N), H // G, 0)      # noqa: E731
        Bm, eB = rep(u[d:d + G * N]), rep(eu[d:d + G * N])
        Cm, eC = rep(u[d + G * N:]), rep(eu[d + G * N:])
        raw = dt[b] + dt_bias
        ed = 2 * U * (np.abs(dt[b]) + np.abs(dt_bias))
        if softplus:
            ed = ed * sigmoid(raw)
            d_ = np.maximum(raw, 0) + np.log1p(np.exp(-np.abs(raw)))
            ed = ed + 2.0 ** -21 * d_
        else:
            d_ = raw
        decay = np.exp(d_ * A)
        edecay = decay * (np.abs(A) * ed + 2.0 ** -21 * (1 + np.abs(d_ * A)))
        old = state[q] if t > 0 else np.zeros_like(state[q])
        keep = decay[:, None, None] * old
        add = (d_[:, None] * x)[:, :, None] * Bm[:, None, :]
        h = keep + add
        e = edecay[:, None, None] * np.abs(old) + 3 * U * (np.abs(keep) + np.abs(add)) + U * np.abs(h)
        e += (ed[:, None] * np.abs(x) + d_[:, None] * ex)[:, :, None] * np.abs(Bm)[:, None, :]
        e += (d_[:, None] * (np.abs(x) + ex))[:, :, None] * eB[:, None, :]
        hs[b], eh[b] = h, e
        Dx = np.zeros(H) if D is None else D
        y[b] = np.einsum("hpn,hn->hp", h, Cm) + Dx[:, None] * x
        ey[b] = (np.einsum("hpn,hn->hp", e, np.abs(Cm)) + np.einsum("hpn,hn->hp", np.abs(h) + e, eC)
                 + (N / 8 + 6) * U * np.einsum("hpn,hn->hp", np.abs(h), np.abs(Cm))
                 + np.abs(Dx)[:, None] * ex + 2 * U * (np.abs(y[b]) + np.abs(Dx[:, None] * x)))
        if z is not None:
            gate, eg = silu(z[b].reshape(H, P))
            ey[b] = ey[b] * np.abs(gate) + (np.abs(y[b]) + ey[b]) * eg
            y[b] = y[b] * gate
    return y, ey, hs, eh, ring


def norm(y, z, w, group, eps, after):
    rows, cols = y.shape
    gate, eg = (1.0, 0.0) if z is None else silu(z)
    v = y if after or z is None else y * gate
    g = v.reshape(rows, -1, group)
    r = 1.0 / np.sqrt((g * g).mean(-1, keepdims=True) + eps)
    out = (g * r).reshape(rows, cols) * (1.0 if w is None else w)
    if after and z is not None:
        out = out * gate
    # relative: the gate's, half the sum's (each term twice the gate's worst, plus a tree of additions), five products
    rel = 0.0 if z is None else (2.0 ** -20 + np.abs(z) * 2.0 ** -23) + (2.0 ** -20 + np.abs(z).max() * 2.0 ** -23)
    return out, np.abs(out) * (rel + (group / 64 + 32) * U)


# ---------------------------------------------------------------------------
# stored states
# ---------------------------------------------------------------------------
def random_bytes(seed, elements):
    """The random byte of every flat element index of an 8-bit cache."""
    e = np.asarray(elements, dtype=np.uint64)
    q = e >> np.uint64(4)
    w = oracle.philox4x32_10([q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full(q.shape, 2, np.uint64),
                              np.zeros(q.shape, np.uint64)],
                             (int(seed) & 0xFFFFFFFF, (int(seed) >> 32) & 0xFFFFFFFF))
    word = np.choose(((e >> np.uint64(2)) & np.uint64(3)).astype(np.int64), w)
    return (word >> ((e & np.uint64(3)) * np.uint64(8)).astype(np.uint32)) & np.uint32(0xFF)


def codes(v, kind, rnd=None):
    """Scaled values to code values, monotone in v."""
    if kind == "i8":
        if rnd is None:
            return np.clip(np.rint(v), -127, 127)
        return np.clip(np.floor(v + (rnd + 0.5) / 256.0), -127, 127)
    a = np.minimum(np.abs(v), 448.0)
    if rnd is None:
        unit = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6) - 3)
        return np.copysign(np.rint(a / unit) * unit, v)
    bits = (a / 256.0).astype(np.float16).view(np.uint16).astype(np.int64)
    cut = ((bits + (rnd.astype(np.int64) & 0x7F)) >> 7) << 7
    return np.copysign(cut.astype(np.uint16).view(np.float16).astype(np.float64) * 256.0, v)


def check_codes(code_values, scale, h, eh, kind, rnd=None, clear=0.9):
    """Codes (as numbers) and scales of rows [..., N] against the exact rows h within eh."""
    m = np.abs(h).max(-1)
    em = eh.max(-1)
    assert np.all(np.abs(scale - m / LIM[kind]) <= (em + 4 * U * m) / LIM[kind] + 1e-45), "scales"
    live = scale > 0
    s = np.where(live, scale, 1.0)[..., None]
    v = np.where(live[..., None], h / s, 0.0)
    # the scale's roundings and, drawn, the sum of the value and a number below 1
    ev = np.where(live[..., None], eh / s, 0.0) + 6 * U * np.abs(v) + (0.0 if rnd is None else U * (np.abs(v) + 1))
    lo, hi = codes(v - ev, kind, rnd), codes(v + ev, kind, rnd)
    assert np.all((code_values >= lo) & (code_values <= hi)), "codes outside the bounds: %d" % int(
        np.sum((code_values < lo) | (code_values > hi)))
    share = float(np.mean(lo == hi))
    assert share >= clear, "only %.3f of the codes had one right value" % share


def check(got, want, err, dtype, what):
    tol = err + HALF[dtype] * (np.abs(want) + err) + (2.0 ** -25 if dtype == "f16" else 1e-38)
    assert np.all(np.isfinite(got)), what + ": not finite"
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d outside the bound, worst %.3g x" % (
        what, int(bad.sum()), bad.size, float((np.abs(got - want) / tol).max()))
