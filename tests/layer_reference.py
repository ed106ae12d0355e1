"""The layer operators in 64 bits (numpy), each with a bound of what fp32
arithmetic may add to it.

  * residual norm: the sum is rounded once (U |v|); the mean square's relative error
    is that of its terms (4 U) and of its additions, at most (columns / 1024 + 40) of
    them in a row; its root halves that; root, division and two products round once
    each;
  * products with 4-bit weights: every addition on a term's way to the output, a
    tensor core's among them, which may cut off instead of rounding, loses at most
    2^-23 of the sum of the terms' magnitudes; a term itself has at most four
    roundings.  There are at most in / 16 + 40 additions one after another;
  * verification gives whole numbers; the sums behind them are exact to about
    2^-44, so that a random number decides otherwise with a chance below 2^-20.
"""
import numpy as np

U = 2.0 ** -24
LIM = {"e4m3": 448.0, "i8": 127.0}


def residual_norm(x, residual, weight, eps):
    """(sum, its bound), (normed, its bound)."""
    v = x if residual is None else x + residual
    ev = 0.0 * v if residual is None else U * np.abs(v)
    columns = x.shape[1]
    mean = (v * v).mean(1, keepdims=True)
    n = v / np.sqrt(mean + eps) * (1.0 if weight is None else weight)
    return (v, ev), (n, np.abs(n) * U * (1 + (4 + columns / 1024 + 40) / 2 + 6))


def unpacked(weight, K):
    """Codes [out, K] of packed bytes."""
    full = np.empty((weight.shape[0], 2 * weight.shape[1]))
    full[:, 0::2], full[:, 1::2] = weight & 15, weight >> 4
    return full[:, :K]


def matvec4(x, weight, scale, zero, bias, group, x_scale=None, x_group=1):
    """The product and its bound."""
    K = x.shape[1]
    at = np.arange(K) // group
    w = (unpacked(weight, K) - (8.0 if zero is None else zero.astype(np.float64)[:, at])) * scale[:, at]
    if x_scale is not None:
        x = x * x_scale[:, np.arange(K) // x_group]
    b = 0.0 if bias is None else bias
    size = np.abs(x) @ np.abs(w).T + np.abs(b)
    return x @ w.T + b, size * (2.0 ** -23 * (K / 16 + 40) + 4 * U)


def verify(target, draft, tokens, cu, accept_u, sample_u, ring, out_tokens, out_accepted):
    """Tokens, accepted and ring counts, from the arrays that the outputs held before, and the status bits."""
    out, acc, status = out_tokens.copy(), out_accepted.copy(), 0
    ring = None if ring is None else ring.copy()
    T, V = target.shape
    drafts = 0 if accept_u is None else len(accept_u)
    clip = lambda u: min(max(float(u), 0.0), 1.0) if u == u else 0.0      # noqa: E731
    for s in range(len(cu) - 1):
        a, b = int(cu[s]), int(cu[s + 1])
        k, d0 = b - a - 1, a - s
        if a < 0 or b < a or b > T or (k > 0 and (d0 < 0 or d0 + k > drafts)):
            status |= 2
            continue
        if k < 0:
            continue
        n, bad = 0, False
        while n < k:
            tok = int(tokens[a + n + 1])
            if not 0 <= tok < V:
                bad = True
                break
            q = 1.0 if draft is None else float(draft[d0 + n, tok])
            if not clip(accept_u[d0 + n]) * q < float(target[a + n, tok]):
                break
            n += 1
        if bad:
            status |= 64
            continue
        p = target[a + n].astype(np.float64)
        usable = lambda w: np.where((w > 0) & (w < np.inf), w, 0.0)         # noqa: E731
        w = usable(p)
        if n < k:
            if draft is None:
                r = w.copy()
                r[int(tokens[a + n + 1])] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    r = usable(p - draft[d0 + n].astype(np.float64))
            w = r if r.sum() > 0 else w
        new = -1
        if w.sum() > 0:
            c = np.cumsum(w)
            over = np.nonzero((c > clip(sample_u[s]) * c[-1]) & (w > 0))[0]
            new = int(over[0]) if len(over) else int(np.nonzero(w)[0][-1])
        else:
            status |= 128
        out[a:a + n] = tokens[a + 1:a + n + 1]
        out[a + n] = new
        out[a + n + 1:b] = -1
        acc[s] = n
        if ring is not None:
            ring[s] += n + 1
    return out, acc, ring, status
