"""Measured cases of the operators around the mixer and of the decoding loop: the
residual's addition with the RMS norm (8-bit output among its types), the product
of few rows with 4-bit weights, and the verification of drafted tokens.

``own = False`` computes them in elementary torch operations, in 32 bits (the sums
that pick a token in 64) and rounded once at the end; ``own = True`` calls the
package's kernels.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "i8": 1, "none": 0}
LIM = {"e4m3": 448.0, "i8": 127.0}
TINY = 2.0 ** -100      # a group whose largest magnitude is below this is held as zeros
EPS = 1e-5
KEEP = 0.7              # about the share of drafts that is accepted


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's decode step: the norm before the in-projection, fp32 residual stream
        {"name": "norm_one", "op": "norm", "T": 1, "D": 4096, "io": "bf16", "res": "f32", "code": "none", "group": 0},
        # 8 prompts of 2048 tokens, residual stream in fp32
        {"name": "norm_prompts", "op": "norm", "T": 16384, "D": 2560, "io": "bf16", "res": "f32", "code": "none", "group": 0},
        # a prefill batch of 61,773 tokens, 8-bit activations for the in-projection
        {"name": "norm_codes", "op": "norm", "T": 61773, "D": 4096, "io": "bf16", "res": "bf16", "code": "e4m3", "group": 128},
        # one user's decode step: in-projection to 128 heads (z, x, B, C, dt) and the out-projection back
        {"name": "mv_in", "op": "mv", "M": 1, "K": 4096, "O": 18560, "x": "bf16", "w": 128, "zero": 0, "bias": 0, "scale": "bf16"},
        {"name": "mv_out", "op": "mv", "M": 1, "K": 8192, "O": 4096, "x": "bf16", "w": 128, "zero": 1, "bias": 0, "scale": "f16"},
        # one window of three tokens behind the 8-bit norm
        {"name": "mv_window", "op": "mv", "M": 3, "K": 4096, "O": 18560, "x": "e4m3", "w": 64, "zero": 0, "bias": 0, "scale": "bf16"},
        # a batch of 16 requests, in-projection to 80 heads
        {"name": "mv_batch", "op": "mv", "M": 16, "K": 2560, "O": 10576, "x": "bf16", "w": 32, "zero": 1, "bias": 1, "scale": "bf16"},
        # the head of a vocabulary of 2^17 tokens for one window of three tokens
        {"name": "mv_head", "op": "mv", "M": 3, "K": 4096, "O": 131072, "x": "bf16", "w": 128, "zero": 0, "bias": 0, "scale": "bf16"},
        # a small layer in fp32 at odd sizes
        {"name": "mv_odd", "op": "mv", "M": 5, "K": 1000, "O": 2333, "x": "f32", "w": 50, "zero": 1, "bias": 1, "scale": "f32"},
        # one user's window: two drafts verified
        {"name": "verify_one", "op": "verify", "lens": "same:1:3", "V": 131072, "io": "f32", "draft": 1},
        # 128 windows of three tokens, as the scan's verification batch
        {"name": "verify_batch", "op": "verify", "lens": "same:128:3", "V": 131072, "io": "f32", "draft": 1},
        # ragged windows whose drafts came without probabilities (looked up in the text), odd vocabulary
        {"name": "verify_ragged", "op": "verify", "lens": "ragged:37:9", "V": 50277, "io": "bf16", "draft": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= top and (case["op"] != "verify" or sum(_lens(case)) * case["V"] <= 2 ** 28):
            return case


def _draw(rng):
    op = rng.choice(["norm", "mv", "mv", "verify"])
    if op == "norm":
        code = rng.choice(["none", "e4m3"])
        group = rng.choice([32, 64, 128, 128, 100]) if code != "none" else 1
        D = group * max(1, _log(rng, 16, 16384) // group)
        return {"op": op, "T": _log(rng, 1, 65536), "D": D, "io": rng.choice(["bf16", "bf16", "f32"]),
                "res": rng.choice(["f32", "bf16", "none"]), "code": code,
                "group": 0 if code == "none" else rng.choice([group, group, D])}
    if op == "mv":
        group, K = rng.choice([32, 64, 128, 128, 0]), _log(rng, 128, 16384)
        if rng.random() < 0.85:         # whole groups; otherwise any even number of columns
            K = K // (group or 64) * (group or 64)
        K = K // 2 * 2
        return {"op": op, "M": _log(rng, 1, 64), "K": K, "O": _log(rng, 16, 65536),
                "x": rng.choice(["bf16", "bf16", "f32", "e4m3", "i8"]), "w": group or K, "zero": rng.choice([0, 1]),
                "bias": rng.choice([0, 1]), "scale": rng.choice(["bf16", "f16", "f32"])}
    S = _log(rng, 1, 256)
    return {"op": op, "lens": rng.choice(["same:%d:%d" % (S, rng.randint(1, 6)), "ragged:%d:%d" % (S, rng.randint(2, 12))]),
            "V": _log(rng, 1000, 262144), "io": rng.choice(["f32", "f32", "bf16"]), "draft": rng.choice([0, 1, 1])}


def _lens(c):
    """Window lengths: "same:S:L" or "ragged:S:L" (S windows of 1 to L tokens)."""
    kind, S, L = c["lens"].split(":")
    return [int(L) if kind == "same" else (i * 7919 + 13) % 97 % int(L) + 1 for i in range(int(S))]


def _x_group(c):
    """Columns of an activation scale: what the norm before gives, 128 where that divides the row."""
    return 128 if c["K"] % 128 == 0 else c["K"]


def work(c):
    if c["op"] == "norm":
        n, io, res = c["T"] * c["D"], SIZE[c["io"]], SIZE[c["res"]]
        out = n * io if c["code"] == "none" else n + 4 * n // c["group"]
        return {"bytes": n * (io + 2 * res) + out + c["D"] * io, "flops": n * 8}
    if c["op"] == "mv":
        M, K, O = c["M"], c["K"], c["O"]
        groups, out = -(-K // c["w"]), 4 if c["x"] == "f32" else 2
        return {"bytes": O * -(-K // 2) + O * groups * (SIZE[c["scale"]] + c["zero"]) + M * (K * SIZE[c["x"]] + O * out) +
                c["bias"] * O * out, "flops": 2 * M * K * O}
    lens, io = _lens(c), SIZE[c["io"]]
    # one row of the target's probabilities, and one of the drafts' where a draft is rejected
    rows = sum(1 + c["draft"] * (1 - KEEP ** (n - 1)) for n in lens)
    return {"bytes": int(rows * c["V"] * io) + sum(lens) * 24, "flops": int(rows * c["V"] * 3)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "norm":
        io, T, D = IO[c["io"]], c["T"], c["D"]
        s["x"] = randn(T, D, dtype=io)
        # a residual stream has a few channels that are far larger than the rest
        loud = 1.0 + 20.0 * (rand(D) < 0.01)
        s["residual"] = (randn(T, D) * loud * 3.0).to(IO[c["res"]]) if c["res"] != "none" else None
        s["weight"] = (1.0 + randn(D, scale=0.2)).to(io)
        s["sum"] = torch.empty_like(s["residual"]) if c["res"] != "none" else None
        s["out"] = torch.empty(T, D, dtype=io if c["code"] == "none" else IO[c["code"]], device="cuda")
        s["scale"] = torch.empty(T, D // c["group"], device="cuda") if c["code"] != "none" else None
    elif c["op"] == "mv":
        M, K, O = c["M"], c["K"], c["O"]
        out = torch.float32 if c["x"] == "f32" else torch.bfloat16
        groups = -(-K // c["w"])
        # codes of bell-shaped weights: pairs from a table of 2^12 draws
        nibble = (randn(4096, 2, scale=2.7) + 8).round().clamp(0, 15).to(torch.uint8)
        table = nibble[:, 0] | nibble[:, 1] << 4
        s["weight"] = table[torch.randint(0, 4096, (O, -(-K // 2)), generator=g, device="cuda", dtype=torch.int32)]
        s["scale"] = (torch.exp(randn(O, groups, scale=0.3)) * (0.4 / math.sqrt(K))).to(IO[c["scale"]])
        s["zero"] = torch.randint(6, 11, (O, groups), generator=g, device="cuda", dtype=torch.uint8) if c["zero"] else None
        s["bias"] = randn(O, dtype=out, scale=0.1) if c["bias"] else None
        x = randn(M, K)
        s["x_scale"] = None
        if c["x"] in LIM:
            n = _x_group(c)
            x = x.view(M, -1, n)
            m = x.abs().amax(-1, keepdim=True)
            x = (x * (LIM[c["x"]] / m)).view(M, K)
            x = x.round() if c["x"] == "i8" else x
            s["x_scale"] = (m / LIM[c["x"]]).view(M, -1).contiguous()
        s["x"] = x.to(IO[c["x"]])
        s["out"] = torch.empty(M, O, dtype=out, device="cuda")
    else:
        lens, V, io = _lens(c), c["V"], IO[c["io"]]
        S, T = len(lens), sum(lens)
        cu = torch.tensor([0] + lens).cumsum(0)
        s["cu"] = cu.to(torch.int32).to("cuda")
        first = torch.zeros(T, dtype=torch.bool)
        first[cu[:-1]] = True
        behind = (~first).nonzero().view(-1).cuda()     # tokens of the windows that were drafted, in order
        logits = randn(T, V, scale=2.5)
        p = torch.softmax(logits, 1)
        s["target"] = p.to(io)
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        if c["draft"]:      # a draft model that is a little off the target
            q = torch.softmax(logits[behind - 1] + randn(T - S, V, scale=0.8), 1).to(io)
        else:
            q = p[behind - 1]
        if T > S:
            pick = q.double().cumsum(1)
            u = rand(T - S, 1).double() * pick[:, -1:]
            tokens[behind] = torch.searchsorted(pick, u, right=True).view(-1).clamp(max=V - 1)
            if not c["draft"]:      # a text that repeats itself: many of the drafts are what the target expects
                sure = rand(T - S) < KEEP
                rows = (behind - 1)[sure]
                s["target"][rows] = (0.1 * p[rows]).to(io)
                s["target"][rows, tokens[behind[sure]]] = 0.9
        s["draft"] = q if c["draft"] else None
        s["tokens"] = tokens.to(torch.int32)
        s["accept_u"], s["sample_u"] = rand(T - S), rand(S)
        s["ring"] = torch.randint(0, 9, (S,), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty(S, dtype=torch.int32, device="cuda")
    if own:
        # what a serving program keeps for a layer: the filled argument block of the call
        from state_space_model_varlen_gb300 import layer
        s["params"] = _params(layer, s)
    return s


def _params(layer, s):
    c = s["case"]
    if c["op"] == "norm":
        codes = c["code"] != "none"
        return layer.make_residual_norm_params(s["x"], s["weight"], None if codes else s["out"], residual=s["residual"],
                                               residual_out=s["sum"], codes=s["out"] if codes else None, scale=s["scale"],
                                               eps=EPS)
    if c["op"] == "mv":
        return layer.make_matvec4_params(s["x"], s["weight"], s["scale"], s["out"], group_size=c["w"], zero=s["zero"],
                                         bias=s["bias"], x_scale=s["x_scale"])
    return layer.make_verify_params(s["target"], s["tokens"], s["cu"], s["accept_u"], s["sample_u"], s["out"], s["accepted"],
                                    draft_probs=s["draft"], ring_count=s["ring"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        from state_space_model_varlen_gb300 import layer
        stream = torch.cuda.current_stream().cuda_stream
        if c["op"] == "norm":
            layer.call_residual_norm(s["params"], stream)
            return {"out": s["out"], "sum": s["sum"], "scale": s["scale"]}
        if c["op"] == "mv":
            layer.call_matvec4(s["params"], stream)
            return s["out"]
        layer.call_verify(s["params"], stream)
        return {"tokens": s["out"], "accepted": s["accepted"], "ring": s["ring"]}
    return {"norm": _norm, "mv": _mv, "verify": _verify}[c["op"]](s)


def _norm(s):
    c = s["case"]
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    total = None if s["residual"] is None else v.to(s["residual"].dtype)
    if c["code"] == "none":
        return {"out": n.to(s["x"].dtype), "sum": total, "scale": None}
    n = n.view(c["T"], -1, c["group"])
    lim, m = LIM[c["code"]], n.abs().amax(-1, keepdim=True)
    m = torch.where(m < TINY, 0.0, m)
    code = n * torch.where(m > 0, lim / m, 0.0)
    return {"out": code.view(c["T"], c["D"]).to(IO[c["code"]]), "sum": total, "scale": m[..., 0] / lim}


def _columns(t, K, group):
    """Values of groups of columns, for each of the K columns."""
    return t.repeat_interleave(group, 1)[:, :K]


def _mv(s):
    c = s["case"]
    K, w = c["K"], s["weight"]
    code = torch.stack([w & 15, w >> 4], 2).view(c["O"], -1)[:, :K].float()
    code = code - (8.0 if s["zero"] is None else _columns(s["zero"].float(), K, c["w"]))
    code = code * _columns(s["scale"].float(), K, c["w"])
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * _columns(s["x_scale"], K, _x_group(c))
    out = x @ code.t()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return out.to(s["out"].dtype)


def _verify(s):
    cu, tokens, target, draft = s["cu"].long(), s["tokens"].long(), s["target"], s["draft"]
    S, T, V = cu.shape[0] - 1, tokens.shape[0], target.shape[1]
    lens, at = cu[1:] - cu[:-1], torch.arange(T, device=cu.device)
    seq = torch.repeat_interleave(torch.arange(S, device=cu.device), lens, output_size=T)
    place = at - cu[seq]                                # of a token in its window
    row = (at - seq - 1).clamp(min=0)                   # of a drafted token among the drafts
    if T > S:
        q = 1.0 if draft is None else draft[row, tokens].double()
        ok = s["accept_u"][row].double() * q < target[(at - 1).clamp(min=0), tokens].double()
        # the first rejected place of each window
        n = torch.where(ok | (place == 0), lens[seq], place)
        n = torch.full((S,), T, device=cu.device).scatter_reduce(0, seq, n, "amin") - 1
    else:
        n = lens - 1
    stop, last = cu[:-1] + n, n == lens - 1
    w = target[stop].double()
    if T > S:
        i = (stop - torch.arange(S, device=cu.device)).clamp(max=T - S - 1)
        if draft is None:
            less = torch.nn.functional.one_hot(tokens[(stop + 1).clamp(max=T - 1)], V).double()
        else:
            less = draft[i].double()
        rest = (w - less).clamp(min=0.0)
        rest = torch.where((rest.sum(1) > 0)[:, None], rest, w)
        w = torch.where(last[:, None], w, rest)
    total = w.cumsum(1)
    new = (total <= s["sample_u"].double()[:, None] * total[:, -1:]).sum(1).clamp(max=V - 1)
    # drafts up to the rejected one, then the new token
    following = torch.cat([tokens[1:], tokens[:1]])
    out = torch.where(place < n[seq], following, torch.where(place == n[seq], new[seq], -1))
    s["ring"] += (n + 1).int()
    return {"tokens": out.int(), "accepted": n.int(), "ring": s["ring"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits, row by row
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    d = torch.float64
    if c["op"] == "norm":
        outs, sums, scales = [], [], []
        for a in range(0, c["T"], 8192):
            v = s["x"][a:a + 8192].to(d)
            if s["residual"] is not None:
                v = v + s["residual"][a:a + 8192].to(d)
                sums.append(v)
            n = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["D"] + EPS) * s["weight"].to(d)
            if c["code"] != "none":         # the values that the codes are rounded from
                parts = n.split(c["group"], 1)
                m = torch.stack([p.abs().max(1).values for p in parts], 1) / LIM[c["code"]]
                n = torch.cat([p / m[:, i:i + 1].clamp(min=1e-300) for i, p in enumerate(parts)], 1)
                scales.append(m)
            outs.append(n)
        return {"out": torch.cat(outs), "sum": torch.cat(sums) if sums else None, "scale": torch.cat(scales) if scales else None}
    if c["op"] == "mv":
        K, x, parts = c["K"], s["x"].to(d), []
        if s["x_scale"] is not None:
            n = _x_group(c)
            x = (x.reshape(c["M"], -1, n) * s["x_scale"].to(d)[..., None]).reshape(c["M"], K)
        for a in range(0, c["O"], 8192):
            w = s["weight"][a:a + 8192].int()
            full = torch.empty(w.shape[0], 2 * w.shape[1], dtype=d, device="cuda")
            full[:, 0::2], full[:, 1::2] = w % 16, w // 16
            total = torch.zeros(c["M"], w.shape[0], dtype=d, device="cuda") if s["bias"] is None else \
                s["bias"][a:a + 8192].to(d).expand(c["M"], -1).clone()
            scale = s["scale"][a:a + 8192].to(d)
            if K // c["w"] <= 16:       # group by group
                for i, k in enumerate(range(0, K, c["w"])):
                    z = 8 if s["zero"] is None else s["zero"][a:a + 8192, i:i + 1].to(d)
                    e = min(K, k + c["w"])
                    total += (x[:, k:e] @ (full[:, k:e] - z).t()) * scale[:, i]
            else:
                of = torch.arange(K, device="cuda") // c["w"]
                z = 8 if s["zero"] is None else s["zero"][a:a + 8192].to(d)[:, of]
                total += x @ ((full[:, :K] - z) * scale[:, of]).t()
            parts.append(total)
        return torch.cat(parts, 1)
    cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
    out, accepted, ring = [], [], s["ring"].tolist()
    au, su = s["accept_u"].tolist(), s["sample_u"].tolist()
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        n = 0
        while n < b - a - 1:
            tok = tokens[a + n + 1]
            q = 1.0 if s["draft"] is None else float(s["draft"][a + n - i, tok])
            if not au[a + n - i] * q < float(s["target"][a + n, tok]):
                break
            n += 1
        w = s["target"][a + n].to(d)
        if n < b - a - 1:
            r = w.clone()
            if s["draft"] is None:
                r[tokens[a + n + 1]] = 0.0
            else:
                r = torch.relu(w - s["draft"][a + n - i].to(d))
            w = r if float(r.sum()) > 0 else w
        c_ = torch.cumsum(w, 0)
        pick = int(torch.nonzero(c_ > su[i] * c_[-1])[0])
        out += tokens[a + 1:a + n + 1] + [pick] + [-1] * (b - a - n - 1)
        accepted.append(n)
        ring[i] += n + 1
    return {"tokens": torch.tensor(out), "accepted": torch.tensor(accepted), "ring": torch.tensor(ring)}
