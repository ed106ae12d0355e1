"""A Mamba2 mixer layer on the package's operators: packed prompts through the
convolution, the scan and the gated norm, then single tokens through the step
and the norm, on one set of caches.

    python examples/mamba2_mixer.py [--state f32|bf16|e4m3|i8] [--tokens 16]

Random weights.  Three prompts of different lengths are prefilled (the longest
one in two calls), decoded for a few tokens in a CUDA graph, and compared with
the same tokens as longer prompts.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_varlen_gb300 import mixer, ssd_scan_varlen  # noqa: E402

STATES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


class Mamba2Mixer:
    """Weights of one layer and its caches: the convolution's ring and the states, by slot."""

    def __init__(self, hidden=1024, nheads=32, headdim=64, dstate=128, ngroups=1, width=4, slots=8, state="f32",
                 device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale=1.0, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

        self.H, self.P, self.N, self.G = nheads, headdim, dstate, ngroups
        self.inner, self.channels = nheads * headdim, nheads * headdim + 2 * ngroups * dstate
        self.w_in = randn(self.inner + self.channels + nheads, hidden, scale=hidden ** -0.5)
        self.w_out = randn(hidden, self.inner, scale=self.inner ** -0.5)
        self.conv_w, self.conv_b = randn(self.channels, width, scale=0.5), randn(self.channels, scale=0.1)
        self.norm_w = 1 + randn(self.inner, scale=0.1)
        self.A = -torch.exp(torch.rand(nheads, generator=g, device=device) * 2.7)
        self.dt_bias = torch.full((nheads,), -3.0, device=device)
        self.D = randn(nheads, dtype=torch.float32)
        self.ring = torch.zeros(slots, width, self.channels, dtype=torch.bfloat16, device=device)
        self.state = torch.zeros(slots, nheads, headdim, dstate, device=device).to(STATES[state])
        self.scale = torch.zeros(slots, nheads, headdim, device=device) if state in ("e4m3", "i8") else None
        self.seed = torch.zeros(1, dtype=torch.int64, device=device)      # of the stochastic rounding, one a step

    def _split(self, x):
        """z, (x, B, C) and dt of the in-projection, as column ranges of one tensor."""
        proj = x @ self.w_in.t()
        return proj.split([self.inner, self.channels, self.H], 1)

    def _finish(self, y, z):
        normed = mixer.gated_rms_norm(y.view(-1, self.inner), self.norm_w, z=z, group_size=self.inner // self.G)
        return normed @ self.w_out.t()

    def prefill(self, x, cu_seqlens, slots, start_pos):
        """Packed prompts, or pieces of prompts that continue at start_pos."""
        z, xbc, dt = self._split(x)
        xs, B, C, dt = mixer.conv_varlen(xbc, self.conv_w, cu_seqlens, nheads=self.H, headdim=self.P, ngroups=self.G,
                                         dstate=self.N, bias=self.conv_b, conv_cache=self.ring, slot_idx=slots,
                                         start_pos=start_pos, dt=dt)
        has_init = start_pos > 0
        state, idx = self.state, slots
        if self.scale is not None:      # the scan works on fp32 states; the cache holds 8 bits
            state = mixer.state_load(self.state, self.scale, slots, has_init=has_init)
            idx = torch.arange(slots.shape[0], dtype=torch.int32, device=slots.device)
        y = ssd_scan_varlen(xs, dt, self.A, B, C, cu_seqlens, dt_bias=self.dt_bias, D=self.D, state_cache=state,
                            slot_idx=idx, has_init=has_init)
        if self.scale is not None:
            mixer.state_store(state, self.state, self.scale, slots)
        return self._finish(y, z)

    def decode(self, x, slots, pos):
        """One token for each request; slot -1 is a padding row."""
        z, xbc, dt = self._split(x)
        y = mixer.step(xbc, dt, self.conv_w, self.A, self.ring, self.state, pos, slots, ngroups=self.G,
                       conv_bias=self.conv_b, dt_bias=self.dt_bias, D=self.D, state_scale=self.scale,
                       sr_seed=None if self.scale is None else self.seed)
        return self._finish(y, z)


def run(state="f32", tokens=16, hidden=1024, lens=(200, 33, 1500), **sizes):
    """Relative error of the decoded tokens' outputs against the longer prompts' (worst token)."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    x = [torch.randn(n + tokens, hidden, generator=g, device=dev).to(torch.bfloat16) for n in lens]
    slots = torch.tensor([5, 2, 7][:len(lens)], dtype=torch.int32, device=dev)

    def packed(parts):
        cu = torch.tensor([0] + [p.shape[0] for p in parts]).cumsum(0).to(torch.int32).to(dev)
        return torch.cat(parts), cu

    def starts(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    whole = Mamba2Mixer(hidden=hidden, **sizes)
    data, cu = packed(x)
    want = whole.prefill(data, cu, slots, starts([0] * len(lens)))

    layer = Mamba2Mixer(hidden=hidden, state=state, **sizes)
    cut = [n // 2 if n == max(lens) else n for n in lens]
    data, first = packed([v[:c] for v, c in zip(x, cut)])
    layer.prefill(data, first, slots, starts([0] * len(lens)))
    rest = [i for i, (c, n) in enumerate(zip(cut, lens)) if c < n]
    data, second = packed([x[i][cut[i]:lens[i]] for i in rest])
    layer.prefill(data, second, slots[rest], starts([cut[i] for i in rest]))

    # decoding in a CUDA graph of four rows, the last of them padding
    rows = len(lens) + 1
    now = torch.zeros(rows, hidden, dtype=torch.bfloat16, device=dev)
    row_slots = torch.cat([slots, starts([-1])])
    pos = starts(list(lens) + [0])
    graph_in = (layer.ring.clone(), layer.state.clone(), None if layer.scale is None else layer.scale.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(now, row_slots, pos)                   # warm-up; the caches are put back below
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(now, row_slots, pos)
    for t, kept in zip((layer.ring, layer.state, layer.scale), graph_in):
        if t is not None:
            t.copy_(kept)
    worst = 0.0
    for i in range(tokens):
        now[:len(lens)] = torch.stack([v[n + i] for v, n in zip(x, lens)])
        graph.replay()
        ref = torch.stack([want[int(cu[s]) + lens[s] + i] for s in range(len(lens))]).float()
        got = out[:len(lens)].float()
        worst = max(worst, float((got - ref).norm() / ref.norm()))
        pos += 1
        layer.seed += 1
    return worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--state", choices=sorted(STATES), default="e4m3")
    p.add_argument("--tokens", type=int, default=16)
    a = p.parse_args()
    print("state cache %s: decoded outputs differ from the longer prompts' by %.2g at most (relative, over a token's batch)"
          % (a.state, run(a.state, a.tokens)))
