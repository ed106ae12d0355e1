"""Multi-token decoding of a small Mamba2 model on the package's operators: 4-bit
projections behind a residual norm with 8-bit output, ReplaySSM verification of
drafted windows, and the choice of what stands of them on the device.

    python examples/mtp_decode.py [--tokens 48] [--window 3]

Random weights, greedy decoding.  The prompts are prefilled, then every round runs
one captured graph: the windows through all layers, the head, and verify_drafts,
which advances the rings of the layers.  Decoding with the right drafts has to give
the same tokens as with wrong ones, in fewer rounds.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_varlen_gb300 import binding, layer, mixer, ssd_scan_varlen  # noqa: E402

I32 = torch.int32


class Weights4:
    """A random matrix [out, in] in 4 bits, with a scale for each group of columns of a row."""

    def __init__(self, out, n, group, g, device):
        w = torch.randn(out, n, generator=g, device=device).view(out, -1, group) * n ** -0.5
        self.group = group
        self.scale = (w.abs().amax(2) / 7).to(torch.bfloat16)
        code = (w / self.scale.float()[..., None]).round().clamp(-8, 7).view(out, n).to(torch.int8) + 8
        code = code.to(torch.uint8)
        self.codes = code[:, 0::2] | code[:, 1::2] << 4

    def __call__(self, x, x_scale=None, **kw):
        return layer.matvec4(x, self.codes, self.scale, group_size=self.group, x_scale=x_scale, **kw)


class Layer:
    """Weights of one Mamba2 layer, its convolution ring, and a checkpoint and an input ring for each slot."""

    def __init__(self, hidden, H, P, N, G, width, slots, window, ring_window, g, device):
        def randn(*shape, scale=1.0, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

        self.H, self.P, self.N, self.G = H, P, N, G
        self.inner, self.channels = H * P, H * P + 2 * G * N
        self.norm_w = 1 + randn(hidden, scale=0.1)
        self.w_in = Weights4(self.inner + self.channels + H, hidden, 64, g, device)
        self.w_out = Weights4(hidden, self.inner, 128, g, device)
        self.conv_w, self.conv_b = randn(self.channels, width, scale=0.5), randn(self.channels, scale=0.1)
        self.gate_w = 1 + randn(self.inner, scale=0.1)
        self.A = -torch.exp(torch.rand(H, generator=g, device=device) * 2.7)
        self.dt_bias = torch.full((H,), -3.0, device=device)
        self.D = randn(H, dtype=torch.float32)
        # the ring of the convolution keeps a whole window besides the taps: drafts that fall are overwritten
        self.conv_ring = torch.zeros(slots, width + window, self.channels, dtype=torch.bfloat16, device=device)
        self.state = torch.zeros(slots, H, P, N, device=device)
        rows = ring_window + window
        self.ring_x = torch.zeros(slots, rows, H, P, dtype=torch.bfloat16, device=device)
        self.ring_dt = torch.zeros(slots, rows, H, device=device)
        self.ring_B = torch.zeros(slots, rows, G, N, dtype=torch.bfloat16, device=device)

    def forward(self, x, residual, cu, slots, pos, mix):
        """One layer over packed tokens; `mix` runs the recurrence on (x, dt, B, C).  The residual stream is advanced."""
        codes, scale = layer.residual_rms_norm(x, self.norm_w, residual=residual, residual_out=residual,
                                               code_dtype=torch.float8_e4m3fn, scale_group=128)
        z, xbc, dt = self.w_in(codes, scale).split([self.inner, self.channels, self.H], 1)
        xs, B, C, dt = mixer.conv_varlen(xbc, self.conv_w, cu, nheads=self.H, headdim=self.P, ngroups=self.G,
                                         dstate=self.N, bias=self.conv_b, conv_cache=self.conv_ring, slot_idx=slots,
                                         start_pos=pos, dt=dt)
        y = mix(self, xs, dt, B, C)
        normed = mixer.gated_rms_norm(y.view(-1, self.inner), self.gate_w, z=z, group_size=self.inner // self.G)
        return self.w_out(normed)


class Model:
    def __init__(self, layers=2, hidden=512, vocab=1000, H=16, P=64, N=128, G=1, width=4, slots=6, window=3, ring_window=8,
                 device="cuda", seed=0):
        if not 1 <= window < width:     # the convolution leaves the last width - 1 inputs of a call in its ring
            raise ValueError("a window has 1 to %d tokens" % (width - 1))
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.window, self.ring_window, self.device = hidden, window, ring_window, device
        self.embedding = torch.randn(vocab, hidden, generator=g, device=device).to(torch.bfloat16)
        self.layers = [Layer(hidden, H, P, N, G, width, slots, window, ring_window, g, device) for _ in range(layers)]
        self.norm_w = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.head = Weights4(vocab, hidden, 32, g, device)

    def logits(self, tokens, cu, slots, pos, mix):
        x = self.embedding[tokens.long()]
        residual = torch.zeros(x.shape, device=self.device)
        for one in self.layers:
            x = one.forward(x, residual, cu, slots, pos, mix)
        return self.head(layer.residual_rms_norm(x, self.norm_w, residual=residual), out_dtype=torch.float32)

    def prefill(self, prompts, slots):
        """All tokens of the prompts but the last, which begins the first window."""
        lens = [p.shape[0] - 1 for p in prompts]
        cu = torch.tensor([0] + lens).cumsum(0).to(I32).to(self.device)
        pos = torch.zeros(len(prompts), dtype=I32, device=self.device)

        def mix(one, xs, dt, B, C):
            return ssd_scan_varlen(xs, dt, one.A, B, C, cu, dt_bias=one.dt_bias, D=one.D, state_cache=one.state,
                                   slot_idx=slots)

        self.logits(torch.cat([p[:-1] for p in prompts]), cu, slots, pos, mix)
        return torch.tensor(lens, dtype=I32, device=self.device)

    def decode(self, prompts, slots, tokens, drafts):
        """`tokens` new tokens for each prompt, greedily.  `drafts`: [prompts, tokens + window] guesses of what follows the
        prompts.  Returns the tokens and the rounds that they took."""
        S, L = len(prompts), self.window
        pos = self.prefill(prompts, slots)
        first = pos.clone()
        cu = torch.arange(0, S * L + 1, L, dtype=I32, device=self.device)
        last = torch.stack([p[-1] for p in prompts]).to(I32)
        start, count = (torch.zeros(S, dtype=I32, device=self.device) for _ in range(2))
        start_out, count_out = torch.zeros_like(start), torch.zeros_like(count)
        result = torch.zeros(S, tokens + 2 * L, dtype=I32, device=self.device)
        status = torch.zeros(1, dtype=I32, device=self.device)
        accept_u = torch.full((S * (L - 1),), 0.5, device=self.device)      # greedy: the numbers do not matter
        sample_u = torch.full((S,), 0.5, device=self.device)
        behind = torch.arange(L, device=self.device)

        def mix(one, xs, dt, B, C):
            y = torch.empty_like(xs)
            p = binding.make_params(xs, dt, one.A, B, C, cu, dt_bias=one.dt_bias, D=one.D, state_cache=one.state,
                                    slot_idx=slots, write_final=False, out_y=y, max_seqlen=L, device_status=status)
            binding.call_replay(binding.make_replay_params(p, one.ring_x, one.ring_dt, one.ring_B, self.ring_window, start,
                                                           count, start_out, count_out),
                                torch.cuda.current_stream().cuda_stream)
            return y

        def a_round():
            done = (pos - first).long()                     # tokens that each prompt has been given
            guesses = drafts.gather(1, (done[:, None] + behind[:-1]).clamp(max=drafts.shape[1] - 1))
            window = torch.cat([last[:, None], guesses.to(I32)], 1).view(-1)
            logits = self.logits(window, cu, slots, pos, mix)
            target = torch.nn.functional.one_hot(logits.argmax(1), logits.shape[1]).float()
            new, accepted = layer.verify_drafts(target, window, cu, accept_u, sample_u, ring_count=count_out,
                                                device_status=status)
            new = new.view(S, L)
            result.scatter_(1, (done[:, None] + behind).clamp(max=result.shape[1] - 1), new)
            last.copy_(new.gather(1, accepted[:, None].long())[:, 0])
            pos.add_(accepted + 1)
            start.copy_(start_out)
            count.copy_(count_out)

        kept = [(t, t.clone()) for t in (pos, last, start, count, result,
                                         *(t for one in self.layers for t in (one.conv_ring, one.state, one.ring_x,
                                                                              one.ring_dt, one.ring_B)))]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a_round()                                       # warm-up; what it changed is put back
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a_round()
        for t, before in kept:
            t.copy_(before)
        rounds = 0
        while int((pos - first).min()) < tokens:
            graph.replay()
            rounds += 1
        assert int(status) == 0
        return result[:, :tokens].clone(), rounds


def run(tokens=48, window=3, lens=(9, 60, 200), seed=0, **sizes):
    """(tokens with wrong drafts, its rounds, tokens with the right drafts, its rounds)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    slots = torch.tensor([4, 1, 3][:len(lens)], dtype=I32, device="cuda")
    vocab = sizes.get("vocab", 1000)
    prompts = [torch.randint(0, vocab, (n,), generator=g, device="cuda").to(I32) for n in lens]
    # a wrong draft now and then hits; what is compared does not depend on it
    wrong = torch.randint(0, vocab, (len(lens), tokens + window), generator=g, device="cuda")
    a, rounds_a = Model(window=window, seed=seed, **sizes).decode(prompts, slots, tokens, wrong)
    right = torch.cat([a.long(), wrong[:, :window]], 1)
    b, rounds_b = Model(window=window, seed=seed, **sizes).decode(prompts, slots, tokens, right)
    return a, rounds_a, b, rounds_b


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=48)
    p.add_argument("--window", type=int, default=3)
    args = p.parse_args()
    a, rounds_a, b, rounds_b = run(args.tokens, args.window)
    print("%d tokens for each of %d prompts: %d rounds with wrong drafts, %d with the right ones, the tokens are %s"
          % (args.tokens, a.shape[0], rounds_a, rounds_b, "the same" if torch.equal(a, b) else "NOT the same"))
