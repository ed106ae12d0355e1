"""The layer operators together with the mixer's and the scan's, as a decoding loop uses them."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,lens", [(3, (9, 60, 200)), (2, (5, 2)), (1, (33,))])
def test_drafts_change_the_rounds_and_not_the_tokens(window, lens):
    import torch
    from examples import mtp_decode
    tokens = 24
    a, rounds_a, b, rounds_b = mtp_decode.run(tokens, window, lens)
    assert a.shape == (len(lens), tokens) and int(a.min()) >= 0 and torch.equal(a, b)
    # the right drafts stand: a window of tokens a round
    assert rounds_b == -(-tokens // window) and rounds_a >= rounds_b + (window > 1)


def test_verified_counts_feed_the_replay():
    """The ring counts that verify_drafts leaves are those that the next window's replay needs: two windows with part of the
    drafts accepted give the states of the tokens that stand, run one after another."""
    import torch
    from state_space_model_varlen_gb300 import binding, layer, ssd_scan_varlen
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    S, L, H, P, N, V, I32 = 3, 3, 4, 64, 128, 64, torch.int32
    bf = torch.bfloat16
    x, B, C = randn(2, S, L, H, P, dtype=bf), randn(2, S, L, 1, N, dtype=bf, scale=0.1), randn(2, S, L, 1, N, dtype=bf)
    dt, A = randn(2, S, L, H) * 0.3 - 2, -torch.rand(H, generator=g, device="cuda")
    cu, slots = torch.arange(0, S * L + 1, L, dtype=I32, device="cuda"), torch.tensor([2, 0, 1], dtype=I32, device="cuda")
    state = randn(S, H, P, N, scale=0.1)
    begin = state.clone()
    rx, rdt, rB = randn(S, 7, H, P, dtype=bf), randn(S, 7, H), randn(S, 7, 1, N, dtype=bf)
    start, count, so, co = (torch.zeros(S, dtype=I32, device="cuda") for _ in range(4))
    stream = torch.cuda.current_stream().cuda_stream

    def window(i):
        y = torch.empty(S * L, H, P, dtype=bf, device="cuda")
        p = binding.make_params(x[i].view(S * L, H, P), dt[i].reshape(S * L, H), A, B[i].view(S * L, 1, N), C[i].view(S * L, 1, N),
                                cu, state_cache=state, slot_idx=slots, write_final=False, out_y=y, max_seqlen=L)
        binding.call_replay(binding.make_replay_params(p, rx, rdt, rB, 4, start, count, so, co), stream)
        return y.view(S, L, H, P)

    window(0)
    # request s keeps s drafts: its target expects them, and token 63 where it stops
    tokens = torch.arange(S * L, dtype=I32, device="cuda")
    target = torch.zeros(S * L, V, device="cuda")
    for s in range(S):
        for i in range(L):
            target[s * L + i, int(tokens[s * L + i + 1]) if i < s else 63] = 1.0
    out, accepted = layer.verify_drafts(target, tokens, cu, torch.full((S * (L - 1),), 0.9, device="cuda"),
                                        torch.full((S,), 0.9, device="cuda"), ring_count=co)
    assert accepted.tolist() == [0, 1, 2] and co.tolist() == [1, 2, 3]
    assert out.view(S, L).tolist() == [[63, -1, -1], [4, 63, -1], [7, 8, 63]]
    start.copy_(so)
    count.copy_(co)
    y = window(1)
    for s in range(S):
        stand = [(0, s, i) for i in range(s + 1)] + [(1, s, i) for i in range(L)]
        pick = lambda t: torch.stack([t[a] for a in stand])         # noqa: E731
        want = ssd_scan_varlen(pick(x), pick(dt), A, pick(B), pick(C), torch.tensor([0, len(stand)], dtype=I32, device="cuda"),
                               state_cache=begin, slot_idx=slots[s:s + 1], write_final=False,
                               has_init=torch.ones(1, dtype=torch.uint8, device="cuda"))
        # bf16 outputs of two ways to the same fp32 sums: half a step each, and the sums' own roundings
        ref = want[-L:].float()
        assert ((y[s].float() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2e-2 * ref.square().mean().sqrt()).all()
