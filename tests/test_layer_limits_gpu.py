"""The layer operators at the ends of what their calls allow, on the GPU."""
import numpy as np
import pytest

from state_space_model_varlen_gb300 import layer
from tests import layer_reference as R
from tests.test_layer_gpu import Draw, _norm_case, _np, _probs, _t, _torch, _verify_check, _windows

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# verification: many windows of a large vocabulary, where a sum that is left covers several blocks of a row
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("S,V", [(192, 131072), (256, 100003), (700, 17000), (1024, 50280), (1024, 32000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_many_windows_of_large_vocabularies(S, V, dtype):
    """Windows of one token and of two, the draft of every other one rejected, so that rows of p and of p - q are sampled, at
    0, inside, just below 1, at 1 and above; rows whose last blocks, or all but one, are without weight."""
    torch = _torch()
    d = Draw(S + V)
    lens = [1 + s % 2 for s in range(S)]
    T, D = sum(lens), S // 2
    cu = _windows(lens)
    target, q = _probs(d, T, V, dtype), _probs(d, D, V, dtype)
    tokens = d.ints(1, V, T)
    au = torch.zeros(D, device="cuda")
    au[::2] = 1.0                               # above what p / q can be at the token: rejected
    first = cu[1:-1:2].long()                   # of the windows of two
    ones = cu[:-1:2].long()
    drafted = tokens[first + 1].long()
    target[first[::2], drafted[::2]] = 0.0
    for i, live in enumerate((V - 600, V // 3, 700, 1)):        # columns behind which there is nothing
        for rows in (ones[1 + i::7], first[2 * (1 + i)::14]):
            target[rows, live:] = 0.0
    q[2::4, :] = 0.0                            # all of the target's row is left
    su = d.rand(S)
    at = torch.arange(S, device="cuda") // 2 % 6
    for i, u in enumerate((0.0, 1.0 - 2.0 ** -24, 1.0, 2.0)):
        su[at == i] = u
    out, acc, _, status = _verify_check(target, q, tokens, cu, au, su)
    assert status == 0 and (acc[1::4] == 0).all() and (acc[0::2] == 0).all()
    # without the oracle: at 1 and above the last token of any weight
    picked = torch.from_numpy(out).cuda()[ones]
    last = (torch.arange(V, device="cuda") * (target[ones] > 0)).amax(1)
    end = su[::2] >= 1
    assert end.sum() > S // 8 and torch.equal(picked[end].long(), last[end])


def test_verify_gives_a_window_the_same_token_whatever_stands_beside_it():
    torch = _torch()
    d = Draw(17)
    V = 131072
    rows = _probs(d, 6, V, "f32")
    u = torch.tensor([0.0, 0.3, 1.0 - 2.0 ** -24, 1.0, 2.0, 0.999], device="cuda")
    zeros = torch.zeros(6, dtype=torch.int32, device="cuda")
    alone = _verify_check(rows, None, zeros, _windows([1] * 6), None, u)[0]
    S = 300
    many = _verify_check(rows.repeat(S // 6, 1), None, zeros.repeat(S // 6), _windows([1] * S), None, u.repeat(S // 6))[0]
    assert np.array_equal(many.reshape(-1, 6), np.tile(alone, (S // 6, 1)))
    assert alone[3] == alone[4] == V - 1


@pytest.mark.parametrize("S", [5, 400])
def test_verify_rows_whose_sum_is_no_fp32_number(S):
    """Finite weights that add up to more than fp32 holds pick no token; others beside them, up to its end, do."""
    torch = _torch()
    V, big = 20000, 2.0 ** 127
    p = torch.zeros(2 * S, V, device="cuda")
    q = torch.zeros(S, V, device="cuda")
    tokens = torch.full((2 * S,), 7, dtype=torch.int32, device="cuda")
    p[0::2, 8] = big
    p[0::2, 9000] = big * 0.5                   # 0.75 2^128: u = 0.5 is token 8, 0.75 token 9000
    over = torch.arange(S) % 3 == 1
    p[0::2][over, V - 1] = big * 0.75
    su = torch.where(torch.arange(S, device="cuda") % 2 == 0, 0.5, 0.75)
    out, acc = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (2 * S, S))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for draft in (q, None):
        out.fill_(-77)
        status.zero_()
        layer.verify_drafts(p, tokens, _windows([2] * S), torch.full((S,), 0.5, device="cuda"), su, draft_probs=draft,
                            out_tokens=out, out_accepted=acc, device_status=status)
        want = torch.where(su == 0.5, 8, 9000).int()
        want[over.cuda()] = -1
        assert torch.equal(out[0::2], want) and (out[1::2] == -1).all() and (acc == 0).all() and int(status) == 128


@pytest.mark.parametrize("unit", [2.0 ** -149, 2.0 ** -130, 2.0 ** -100, 2.0 ** -59, 2.0 ** 90])
@pytest.mark.parametrize("S,V", [(64, 300), (400, 20000)])
def test_verify_rows_of_any_magnitude(unit, S, V):
    """Whole multiples of a unit: sums and, with random numbers of few bits, products are exact in 64 bits.  Tokens do not
    depend on the unit, that of fp32's smallest number among them."""
    torch = _torch()
    d = Draw(V)
    w = d.ints(0, 4, 1, V).float() * (torch.arange(V, device="cuda") % 7 == 3)
    p = (w.double() * unit).float().repeat(S, 1)
    assert torch.equal(p[0].double() / unit, w[0].double())
    u = torch.arange(S, device="cuda").float() / 512
    zeros = torch.zeros(S, dtype=torch.int32, device="cuda")
    got = _verify_check(p, None, zeros, _windows([1] * S), None, u)
    assert np.array_equal(got[0], _verify_check(w.repeat(S, 1), None, zeros, _windows([1] * S), None, u)[0])


# ---------------------------------------------------------------------------
# residual norm: groups of codes whose shared memory is at the limit of a launch
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cols,group", [(9189, 3), (9192, 3), (9195, 3), (9213, 3), (9219, 3), (10210, 5), (10215, 5), (10240, 5),
                                        (10245, 5)])
@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "f32")])
def test_norm_codes_of_long_rows_in_small_odd_groups(cols, group, io, res):
    _norm_case(2, cols, io, res, "e4m3", group, seed=cols)
    _norm_case(2, cols, io, None, "i8", group, out=False, seed=cols)


# ---------------------------------------------------------------------------
# 4-bit products: rows so long that a bound of roundings says little
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,K,O", [(2, (1 << 20) + 64, 5), (9, (1 << 20) + 7, 3), (3, 1 << 20, 5), (2, 65536, 70), (20, 32768, 40),
                                      (3, 65502, 33)])
@pytest.mark.parametrize("x", ["bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("group", [128, 32, 50, 7, 1 << 30])
def test_matvec_long_rows_exactly(rows, K, O, x, group):
    """Few columns of x are not zero, and scales are powers of two: every sum is a multiple of 2^-4 below 2^20, which fp32
    holds whatever the order, so that the product has to be the exact one."""
    torch = _torch()
    d = Draw(rows + K + O)
    groups = -(-K // group)
    w, z = d.ints(0, 256, O, (K + 1) // 2, dtype="u8"), d.ints(6, 11, O, groups, dtype="u8")
    s = torch.exp2(d.ints(-2, 3, O, groups).float())
    values = d.ints(0, 2, rows, K).float() * 2 - 1
    xv = torch.where(d.rand(rows, K) < min(1.0, 4000.0 / K), values, 0.0)
    for k in (0, 1, 1023, 1024, K // 2, (1 << 20) - 1, 1 << 20, K - 2, K - 1):      # ends of rows and of chunks
        if k < K:
            xv[:, k] = 100.0 if x != "e4m3" else 104.0
    xs, x_group = None, 1
    if x in R.LIM:
        x_group = K // 2 if K % 2 == 0 else K
        xs = torch.exp2(d.ints(-2, 1, rows, K // x_group).float())
    got = layer.matvec4(xv.to(_t(x)), w, s, group_size=group, zero=z, x_scale=xs, out_dtype=torch.float32)
    size = np.abs(_np(xv)).sum(1).max() * 10 * 4
    assert size < 2 ** 20
    want, _ = R.matvec4(_np(xv), w.cpu().numpy(), _np(s), z.cpu().numpy(), None, group, _np(xs), x_group)
    assert np.array_equal(_np(got), want)


@pytest.mark.parametrize("cols", [32, 640, 2009, 40000])
@pytest.mark.parametrize("code", [None, "e4m3"])
def test_norm_rows_whose_squares_fp32_does_not_hold(cols, code):
    """A sum of squares beyond fp32 gives zeros, NaN where the row is not finite; zeros with eps = 0 give NaN; the row
    beside them is as it is alone."""
    torch = _torch()
    d = Draw(cols)
    x = d.randn(4, cols)
    x[0], x[2], x[3, 1] = 2.0 ** 66, 0.0, float("inf")
    kw = dict(eps=0.0, **(dict(code_dtype=_t(code), scale_group=cols) if code else {}))
    got, alone = layer.residual_rms_norm(x, **kw), layer.residual_rms_norm(x[1:2], **kw)
    if code:
        (got, scale), (alone, s1) = got, alone
        assert float(scale[0]) == 0.0 and torch.isnan(scale[2:]).all() and float(scale[1]) == float(s1)
    else:
        assert torch.isnan(got[2]).all() and torch.isnan(got[3, 1]) and (got[3, 2:] == 0).all()
    assert (got[0].float() == 0).all() and torch.equal(got[1:2].float(), alone.float())
