"""What the scan holds inside: its bf16 results are fp32 sums rounded once, and its fp32 results
good to fp32.

The inputs leave one or a few positive terms in every sum, so that nothing averages an operand's
rounding away and the bound is relative to the result itself."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# Before the rounding to bf16, in half steps of fp32 (2^-24, relative): a step size 16 (8 * 2^-23),
# a decay whose exponent is below 1 the 16 of its step size, 8 for exp(A_log) and the products that
# make the exponent, 2 for the hardware's exp2, an operand in three bf16 parts 1 (2^-25 and the
# parts' products), up to 12 matrix instructions of one nonzero term each 12, and the products and
# sums behind them 8: 63 in all.  One operand in two parts would be off by up to 2^-17 = 128 half steps.
REL = 64 * R.U


def half_step(v):
    """Half a step of bf16 at v: of 8 bits, so 2^(e - 8) for 2^e <= |v| < 2^(e + 1)."""
    return torch.ldexp(torch.ones_like(v), torch.frexp(v.abs())[1] - 1 - 8)


def check_once(got, want, label):
    """A sum good to REL, rounded to bf16."""
    got = R.d(got)
    assert got.shape == want.shape, label
    off = ((got - want).abs() - half_step(want)) / want.abs()
    off = torch.where(want == 0, got.abs(), off)
    say("%s: beyond half a step %.3g of %.3g" % (label, float(off.max()), REL))
    assert float(off.max()) <= REL, label


def positive(g, *shape):
    return 0.5 + torch.rand(*shape, generator=g)


def hot(g, n, groups, width):
    """[n, 1, groups, width] with a one in a place of its own for every sequence and group; the places."""
    at = torch.randint(width, (n, groups), generator=g)
    return torch.nn.functional.one_hot(at, width)[:, None].to(BF).cuda(), at


N, H, P, S = 1024, 8, 64, 128


def steps(g, n=N, T=1):
    """dt, A_log and dt_bias: step sizes around 0.05, decays around e^-0.1; the step sizes and
    log-decays in 64 bits, [n, T, H]."""
    dt = (0.3 * torch.randn(n, T, H, generator=g)).to(BF)
    A_log, bias = torch.log(positive(g, H)), torch.full((H,), -3.0)
    step = torch.nn.functional.softplus(R.d(dt) + R.d(bias), threshold=100)
    return dt.cuda(), A_log.cuda(), bias.cuda(), step, -torch.exp(R.d(A_log)) * step


def test_outputs_from_the_state():
    """x = 0 and a one-hot C: y is an entry of the state times its decay."""
    g = torch.Generator().manual_seed(1)
    dt, A_log, bias, _, a = steps(g)
    C, at = hot(g, N, 1, S)
    s = positive(g, N, H, P, S)
    x = torch.zeros(N, 1, H, P, dtype=BF, device="cuda")
    y, _ = kda.ssm_fwd(x, dt, C, C, A_log, bias, initial_state=s.cuda())
    entry = R.d(s).gather(3, at.view(N, 1, 1, 1).expand(N, H, P, 1))[..., 0]
    check_once(y[:, 0], entry * torch.exp(a[:, 0])[..., None], "outputs from the state")


@pytest.mark.parametrize("skip", [False, True])
def test_outputs_from_the_token(skip):
    """No state and B = C one-hot: y = dt x, or (dt + D) x."""
    g = torch.Generator().manual_seed(2)
    dt, A_log, bias, step, _ = steps(g)
    C, _ = hot(g, N, 1, S)
    D = positive(g, H)
    x = positive(g, N, 1, H, P).to(BF)
    y, _ = kda.ssm_fwd(x.cuda(), dt, C, C, A_log, bias, D.cuda() if skip else None)
    m = step[..., None] + (R.d(D)[:, None] if skip else 0)
    check_once(y, m * R.d(x), "outputs from the token")


@pytest.mark.parametrize("first", [0, 5, 16, 40])
def test_outputs_from_a_token_before(first):
    """Only one token of the chunk has an input: the outputs behind it are its share, decayed."""
    n, T = 32, 64
    g = torch.Generator().manual_seed(3)
    dt, A_log, bias, step, a = steps(g, n, T)
    A_log = A_log - 3  # exponents below 1 over the chunk
    a = a * torch.exp(torch.tensor(-3.0, dtype=torch.float64))
    B = torch.zeros(n, T, 1, S, dtype=BF, device="cuda")
    B[..., 3] = 1
    x = torch.zeros(n, T, H, P, dtype=BF)
    x[:, first] = positive(g, n, H, P).to(BF)
    y, _ = kda.ssm_fwd(x.cuda(), dt, B, B, A_log, bias)
    G = a.cumsum(1)
    want = torch.exp(G[:, first:] - G[:, first:first + 1])[..., None] * (step[:, first, :, None] * R.d(x)[:, first])[:, None]
    assert (y[:, :first] == 0).all()
    check_once(y[:, first:], want, "outputs from token %d" % first)


def test_gradients_from_the_token():
    """T = 1, no state: dx = dt dy (one-hot B = C), dB = dC = dt dy_p x_p C (one-hot x)."""
    g = torch.Generator().manual_seed(4)
    dt, A_log, bias, step, _ = steps(g)
    C, _ = hot(g, N, 1, S)
    dy = positive(g, N, 1, H, P).to(BF)
    x = torch.ones(N, 1, H, P, dtype=BF, device="cuda")
    got = kda.ssm_bwd(x, dt, C, C, A_log, bias, None, dy.cuda())
    check_once(got["dx"], step[..., None] * R.d(dy), "dx")
    # one head for dB and dC, which sum over heads and channels
    xs, at = hot(g, N, 1, P)
    C = positive(g, N, 1, 1, S).to(BF)
    one = [t[..., :1].contiguous() for t in (dt, A_log, bias)]
    got = kda.ssm_bwd(xs, one[0], C.cuda(), C.cuda(), one[1], one[2], None, dy[:, :, :1].contiguous().cuda())
    w = step[..., :1] * R.d(dy)[:, :, 0].gather(2, at.view(N, 1, 1))
    for k in ("dB", "dC"):
        check_once(got[k], w[..., None] * R.d(C), k)


def test_gradients_from_the_states():
    """T = 1, dy = 0: dx = dt D B (one-hot B), dB = dt D^T x (one-hot x); and dC = e^a S^T dy (one-hot dy, B = 0)."""
    g = torch.Generator().manual_seed(5)
    dt, A_log, bias, step, a = steps(g)
    B, at = hot(g, N, 1, S)
    dfin = positive(g, N, H, P, S)
    none = torch.zeros(N, 1, H, P, dtype=BF, device="cuda")
    got = kda.ssm_bwd(torch.ones_like(none), dt, B, torch.zeros_like(B), A_log, bias, None, none, d_final_state=dfin.cuda())
    entry = R.d(dfin).gather(3, at.view(N, 1, 1, 1).expand(N, H, P, 1))[..., 0]
    check_once(got["dx"][:, 0], step[:, 0, :, None] * entry, "dx")
    xs, at = hot(g, N, 1, P)
    one = [t[..., :1].contiguous() for t in (dt, A_log, bias)]
    row = lambda t: R.d(t)[:, 0].gather(1, at.view(N, 1, 1).expand(N, 1, S))[:, 0]  # noqa: E731
    got = kda.ssm_bwd(xs, one[0], B, torch.zeros_like(B), one[1], one[2], None, none[:, :, :1].contiguous(),
                      d_final_state=dfin[:, :1].contiguous().cuda())
    check_once(got["dB"][:, 0, 0], step[:, 0, :1] * row(dfin), "dB")
    got = kda.ssm_bwd(none[:, :, :1].contiguous(), one[0], torch.zeros_like(B), B, one[1], one[2], None, xs,
                      initial_state=dfin[:, :1].contiguous().cuda())
    check_once(got["dC"][:, 0, 0], torch.exp(a[:, 0, :1]) * row(dfin), "dC")
