"""The scan's fp32 gradients (A_log, dt_bias, D, initial state) and its step sizes' to fp32: the
states and their gradients enter in three bf16 parts, and no sum of pairs of tokens cancels that
the formula does not have."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say
from tests.test_gpu_ssm import CASES, LENS, loss_grads, make, ref_grads
from tests.test_gpu_ssm_precision import half_step, hot, positive

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# Half steps of fp32 (2^-24, relative) in a term of these sums: its decay 2, and 25 times its
# exponent (a step size 16, exp(A_log) 8, their product 1), which with the decay itself is 9 at most
# far away and 25 at an exponent of 1; a step size before and one behind the sum 16 each, A 8,
# softplus's slope 8; three products deep on the matrix cores 12 each, their operands' parts 4; the
# states' sums over up to 8 chunks and pieces 16; the rest is joined in 64 bits.  140 in all.
REL = 144 * R.U


def magnitudes(a, s, lens, dy, dfin):
    """Sums over magnitudes of what the formulas add: of u, which multiplies a token's input, and of l, the
    logarithm of its decay; per token and head."""
    M = sum(lens)
    H, P = a["x"].shape[2:]
    f = lambda k: R.d(a[k]).reshape(-1, *a[k].shape[2:])[:M]  # noqa: E731
    raw = f("dt") + (0 if a["dt_bias"] is None else R.d(a["dt_bias"]))
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A = torch.exp(R.d(a["A_log"]))
    u, l = step.clone().requires_grad_(), (-A * step).requires_grad_()
    x = f("x").abs()
    B, C = (f(k).abs().repeat_interleave(H // a[k].shape[2], 1) for k in ("B", "C"))
    at, ys, fins = R.bounds(lens), [], []
    for n, k in enumerate(lens):
        st = torch.zeros(H, P, B.shape[-1], dtype=torch.float64) if s is None else R.d(s)[n].abs()
        for t in range(at[n], at[n] + k):
            st = torch.exp(l[t])[:, None, None] * st + (u[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            ys.append((st * C[t][:, None, :]).sum(-1))
        fins.append(st)
    loss = (torch.stack(ys) * R.d(dy).abs().reshape(-1, H, P)[:M]).sum() if ys else torch.zeros((), dtype=torch.float64)
    if dfin is not None:
        loss = loss + (torch.stack(fins) * R.d(dfin).abs()).sum()
    gu, gl = R.grads(loss, [u, l])
    slope = torch.sigmoid(raw)
    return {"ddt": (gu + A * gl) * slope, "ddt_bias": ((gu + A * gl) * slope).sum(0), "dA_log": (gl * A * step).sum(0)}


def check(a, s, lens, dy, dfin, g):
    want, size = ref_grads(a, s, lens, dy, dfin), ref_grads(a, s, lens, dy, dfin, True)
    size.update(magnitudes(a, s, lens, dy, dfin))
    for k in ("dA_log", "ddt_bias", "dD", "d_initial_state"):
        if want[k] is not None:
            off = ((R.d(g[k]) - want[k]).abs() / size[k].abs().clamp(min=1e-300)).max() if want[k].numel() else 0.0
            say("%s off by %.3g of %.3g" % (k, float(off), REL))
            R.check(g[k], want[k], F32, REL * size[k].abs(), k)


@pytest.mark.parametrize("B,T,H,P,G,S,state", CASES + [(1, 12, 1, 64, 1, 64, None), (1, 63, 2, 64, 1, 128, F32), (1, 12, 8, 64, 1, 64, F32)])
@pytest.mark.parametrize("pc", [0, 1])
def test_batches(B, T, H, P, G, S, state, pc):
    T = min(T, 330)
    a, s = make(B, T, H, P, G, S, B, state, seed=41, params=H != 3)
    dy, dfin = loss_grads(a, s, B, 42)
    say("case ssm bwd precision %s state %s pieces of %d" % ((B, T, H, P, G, S), state, pc))
    check(a, s, [T] * B, dy, dfin, kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, piece_chunks=pc))


@pytest.mark.parametrize("lens", LENS)
def test_packed(lens):
    a, s = make(1, sum(lens), 4, 128, 2, 128, len(lens), F32, seed=43)
    dy, dfin = loss_grads(a, s, len(lens), 44)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    say("case ssm bwd precision packed %s" % lens)
    check(a, s, lens, dy, dfin, kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, cu_seqlens=cu, piece_chunks=1))


def one_token(g, H, P):
    A_log, bias = torch.log(positive(g, H)), torch.full((H,), -3.0)
    step = torch.nn.functional.softplus(R.d(bias), threshold=100)
    return torch.zeros(1, 1, H, dtype=BF, device="cuda"), A_log.cuda(), bias.cuda(), step, torch.exp(R.d(A_log))


def test_a_single_entry_of_the_state():
    """T = 1 and one nonzero product per head: dA_log is -A dt times the decayed entry of the state that C and dy
    point at, ddt_bias the slope times -A times it, or times the entry of the final state's gradient that B and x
    point at.  In half steps: A 8, dt 16, the decay 5, the parts and the product 14, slope 8, sums 8: below 64."""
    H, P, S = 512, 64, 64
    g = torch.Generator().manual_seed(5)
    dt, A_log, bias, step, A = one_token(g, H, P)
    vec, at = hot(g, 1, 1, S)
    chan = torch.randint(P, (H,), generator=g)
    point = torch.nn.functional.one_hot(chan, P).view(1, 1, H, P).to(BF).cuda()
    st = positive(g, 1, H, P, S)
    entry = R.d(st)[0, torch.arange(H), chan, int(at)]
    two = entry.to(BF).double() + (entry - entry.to(BF).double()).to(BF).double()
    assert ((two - entry).abs() > 80 * R.U * entry).any()  # what two bf16 parts would do to them
    none = torch.zeros_like(point)
    got = kda.ssm_bwd(none, dt, torch.zeros_like(vec), vec, A_log, bias, None, point, initial_state=st.cuda())
    slope = torch.sigmoid(R.d(bias))
    want = -A * torch.exp(-A * step) * entry
    R.check(got["dA_log"], want * step, F32, 64 * R.U * (want * step).abs(), "dA_log from the state")
    R.check(got["ddt_bias"], want * slope, F32, 64 * R.U * (want * slope).abs(), "ddt_bias from the state")
    got = kda.ssm_bwd(point, dt, vec, torch.zeros_like(vec), A_log, bias, None, none, d_final_state=st.cuda())
    R.check(got["ddt_bias"], entry * slope, F32, 64 * R.U * entry * slope, "ddt_bias from the state's gradient")
    assert (got["dA_log"] == 0).all()


@pytest.mark.parametrize("T", [12, 16, 40, 63])
def test_pairs_behind_a_token_do_not_reach_it(T):
    """Tokens 0 to 3, and those behind them with products 2^14 times as large that share no entry of the state with
    them: the step sizes' gradients of the first four are those of the four alone.  A sum that takes the pairs
    behind a token in and out again would lose 14 bits there."""
    n, H, P, S = 8, 16, 64, 64
    g = torch.Generator().manual_seed(6)
    a = {"x": positive(g, n, T, H, P), "dt": 0.3 * torch.randn(n, T, H, generator=g), "B": torch.zeros(n, T, 1, S),
         "C": torch.zeros(n, T, 1, S), "A_log": torch.log(1 + 3 * torch.rand(H, generator=g)), "dt_bias": torch.full((H,), -3.0), "D": None}
    dy = positive(g, n, T, H, P)
    a["x"][:, 4:] *= 128
    dy[:, 4:] *= 128
    for k in ("B", "C"):
        a[k][:, :4, 0, 3], a[k][:, 4:, 0, 40] = 1, 1
    a = {k: None if v is None else (v.to(BF) if k in ("x", "dt", "B", "C") else v).cuda() for k, v in a.items()}
    dy = dy.to(BF).cuda()
    got = R.d(kda.ssm_bwd(*a.values(), dy)["ddt"])[:, :4]
    four = {k: v[:, :4].contiguous() if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
    lens = [4] * n
    want = ref_grads(four, None, lens, dy[:, :4].contiguous(), None)["ddt"].view(n, 4, H)
    size = magnitudes(four, None, lens, dy[:, :4].contiguous(), None)["ddt"].view(n, 4, H)
    off = ((got - want).abs() - half_step(want)) / size
    say("T = %d: beyond half a step %.3g of %.3g" % (T, float(off.max()), REL))
    assert float(off.max()) <= REL
