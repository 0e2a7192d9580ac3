"""The selective state-space scan against its recurrence in 64 bits: prompts,
packed batches, one-token steps, states, pieces, gradients."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ARGS = ("x", "dt", "B", "C", "A_log", "dt_bias", "D")


def make(B, T, H, P, G, S, N, state=None, seed=0, params=True, dt_scale=1.0):
    """x, B and C are slices of one tensor, as a convolution over all three leaves them."""
    g = torch.Generator().manual_seed(seed + T * 31 + H * 7 + S)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    xbc = n(B, T, H * P + 2 * G * S).to(BF).cuda()
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    a = {"x": xbc[..., :H * P].unflatten(-1, (H, P)), "dt": (dt_scale * n(B, T, H)).to(BF).cuda(),
         "B": xbc[..., H * P:H * P + G * S].unflatten(-1, (G, S)), "C": xbc[..., H * P + G * S:].unflatten(-1, (G, S)),
         "A_log": torch.log(1 + 15 * torch.rand(H, generator=g)).cuda(),
         "dt_bias": (step + torch.log(-torch.expm1(-step))).cuda() if params else None,
         "D": (1 + 0.1 * n(H)).cuda() if params else None}
    s = None if state is None else (0.5 * n(N, H, P, S)).to(state).cuda()
    return a, s


def ref(a, s, lens, M=None):
    M = sum(lens)
    f = lambda k: None if a[k] is None else R.d(a[k])  # noqa: E731
    t = lambda k: f(k).reshape(-1, *a[k].shape[2:])[:M]  # noqa: E731
    return R.scan(t("x"), t("dt"), t("B"), t("C"), f("A_log"), f("dt_bias"), f("D"), R.d(s), lens)


def sizes(a, s, lens):
    """The same sums over magnitudes: what a rounding inside is relative to."""
    b = {k: v if k in ("dt", "A_log", "dt_bias") or v is None else v.abs() for k, v in a.items()}
    return ref(b, None if s is None else s.abs(), lens)


# Within the scan every product is exact to fp32 or better and every decay's
# exponent, a sum of up to 64 fp32 terms, to some 2^-24 of its magnitude; decays that
# matter (above e^-16) have exponents below 16, and a state passes a chunk's end per
# 64 tokens: 128 half steps of the magnitudes' sum cover them.
REL = 128 * R.U


def check(a, s, lens, y, fin, label, out_dtype=BF):
    H, P = a["x"].shape[2:]
    yr, fr = ref(a, s, lens)
    ys, fs = sizes(a, s, lens)
    M = sum(lens)
    R.check(y.reshape(-1, H, P)[:M], yr, out_dtype, REL * ys, label + " y")
    if fin is not None:
        R.check(fin, fr, fin.dtype, REL * fs, label + " state")


@pytest.mark.parametrize("N,H,P,G,S,state", [(1, 1, 64, 1, 64, F32), (3, 4, 64, 2, 128, BF), (5, 3, 128, 1, 64, F32),
                                              (2, 8, 128, 8, 128, None), (70, 5, 64, 1, 128, F32)])
def test_decode(N, H, P, G, S, state):
    a, s = make(N, 1, H, P, G, S, N, state, seed=1, params=H != 3)
    say("case ssm decode N=%d H=%d P=%d G=%d S=%d state %s" % (N, H, P, G, S, state))
    fin = torch.full((N, H, P, S), float("nan"), dtype=state or F32, device="cuda")
    y, _ = kda.ssm_decode(*a.values(), initial_state=s, final_state=fin)
    torch.cuda.synchronize()
    check(a, s, [1] * N, y, fin, "decode")
    if s is not None:
        st = s.clone()
        y2, _ = kda.ssm_decode(*a.values(), initial_state=st, final_state=st)
        assert torch.equal(y2, y) and torch.equal(st, fin)


def test_decode_extremes():
    """Step sizes from far below to far above one: no overflow, the state replaced or kept."""
    a, s = make(4, 1, 2, 64, 1, 64, 4, F32, seed=2, params=False)
    a["dt"][0], a["dt"][1], a["dt"][2], a["dt"][3] = -100.0, -20.0, 30.0, 100.0
    fin = torch.empty_like(s)
    y, _ = kda.ssm_decode(*a.values(), initial_state=s, final_state=fin)
    check(a, s, [1] * 4, y, fin, "decode extremes")
    assert torch.equal(fin[0], s[0])


def test_decode_refusals():
    a, s = make(2, 1, 2, 64, 1, 64, 2, F32)
    v = list(a.values())
    for bad in (lambda: kda.ssm_decode(*v, initial_state=s), lambda: kda.ssm_decode(v[0].float(), *v[1:], final_state=s),
                lambda: kda.ssm_decode(v[0][..., :32], *v[1:], final_state=s[:, :, :32]),
                lambda: kda.ssm_decode(*v, initial_state=s, final_state=s.to(BF)[:1]),
                lambda: kda.ssm_decode(*v[:4], v[4].to(BF), final_state=s),
                lambda: kda.ssm_decode(*v, final_state=s, out=v[0]),
                lambda: kda.ssm_decode(v[0].repeat(1, 2, 1, 1), *v[1:], final_state=s)):
        with pytest.raises(ValueError):
            bad()
