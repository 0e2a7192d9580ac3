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


CASES = [(1, 1, 2, 64, 1, 64, None), (2, 63, 4, 64, 2, 128, BF), (1, 64, 3, 128, 1, 64, F32), (3, 65, 2, 64, 2, 128, F32),
         (1, 130, 8, 64, 8, 64, None), (2, 200, 6, 128, 2, 128, BF), (1, 1000, 2, 64, 1, 128, F32)]
LENS = [[5], [1, 0, 2, 17, 64], [0, 0, 133, 1, 1, 65, 0], [300, 3, 64, 0, 128], [0], [2] * 20]


@pytest.mark.parametrize("B,T,H,P,G,S,state", CASES)
@pytest.mark.parametrize("pc", [0, 1, 2])
def test_fwd_batches(B, T, H, P, G, S, state, pc):
    a, s = make(B, T, H, P, G, S, B, state, seed=3, params=H != 3)
    say("case ssm %s state %s pieces of %d" % ((B, T, H, P, G, S), state, pc))
    fin = torch.full((B, H, P, S), float("nan"), dtype=state or F32, device="cuda")
    y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=fin, piece_chunks=pc)
    torch.cuda.synchronize()
    check(a, s, [T] * B, y, fin, "ssm")


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,P,G,S,state", [(2, 64, 1, 64, F32), (4, 128, 2, 128, BF), (1, 64, 1, 128, None)])
@pytest.mark.parametrize("pc", [0, 1])
def test_fwd_packed(lens, H, P, G, S, state, pc):
    tail = 7
    T, N = sum(lens) + tail, len(lens)
    a, s = make(1, T, H, P, G, S, N, state, seed=4)
    for k in ("x", "dt", "B", "C"):   # what stands behind the last sequence reaches nothing
        a[k][0, T - tail:] = float("nan")
    say("case ssm packed %s %s pieces of %d" % (lens, (H, P, G, S), pc))
    out = torch.full((1, T, H, P), 7.0, dtype=BF, device="cuda")
    fin = torch.full((N, H, P, S), float("nan"), dtype=F32, device="cuda")
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    kda.ssm_fwd(*a.values(), initial_state=s, final_state=fin, cu_seqlens=cu, out=out, piece_chunks=pc)
    torch.cuda.synchronize()
    assert (out[0, T - tail:] == 7.0).all()
    check(a, s, lens, out, fin, "ssm packed")


def test_state_in_place_and_steps():
    """A prompt cut in two, and token by token, continues from the state as it does in one piece."""
    a, s = make(2, 150, 4, 64, 2, 64, 2, F32, seed=5)
    lens = [150, 150]
    for cut in (1, 64, 100):
        st = s.clone()
        first = {k: v[:, :cut] if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
        rest = {k: v[:, cut:] if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
        y1, _ = kda.ssm_fwd(*first.values(), initial_state=st, final_state=st, piece_chunks=1)
        y2, _ = kda.ssm_fwd(*rest.values(), initial_state=st, final_state=st, piece_chunks=1)
        check(a, s, lens, torch.cat([y1, y2], 1), st, "cut at %d" % cut)
    st, ys = s.clone(), []
    for t in range(20):
        one = {k: v[:, t:t + 1] if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
        y, _ = kda.ssm_decode(*one.values(), initial_state=st, final_state=st)
        ys.append(y)
    head = {k: v[:, :20] if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
    check(head, s, [20, 20], torch.cat(ys, 1), st, "steps")


def test_decay_extremes():
    """Step sizes from none to ones that empty the state at once, within one chunk."""
    a, s = make(1, 200, 2, 64, 1, 64, 1, F32, seed=6, dt_scale=12.0)
    fin = torch.empty_like(s)
    y, _ = kda.ssm_fwd(*a.values(), initial_state=s, final_state=fin, piece_chunks=1)
    torch.cuda.synchronize()
    assert torch.isfinite(y.float()).all() and torch.isfinite(fin).all()
    yr, fr = ref(a, s, [200])
    # exponents up to some hundreds here: each decay is good to 2^-24 of its exponent
    ys, fs = sizes(a, s, [200])
    R.check(y[0], yr, BF, 2048 * R.U * ys, "y")
    R.check(fin, fr, F32, 2048 * R.U * fs, "state")


def test_no_tokens():
    a, s = make(2, 0, 2, 64, 1, 64, 2, BF)
    y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s))
    assert y.shape == (2, 0, 2, 64) and torch.equal(fin, s)
    y, fin = kda.ssm_fwd(*a.values(), final_state=torch.full_like(s, 3.0))
    assert (fin == 0).all()


def test_other_sequences_are_left_alone_by_nan():
    lens = [70, 70, 70]
    a, s = make(1, 210, 2, 64, 1, 64, 3, None, seed=7)
    a["x"][0, 100, 0, 5] = float("nan")
    a["B"][0, 101] = float("inf")
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    y, _ = kda.ssm_fwd(*a.values(), cu_seqlens=cu, piece_chunks=1)
    assert torch.isfinite(y[0, :70].float()).all() and torch.isfinite(y[0, 140:].float()).all()
    assert not torch.isfinite(y[0, 101:140].float()).all()


def test_wrong_lengths_stay_inside():
    """Contents of cu_seqlens that no batch has: clamped on the device, nothing outside the tensors is touched."""
    a, _ = make(1, 100, 2, 64, 1, 64, 3, None, seed=8)
    out = torch.zeros(3, 100, 2, 64, dtype=BF, device="cuda")  # the call's output is the middle one
    for cu in ([0, -5, 1000, 50], [70, 20, 90, 30], [0, 1 << 40, 5, 1 << 50], [0, 100] * 20, [100, 0] * 20):
        kda.ssm_fwd(*a.values(), cu_seqlens=torch.tensor(cu, device="cuda"), out=out[1:2], piece_chunks=1)
        torch.cuda.synchronize()
        assert (out[0] == 0).all() and (out[2] == 0).all()


def test_fwd_graph():
    lens = [100, 0, 29, 200]
    a, s = make(1, 340, 4, 64, 2, 128, 4, F32, seed=9)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    ws = torch.empty(kda.ssm_workspace_size(1, 340, 4, 64, 2, 128, 4, 1), dtype=torch.uint8, device="cuda")
    out, fin = torch.zeros(1, 340, 4, 64, dtype=BF, device="cuda"), torch.empty_like(s)

    def call():
        kda.ssm_fwd(*a.values(), initial_state=s, final_state=fin, cu_seqlens=cu, out=out, workspace=ws, piece_chunks=1)
    call()
    torch.cuda.synchronize()
    want = out.clone(), fin.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        out.zero_(), fin.zero_(), ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(fin, want[1]), rep


def test_fwd_refusals():
    a, s = make(2, 10, 4, 64, 2, 64, 2, F32)
    v = list(a.values())
    cu = torch.tensor([0, 10], device="cuda")
    for bad in (lambda: kda.ssm_fwd(v[0].float(), *v[1:]), lambda: kda.ssm_fwd(v[0][:, :5], *v[1:]),
                lambda: kda.ssm_fwd(v[0][:, :, :3], v[1][:, :, :3], *v[2:]), lambda: kda.ssm_fwd(*v, cu_seqlens=cu),
                lambda: kda.ssm_fwd(v[0][..., :32], *v[1:]), lambda: kda.ssm_fwd(*v, out=v[0]),
                lambda: kda.ssm_fwd(*v, initial_state=s, final_state=s[:1]), lambda: kda.ssm_fwd(*v, piece_chunks=-1),
                lambda: kda.ssm_fwd(v[0], v[1], v[2][..., 1:], v[3][..., 1:], *v[4:]),
                lambda: kda.ssm_fwd(*v[:4], v[4].double(), *v[5:])):
        with pytest.raises(ValueError):
            bad()
