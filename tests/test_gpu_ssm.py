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


@pytest.mark.parametrize("step", [True, False])
def test_small_step_sizes_keep_their_precision(step):
    """With x = B = 1 the state after one token is dt = softplus(dt_bias) itself.  Its roundings: the
    hardware's exp2 and reciprocal are good to 2^-23, the sums and products between them and the state's
    own products round six times at 2^-24, and log1p's relative change is at most 1.1 times its
    argument's (z = 1/3): 6.5 * 2^-23 in all, below 8 * 2^-23."""
    H, P, S = 61, 64, 64
    bias = torch.linspace(-14, 16, H)
    x = torch.ones(1, 1, H, P, dtype=BF, device="cuda")
    bc = torch.ones(1, 1, 1, S, dtype=BF, device="cuda")
    fin = torch.empty(1, H, P, S, dtype=F32, device="cuda")
    (kda.ssm_decode if step else kda.ssm_fwd)(x, torch.zeros(1, 1, H, dtype=BF, device="cuda"), bc, bc,
                                              torch.zeros(H, device="cuda"), bias.cuda(), final_state=fin)
    want = torch.nn.functional.softplus(bias.double(), threshold=100)[None, :, None, None]
    assert float(((fin.double().cpu() - want).abs() / want).max()) <= 8 * 2.0 ** -23


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


# ---- gradient ----

def ref_grads(a, s, lens, dy, dfin, absolute=False):
    """Gradients in 64 bits, or (absolute) the same sums over magnitudes."""
    M = sum(lens)
    mag = (lambda t: t.abs()) if absolute else (lambda t: t)
    leaves = {}
    for k in ARGS:
        t = None if a[k] is None else R.d(a[k])
        if t is not None and k in ("x", "dt", "B", "C"):
            t = t.reshape(-1, *t.shape[2:])[:M]
        leaves[k] = None if t is None else (t if k in ("dt", "A_log", "dt_bias") else mag(t)).requires_grad_()
    h = None if s is None else mag(R.d(s)).requires_grad_()
    y, fin = R.scan(*leaves.values(), h, lens)
    H, P = a["x"].shape[2:]
    loss = (y * mag(R.d(dy)).reshape(-1, H, P)[:M]).sum()
    if dfin is not None:
        loss = loss + (fin * mag(R.d(dfin))).sum()
    return dict(zip(("dx", "ddt", "dB", "dC", "dA_log", "ddt_bias", "dD", "d_initial_state"),
                    R.grads(loss, list(leaves.values()) + [h])))


def step_grad_sizes(a, s, lens, dy, dfin):
    """Sizes for ddt, dA_log and ddt_bias: the gradients of dt as the scale of the sums of both signs that
    make them, from the magnitudes' loss with the decay's and the input's share of every step taken apart."""
    M = sum(lens)
    H, P = a["x"].shape[2:]
    f = lambda k: R.d(a[k]).reshape(-1, *a[k].shape[2:])[:M]  # noqa: E731
    raw = f("dt") + (0 if a["dt_bias"] is None else R.d(a["dt_bias"]))
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A = torch.exp(R.d(a["A_log"]))
    # u multiplies the input, e^l the decay: both with positive gradients
    u, l = step.clone().requires_grad_(), (-A * step).requires_grad_()
    x, B, C = f("x").abs(), f("B").abs(), f("C").abs()
    G = B.shape[1]
    Bh, Ch = (t.repeat_interleave(H // G, 1) for t in (B, C))
    at, ys, fins = R.bounds(lens), [], []
    for n, k in enumerate(lens):
        st = torch.zeros(H, P, B.shape[-1], dtype=torch.float64) if s is None else R.d(s)[n].abs()
        for t in range(at[n], at[n] + k):
            st = torch.exp(l[t])[:, None, None] * st + (u[t][:, None] * x[t])[:, :, None] * Bh[t][:, None, :]
            ys.append((st * Ch[t][:, None, :]).sum(-1))
        fins.append(st)
    loss = (torch.stack(ys) * R.d(dy).abs().reshape(-1, H, P)[:M]).sum() if ys else torch.zeros((), dtype=torch.float64)
    if dfin is not None:
        loss = loss + (torch.stack(fins) * R.d(dfin).abs()).sum()
    gu, gl = R.grads(loss, [u, l])
    per = (gu + A * gl) * torch.sigmoid(raw)
    # pairs of tokens of one chunk behind t appear in its sums with both signs: rounded 24
    # bits down, they leave 16 half steps of their size, which the chunk's gl add up to
    pairs = torch.zeros_like(gl)
    for n, k in enumerate(lens):
        for c in range(at[n], at[n] + k, 64):
            e = min(c + 64, at[n] + k)
            pairs[c:e] = gl[c:e].sum(0)
    extra = 16 * R.U * A * pairs * torch.sigmoid(raw) / GREL
    return {"ddt": per + extra, "ddt_bias": (per + extra).sum(0), "dA_log": ((gl + 16 * R.U * pairs / GREL) * A * step).sum(0)}


# The states and their gradients enter the products rounded to two bf16 parts (2^-17
# relative), and so do M and W: 4 such roundings at most meet in one result, beside
# the fp32 sums (REL).
GREL = 4 * 2.0 ** -17 + REL


def check_bwd(a, s, lens, dy, dfin, g, rel=GREL):
    M = sum(lens)
    want, size = ref_grads(a, s, lens, dy, dfin), ref_grads(a, s, lens, dy, dfin, True)
    size.update(step_grad_sizes(a, s, lens, dy, dfin))
    for k, v in want.items():
        if v is None:
            assert g[k] is None, k
            continue
        got = g[k]
        if k in ("dx", "ddt", "dB", "dC"):
            got = got.reshape(-1, *got.shape[2:])[:M]
        R.check(got, v, got.dtype, rel * size[k].abs(), k)


def loss_grads(a, s, N, seed):
    g = torch.Generator().manual_seed(seed)
    B, T, H, P = a["x"].shape
    dy = torch.randn(B, T, H, P, generator=g).to(BF).cuda()
    dfin = torch.randn(N, H, P, a["B"].shape[-1], generator=g).to(F32 if s is None else s.dtype).cuda()
    return dy, dfin


@pytest.mark.parametrize("B,T,H,P,G,S,state", CASES)
@pytest.mark.parametrize("pc", [0, 1])
def test_bwd_batches(B, T, H, P, G, S, state, pc):
    T = min(T, 330)
    a, s = make(B, T, H, P, G, S, B, state, seed=23, params=H != 3)
    dy, dfin = loss_grads(a, s, B, 24)
    say("case ssm bwd %s state %s pieces of %d" % ((B, T, H, P, G, S), state, pc))
    g = kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, piece_chunks=pc)
    torch.cuda.synchronize()
    check_bwd(a, s, [T] * B, dy, dfin, g)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,P,G,S,state", [(2, 64, 1, 64, F32), (4, 128, 2, 128, BF), (3, 64, 1, 128, None)])
def test_bwd_packed(lens, H, P, G, S, state):
    tail = 7
    T, N = sum(lens) + tail, len(lens)
    a, s = make(1, T, H, P, G, S, N, state, seed=25)
    dy, dfin = loss_grads(a, s, N, 26)
    for t in (a["x"], a["dt"], a["B"], a["C"], dy):
        t[0, T - tail:] = float("nan")
    say("case ssm bwd packed %s %s" % (lens, (H, P, G, S)))
    outs = {k: torch.full(t.shape, 7.0, dtype=BF, device="cuda") for k, t in
            (("dx", a["x"]), ("ddt", a["dt"]), ("dB", a["B"]), ("dC", a["C"]))}
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    g = kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, cu_seqlens=cu, outputs=outs, piece_chunks=1)
    torch.cuda.synchronize()
    for t in outs.values():
        assert (t[0, T - tail:] == 7.0).all()
    check_bwd(a, s, lens, dy, dfin, g)


def test_bwd_shares_of_heads():
    """Few chunks and many heads in a group: several workgroups add to one dB and dC; no d_final, no initial state."""
    for T, H, G in ((70, 12, 1), (64 * 9, 10, 2)):
        a, s = make(1, T, H, 64, G, 64, 1, None, seed=27)
        dy, _ = loss_grads(a, s, 1, 28)
        g = kda.ssm_bwd(*a.values(), dy)
        torch.cuda.synchronize()
        check_bwd(a, s, [T], dy, None, g)


def test_bwd_strided_d_out():
    a, s = make(2, 70, 2, 64, 1, 64, 2, None, seed=29)
    dy, _ = loss_grads(a, s, 2, 30)
    wide = torch.cat([dy, dy], -1)[..., 64:]
    with pytest.raises(ValueError):
        kda.ssm_bwd(*a.values(), wide)
    wide = torch.cat([dy, dy], 2)[:, :, 2:]
    g, h = kda.ssm_bwd(*a.values(), wide), kda.ssm_bwd(*a.values(), dy)
    for k in g:
        assert (g[k] is None and h[k] is None) or torch.equal(g[k], h[k]), k


def test_bwd_no_tokens():
    a, s = make(2, 0, 2, 64, 1, 64, 2, F32)
    dy, dfin = loss_grads(a, s, 2, 31)
    g = kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s)
    assert torch.equal(g["d_initial_state"], dfin)
    for k in ("dA_log", "ddt_bias", "dD"):
        assert (g[k] == 0).all()


def test_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    args = [n(9, 2, 3), n(9, 2), n(9, 1, 4), n(9, 1, 4), 0.3 * n(2), n(2), n(2), n(2, 2, 3, 4)]
    c, cf = n(9, 2, 3), n(2, 2, 3, 4)

    def f(i, t):
        v = list(args)
        v[i] = t
        y, fin = R.scan(*v, [4, 5])
        return (y * c).sum() + (fin * cf).sum()
    for i in range(8):
        leaf, v = args[i].clone().requires_grad_(), n(*args[i].shape)
        g = torch.autograd.grad(f(i, leaf), leaf)[0]
        want = float(R.difference(lambda t: f(i, t), args[i], v))
        assert abs(float((g * v).sum()) - want) <= 1e-6 * (1 + abs(want)), i


def test_bwd_graph_and_autograd():
    lens = [100, 0, 29]
    a, s = make(1, 140, 4, 64, 2, 128, 3, F32, seed=33)
    dy, dfin = loss_grads(a, s, 3, 34)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    leaves = {k: v.detach().clone().requires_grad_() for k, v in a.items()}
    ls = s.clone().requires_grad_()
    y, fin = kda.ssm_scan(*leaves.values(), initial_state=ls, final_state_dtype=F32, cu_seqlens=cu)
    assert (y[0, 129:] == 0).all()
    ((y * dy).sum() + (fin * dfin).sum()).backward()
    want = kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, cu_seqlens=cu,
                       outputs={k: torch.zeros(t.shape, dtype=BF, device="cuda") for k, t in
                                (("dx", a["x"]), ("ddt", a["dt"]), ("dB", a["B"]), ("dC", a["C"]))})
    for k, leaf in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dA_log", "A_log"), ("ddt_bias", "dt_bias"), ("dD", "D")):
        assert torch.equal(leaves[leaf].grad, want[k]), k
    assert torch.equal(ls.grad, want["d_initial_state"])
    ws = torch.empty(kda.ssm_bwd_workspace_size(1, 140, 4, 64, 2, 128, 3), dtype=torch.uint8, device="cuda")
    outs = {k: torch.zeros_like(v) for k, v in want.items()}

    def call():
        kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, cu_seqlens=cu, workspace=ws, outputs=outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        for t in outs.values():
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in outs.items():
            assert torch.equal(v, want[k]), (rep, k)


def test_a_training_and_a_generation_step_together():
    """The operators as a layer uses them: norm with residual, convolution, scan, backwards through all three;
    then a prompt's states taken on by single tokens."""
    H, P, G, S, D = 2, 64, 1, 64, 2 * 64 + 2 * 64
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, res = n(1, 90, D).to(BF).cuda(), n(1, 90, D).cuda()
    nw, cw, cb = (1 + 0.1 * n(D)).cuda(), (0.5 * n(D, 4)).cuda(), (0.1 * n(D)).cuda()
    dt, A_log = n(1, 90, H).to(BF).cuda(), torch.log(1 + 15 * torch.rand(H, generator=gen)).cuda()
    dtb, Dp, dy = (0.5 * n(H) - 3).cuda(), n(H).cuda(), n(1, 90, H, P).to(BF).cuda()
    cu = torch.tensor([0, 33, 90], device="cuda")
    leaves = [t.requires_grad_() for t in (x, res, nw, cw, cb, dt, A_log, dtb, Dp)]

    def layer(x, res, nw, cw, cb, dt, A_log, dtb, Dp):
        y, h = kda.rms_norm(x, nw, 1e-5, residual=res)
        c, cfin = kda.short_conv(y, cw, cb, "silu", final_state_dtype=F32, cu_seqlens=cu)
        xs, Bm, Cm = c.split([H * P, G * S, G * S], -1)
        o, sfin = kda.ssm_scan(xs.unflatten(-1, (H, P)), dt, Bm.unflatten(-1, (G, S)), Cm.unflatten(-1, (G, S)), A_log, dtb, Dp,
                               final_state_dtype=F32, cu_seqlens=cu)
        return o, h, cfin, sfin
    o, h, cfin, sfin = layer(*leaves)
    ((o * dy).sum() + h.sum()).backward()

    def plain(x, res, nw, cw, cb, dt, A_log, dtb, Dp):
        y, h = R.rmsnorm(x, nw, 1e-5, res)
        c, cfin = R.conv(y[0], cw, cb, "silu", None, [33, 57])
        xs, Bm, Cm = c.split([H * P, G * S, G * S], -1)
        o, sfin = R.scan(xs.unflatten(-1, (H, P)), dt[0], Bm.unflatten(-1, (G, S)), Cm.unflatten(-1, (G, S)), A_log, dtb, Dp,
                         None, [33, 57])
        return o, h, cfin, sfin
    rl = [R.d(t).requires_grad_() for t in leaves]
    ro, rh, rc, rs = plain(*rl)
    grads = R.grads((ro * R.d(dy)[0]).sum() + rh.sum(), rl)
    # the operators hand bf16 tensors on: two roundings (2^-8 each at most, together about
    # 2^-8 in the mean) before the scan's products, three on the way back
    R.check_norm(o[0], ro.detach(), 3 * 2.0 ** -8, "output")
    R.check_norm(sfin, rs.detach(), 3 * 2.0 ** -8, "state")
    R.check_norm(cfin, rc.detach(), 2 * 2.0 ** -8, "convolution state")
    for name, t, g in zip(("x", "res", "nw", "cw", "cb", "dt", "A_log", "dtb", "D"), leaves, grads):
        R.check_norm(t.grad, g, 6 * 2.0 ** -8, "gradient of " + name)
    # generation: one more token for both sequences, against a prompt one token longer
    with torch.no_grad():
        tok = n(2, 1, D).to(BF).cuda()
        y, _ = kda.rmsnorm_fwd(tok, nw, 1e-5)
        cs, ss = cfin.detach().clone(), sfin.detach().clone()
        c, _ = kda.conv_decode(y, cw, cb, "silu", initial_state=cs, final_state=cs)
        xs, Bm, Cm = c.split([H * P, G * S, G * S], -1)
        one = n(2, 1, H).to(BF).cuda()
        o1, _ = kda.ssm_decode(xs.unflatten(-1, (H, P)), one, Bm.unflatten(-1, (G, S)), Cm.unflatten(-1, (G, S)), A_log, dtb, Dp,
                               initial_state=ss, final_state=ss)
        rc1, rcf = R.conv(R.d(y).reshape(2, D), R.d(cw), R.d(cb), "silu", R.d(cfin), [1, 1])
        assert torch.equal(R.d(cs), rcf)
        xs, Bm, Cm = R.d(c).reshape(2, D).split([H * P, G * S, G * S], -1)
        ro1, rs1 = R.scan(xs.unflatten(-1, (H, P)), R.d(one)[:, 0], Bm.unflatten(-1, (G, S)), Cm.unflatten(-1, (G, S)),
                          R.d(A_log), R.d(dtb), R.d(Dp), R.d(sfin), [1, 1])
        R.check_norm(c.reshape(2, D), rc1, 2.0 ** -8, "one token's convolution")
        R.check_norm(o1[:, 0], ro1, 2.0 ** -8, "one token's output")
        R.check_norm(ss, rs1, 2.0 ** -20, "state after it")


@pytest.mark.parametrize("lens", [[64 * 15, 64 * 16, 64 * 17 - 3], [64 * 24, 64 * 31 + 1], [64 * 33, 5, 64 * 8]])
def test_many_pieces(lens):
    """The join of the pieces' states at counts around its batches of 8 and 16, against one piece per sequence."""
    H, P, S = 2, 64, 64
    T, N = sum(lens), len(lens)
    a, s = make(1, T, H, P, 1, S, N, F32, seed=41)
    dy, dfin = loss_grads(a, s, N, 42)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    say("case ssm pieces of one chunk, lengths %s" % lens)
    got, fin = [], []
    for pc in (1, 1 << 20):
        f = torch.empty_like(s)
        y, _ = kda.ssm_fwd(*a.values(), initial_state=s, final_state=f, cu_seqlens=cu, piece_chunks=pc)
        g = kda.ssm_bwd(*a.values(), dy, d_final_state=dfin, initial_state=s, cu_seqlens=cu, piece_chunks=pc)
        torch.cuda.synchronize()
        got.append(y.float())
        fin.append((f, g["d_initial_state"], g["dx"].float()))
    # the joins round each state once more per piece, in fp32, and the decays before it shrink what they round:
    # within REL of the states, and one rounding to bf16 (two halves) of the outputs
    for p, q in zip(fin[0][:2], fin[1][:2]):
        assert float((p - q).norm()) <= REL * float(q.norm())
    for p, q in ((got[0], got[1]), (fin[0][2], fin[1][2])):
        assert float((p - q).abs().max()) <= (2.0 ** -8 + GREL) * float(q.abs().max())
