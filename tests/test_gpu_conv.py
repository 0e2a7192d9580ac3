"""The short causal convolution against its formula in 64 bits: batches, packed
batches, states, odd channel counts, strides, one-token steps, gradients."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(B, T, D, W, N, state=None, bias=True, wdt=F32, seed=0, wide=0, off=0):
    g = torch.Generator().manual_seed(seed + T * 31 + D * 7 + W)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = n(B, T, D + wide).to(BF).cuda()[..., off:off + D]
    w = (0.5 * n(D, W)).to(wdt).cuda()
    b = (0.3 * n(D)).to(wdt).cuda() if bias else None
    s = None if state is None else n(N, W - 1, D).to(state).cuda()
    dy = n(B, T, D + wide).to(BF).cuda()[..., off:off + D]
    dfin = n(N, W - 1, D).to(state or F32).cuda()
    return x, w, b, s, dy, dfin


def cu_of(lens):
    return torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")


# W products and sums, the bias, and silu (Lipschitz constant below 1.1; its exp and
# reciprocal are good to a few half steps relative to the argument's size)
def slack(x, w, b, s, lens):
    size, _ = R.conv(x.abs(), w.abs(), None if b is None else b.abs(), None, None if s is None else s.abs(), lens)
    return 16 * R.U * size


CASES = [(1, 1, 8, 4, None), (2, 3, 64, 4, BF), (1, 17, 520, 4, F32), (3, 100, 77, 3, BF), (2, 33, 5, 2, F32), (2, 16, 2056, 4, None),
         (1, 250, 264, 3, None), (4, 2, 16, 4, F32), (1, 131, 1, 4, BF), (2, 65, 1024, 2, BF)]
LENS = [[5], [1, 0, 2, 17], [0, 0, 33, 1, 1, 1, 16, 0], [130, 3, 64, 0], [2, 2, 2, 2, 2, 2, 2, 2, 2, 2], [0], [3, 200]]


@pytest.mark.parametrize("B,T,D,W,state", CASES)
@pytest.mark.parametrize("act", [None, "silu"])
def test_fwd_batches(B, T, D, W, state, act):
    x, w, b, s, _, _ = make(B, T, D, W, B, state, bias=act is None or T % 2 == 0, wdt=BF if T % 3 == 0 else F32)
    say("case conv %s W=%d state %s" % ((B, T, D), W, state))
    fin = torch.full((B, W - 1, D), float("nan"), dtype=state or F32, device="cuda")
    y, fin = kda.conv_fwd(x, w, b, act, initial_state=s, final_state=fin)
    torch.cuda.synchronize()
    args = (R.d(x).reshape(-1, D), R.d(w), R.d(b), act, R.d(s), [T] * B)
    yr, fr = R.conv(*args)
    R.check(y.reshape(-1, D), yr, BF, slack(args[0], args[1], args[2], args[4], [T] * B), "y")
    assert torch.equal(R.d(fin), fr.to(fin.dtype).double())


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("D,W,state", [(64, 4, F32), (77, 3, BF), (520, 2, None)])
def test_fwd_packed(lens, D, W, state):
    tail = 5   # rows behind the last sequence
    T, N = sum(lens) + tail, len(lens)
    x, w, b, s, _, _ = make(1, T, D, W, N, state, seed=2)
    say("case conv packed %s D=%d W=%d" % (lens, D, W))
    out = torch.full((1, T, D), 7.0, dtype=BF, device="cuda")
    fin = torch.full((N, W - 1, D), float("nan"), dtype=F32, device="cuda")
    kda.conv_fwd(x, w, b, "silu", initial_state=s, final_state=fin, cu_seqlens=cu_of(lens), out=out)
    torch.cuda.synchronize()
    xs = R.d(x)[0, :T - tail]
    yr, fr = R.conv(xs, R.d(w), R.d(b), "silu", R.d(s), lens)
    R.check(out[0, :T - tail], yr, BF, slack(xs, R.d(w), R.d(b), R.d(s), lens), "y")
    assert (out[0, T - tail:] == 7.0).all()
    assert torch.equal(R.d(fin), fr)


@pytest.mark.parametrize("D,wide,off", [(64, 8, 8), (64, 3, 1), (129, 64, 8)])
def test_slices(D, wide, off):
    x, w, b, s, dy, dfin = make(2, 40, D, 4, 2, F32, seed=3, wide=wide, off=off)
    y, _ = kda.conv_fwd(x, w, b, "silu", initial_state=s)
    assert torch.equal(y, kda.conv_fwd(x.contiguous(), w, b, "silu", initial_state=s)[0])
    g = kda.conv_bwd(x, w, b, "silu", dy, dfin, s)
    h = kda.conv_bwd(x.contiguous(), w, b, "silu", dy.contiguous(), dfin, s)
    for k in g:
        assert torch.equal(g[k], h[k]), k
    one = x[:, :1].expand(2, 40, D)   # the same input at every token
    assert torch.equal(kda.conv_fwd(one, w, b, None)[0], kda.conv_fwd(one.contiguous(), w, b, None)[0])


@pytest.mark.parametrize("D,W,state", [(64, 4, BF), (77, 3, F32), (1160, 2, F32)])
def test_state_in_place_and_steps(D, W, state):
    """A prompt cut in two, and token by token, gives what it gives in one piece, states updated in place."""
    T = 11
    x, w, b, s, _, _ = make(3, T, D, W, 3, state, seed=4)
    fin = torch.empty_like(s)
    y, fin = kda.conv_fwd(x, w, b, "silu", initial_state=s, final_state=fin)
    for cut in (1, 2, 7):
        st = s.clone()
        y1, _ = kda.conv_fwd(x[:, :cut], w, b, "silu", initial_state=st, final_state=st)
        y2, _ = kda.conv_fwd(x[:, cut:], w, b, "silu", initial_state=st, final_state=st)
        assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(st, fin)
    st, ys = s.clone(), []
    for t in range(T):
        out, _ = kda.conv_decode(x[:, t:t + 1], w, b, "silu", initial_state=st, final_state=st)
        ys.append(out)
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(st, fin)
    st = torch.full_like(s, float("nan"))   # no initial state: zeros
    out, _ = kda.conv_decode(x[:, :1], w, b, None, final_state=st)
    assert torch.equal(out, kda.conv_fwd(x[:, :1], w, b, None)[0])
    assert (st[:, :W - 2] == 0).all() and torch.equal(st[:, W - 2], x[:, 0].to(state))


def check_bwd(x, w, b, act, s, dy, dfin, lens, g):
    D, W = w.shape
    M = sum(lens)
    lx, lw, lb, ls = (None if t is None else R.d(t).requires_grad_() for t in (x.reshape(-1, D)[:M], w, b, s))
    gy, gf = R.d(dy).reshape(-1, D)[:M], R.d(dfin)
    y, f = R.conv(lx, lw, lb, act, ls, lens)
    dx, dw, db, ds = R.grads((y * gy).sum() + (f * gf).sum(), [lx, lw, lb, ls])
    # the size of the sums: |d_out| (1.1 |silu'| at most) times |w|, |x|; the activation's
    # derivative moves by at most half its argument's error
    ax, aw, gm = lx.detach().abs(), lw.detach().abs(), 1.1 * gy.abs()
    ab = None if b is None else lb.detach().abs()
    az = None if s is None else ls.detach().abs()
    pre, _ = R.conv(ax, aw, ab, None, az, lens)
    gm = gm * (1 + pre)
    leaves = [ax.requires_grad_(), aw.requires_grad_(), None if ab is None else ab.requires_grad_(),
              None if az is None else az.requires_grad_()]
    y, f = R.conv(leaves[0], leaves[1], leaves[2], None, leaves[3], lens)
    sx, sw, sb, ss = R.grads((y * gm).sum() + (f * gf.abs()).sum(), leaves)
    R.check(g["dx"].reshape(-1, D)[:M], dx, BF, 32 * R.U * sx, "dx")
    R.check(g["dweight"], dw, F32, 32 * R.U * sw, "dweight")
    if b is not None:
        R.check(g["dbias"], db, F32, 32 * R.U * sb, "dbias")
    if s is not None:
        R.check(g["d_initial_state"], ds, F32, 32 * R.U * ss, "d_initial_state")


@pytest.mark.parametrize("B,T,D,W,state", CASES)
@pytest.mark.parametrize("act", [None, "silu"])
def test_bwd_batches(B, T, D, W, state, act):
    x, w, b, s, dy, dfin = make(B, T, D, W, B, state, bias=act is None or T % 2 == 0, seed=5)
    say("case conv bwd %s W=%d state %s" % ((B, T, D), W, state))
    g = kda.conv_bwd(x, w, b, act, dy, dfin, s)
    torch.cuda.synchronize()
    assert (g["d_initial_state"] is None) == (s is None)
    check_bwd(x, w, b, act, s, dy, dfin, [T] * B, g)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("D,W,state", [(64, 4, F32), (77, 3, BF), (520, 2, None)])
def test_bwd_packed(lens, D, W, state):
    tail = 6
    T, N = sum(lens) + tail, len(lens)
    x, w, b, s, dy, dfin = make(1, T, D, W, N, state, seed=6)
    say("case conv bwd packed %s D=%d W=%d" % (lens, D, W))
    dx = torch.full((1, T, D), 7.0, dtype=BF, device="cuda")
    g = kda.conv_bwd(x, w, b, "silu", dy, dfin, s, cu_seqlens=cu_of(lens), outputs={"dx": dx})
    torch.cuda.synchronize()
    assert (dx[0, T - tail:] == 7.0).all()
    check_bwd(x, w, b, "silu", s, dy, dfin, lens, g)


def test_no_tokens():
    x, w, b, s, dy, dfin = make(2, 0, 64, 4, 2, F32)
    y, fin = kda.conv_fwd(x, w, b, "silu", initial_state=s, final_state=torch.empty_like(s))
    assert y.shape == (2, 0, 64) and torch.equal(fin, s)
    g = kda.conv_bwd(x, w, b, "silu", dy, dfin, s)
    assert torch.equal(g["d_initial_state"], dfin) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_long_partial_sums():
    """More token runs than partial sums: the gradient's workgroups walk over several."""
    T = 40000
    x, w, b, s, dy, _ = make(1, T, 8, 4, 1, None, seed=8)
    g = kda.conv_bwd(x, w, b, "silu", dy)
    torch.cuda.synchronize()
    check_bwd(x, w, b, "silu", None, dy, torch.zeros(1, 3, 8), [T], g)
    y, _ = kda.conv_fwd(x, w, b, "silu")
    a = (R.d(x)[0], R.d(w), R.d(b))
    R.check(y[0], R.conv(*a, "silu", None, [T])[0], BF, slack(*a, None, [T]), "y")


def test_special_values():
    x, w, b, s, _, _ = make(1, 40, 64, 4, 1, None, seed=9)
    x[0, 20, 3] = float("nan")
    x[0, 20, 4] = float("inf")
    y = kda.conv_fwd(x, w, b, None)[0].cpu().float()[0]
    assert y[20:24, 3].isnan().all() and not y[:20].isnan().any() and not y[24:].isnan().any()
    assert not y[:, 5:].isnan().any() and y[20:24, 4].isinf().all()


def test_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, s, c = n(9, 3), n(3, 4), n(3), n(2, 3, 3), n(9, 3)
    f = lambda t: (R.conv(t, w, b, "silu", s, [4, 5])[0] * c).sum()  # noqa: E731
    leaf, v = x.clone().requires_grad_(), n(9, 3)
    g = torch.autograd.grad(f(leaf), leaf)[0]
    want = float(R.difference(f, x, v))
    assert abs(float((g * v).sum()) - want) <= 1e-7 * (1 + abs(want))


def test_autograd_and_packed_tail():
    lens = [6, 0, 19]
    x, w, b, s, dy, dfin = make(1, 30, 64, 4, 3, BF, seed=10)
    for t in (x, w, b, s):
        t.requires_grad_()
    y, fin = kda.short_conv(x, w, b, "silu", initial_state=s, final_state_dtype=BF, cu_seqlens=cu_of(lens))
    assert (y[0, 25:] == 0).all()
    ((y * dy).sum() + (fin * dfin).sum()).backward()
    g = kda.conv_bwd(x.detach(), w.detach(), b.detach(), "silu", dy, dfin, s.detach(), cu_seqlens=cu_of(lens))
    assert torch.equal(x.grad[0, :25], g["dx"][0, :25]) and (x.grad[0, 25:] == 0).all()
    assert torch.equal(w.grad, g["dweight"]) and torch.equal(b.grad, g["dbias"])
    assert torch.equal(s.grad, g["d_initial_state"].to(BF))


def test_graph():
    lens = [20, 0, 45]
    x, w, b, s, dy, dfin = make(1, 70, 128, 4, 3, F32, seed=11)
    cu = cu_of(lens)
    y, fin = torch.zeros(1, 70, 128, dtype=BF, device="cuda"), torch.empty_like(s)
    outs = {"dx": torch.zeros_like(y), "dweight": torch.empty_like(w), "dbias": torch.empty_like(b),
            "d_initial_state": torch.empty_like(s)}
    ws = torch.empty(kda.conv_bwd_workspace_size(1, 70, 128, 4), dtype=torch.uint8, device="cuda")

    def call():
        kda.conv_fwd(x, w, b, "silu", initial_state=s, final_state=fin, cu_seqlens=cu, out=y)
        kda.conv_bwd(x, w, b, "silu", dy, dfin, s, cu_seqlens=cu, workspace=ws, outputs=outs)
    call()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in {**outs, "y": y, "fin": fin}.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        for t in (*outs.values(), y, fin):
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in {**outs, "y": y, "fin": fin}.items():
            assert torch.equal(v, want[k]), (rep, k)


def test_refusals():
    x, w, b, s, dy, dfin = make(2, 10, 64, 4, 2, F32)
    cu = cu_of([10])
    for bad in (lambda: kda.conv_fwd(x.float(), w, b), lambda: kda.conv_fwd(x, w[:, :1], b), lambda: kda.conv_fwd(x, w[:60], b),
                lambda: kda.conv_fwd(x, w, b.to(BF)), lambda: kda.conv_fwd(x, w, b, "relu"),
                lambda: kda.conv_fwd(x, w, b, cu_seqlens=cu), lambda: kda.conv_fwd(x[:1], w, b, cu_seqlens=cu.int()),
                lambda: kda.conv_fwd(x, w, b, initial_state=s[:1]), lambda: kda.conv_fwd(x, w, b, out=x),
                lambda: kda.conv_fwd(x.transpose(1, 2), w[:10], b[:10]), lambda: kda.conv_decode(x, w, b, final_state=s),
                lambda: kda.conv_decode(x[:, :1], w, b), lambda: kda.conv_decode(x[:, :1], w, b, initial_state=s[:, :, :], final_state=s[:1]),
                lambda: kda.conv_bwd(x, w, b, "silu", dy[:1]), lambda: kda.conv_bwd(x, w, b, "silu", dy, outputs={"dx": x}),
                lambda: kda.conv_fwd(x, w.cpu(), b)):
        with pytest.raises(ValueError):
            bad()
