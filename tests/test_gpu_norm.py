"""RMS normalisation with the residual's addition against its formula in 64 bits:
bf16 and e4m3 outputs, gradients, odd widths, strides, special values, graphs."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(1, 1), (3, 7), (65, 64), (2, 128), (7, 136), (9, 256), (5, 504), (4, 1000), (3, 2048), (2, 4104), (3, 8192),
          (2, 16384), (2, 16392), (2, 20001), (3000, 40), (5000, 128)]


def make(rows, D, res, wdt=F32, seed=0, wide=0, off=0):
    g = torch.Generator().manual_seed(seed + rows * 131 + D)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = n(rows, D + wide).to(BF).cuda()[:, off:off + D]
    w = (1 + 0.2 * n(D)).to(wdt).cuda()
    r = None if res is None else (2 * n(rows, D + wide)).to(res).cuda()[:, off:off + D]
    return x, w, r


# y is rounded once; before that a sum of D squares (relative error at most about
# log2(D) + 8 half steps of fp32 in a tree, 32 allows for it), the root and two products.
F32_REL = 48 * R.U


def check_fwd(x, w, r, y, res):
    yr, h = R.rmsnorm(R.d(x), R.d(w), EPS, None if r is None else R.d(r))
    R.check(y, yr, BF, F32_REL * yr.abs() * 2, "y")
    if r is not None:
        R.check(res, h, r.dtype, R.U * h.abs() * 2, "residual")


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("res", [None, BF, F32])
def test_fwd(rows, D, res):
    x, w, r = make(rows, D, res, BF if D % 3 == 0 else F32)
    say("case rmsnorm %d x %d residual %s" % (rows, D, res))
    y, out = kda.rmsnorm_fwd(x, w, EPS, residual=r)
    torch.cuda.synchronize()
    assert (out is None) == (r is None)
    check_fwd(x, w, r, y, out)


def check_quant(x, w, r, q, s, group):
    yr, _ = R.rmsnorm(R.d(x), R.d(w), EPS, None if r is None else R.d(r))
    rows, D = yr.shape
    g = group or D
    pad = torch.nn.functional.pad(yr, (0, -D % g)).view(rows, -1, g)
    ref = (pad.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    assert s.shape == ref.shape
    R.check(s, ref, F32, 2 * F32_REL * ref, "scales")
    sc = ref.repeat_interleave(g, 1)[:, :D]
    # half a step of e4m3: 2^-4 of the value, or half of the smallest subnormal 2^-9
    tol = yr.abs() * 2.0 ** -4 + sc * 2.0 ** -10 + 4 * F32_REL * yr.abs()
    err = (R.d(q.float()) * R.d(s).repeat_interleave(g, 1)[:, :D] - yr).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("res", [None, BF, F32])
def test_quant(rows, D, group, res):
    x, w, r = make(rows, D, res, seed=3)
    say("case rmsnorm e4m3 %d x %d group %d residual %s" % (rows, D, group, res))
    q, s, out = kda.rmsnorm_quant(x, w, EPS, residual=r, group=group)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn
    check_quant(x, w, r, q, s, group)
    if r is not None:
        R.check(out, R.d(x) + R.d(r), r.dtype, R.U * (R.d(x) + R.d(r)).abs() * 2, "residual")


@pytest.mark.parametrize("D,wide,off", [(64, 8, 8), (64, 8, 3), (1000, 24, 16), (77, 5, 2), (4096, 4096, 4096)])
def test_strides_and_alignment(D, wide, off):
    for res in (None, BF, F32):
        x, w, r = make(6, D, res, wide=wide, off=off, seed=5)
        say("case rmsnorm slice %d of %d from %d" % (D, D + wide, off))
        y, out = kda.rmsnorm_fwd(x, w, EPS, residual=r)
        q, s, _ = kda.rmsnorm_quant(x, w, EPS, residual=r, group=128)
        check_fwd(x, w, r, y, out)
        check_quant(x, w, r, q, s, 128)


def test_shapes_broadcast_and_in_place():
    x, w, r = make(12, 256, BF, seed=7)
    want, wres = kda.rmsnorm_fwd(x, w, EPS, residual=r)
    y, res = kda.rmsnorm_fwd(x.view(3, 4, 256), w, EPS, residual=r.view(3, 4, 256))
    assert y.shape == (3, 4, 256) and torch.equal(y.view(12, 256), want) and torch.equal(res.view(12, 256), wres)
    one = x[:1].expand(12, 256)          # one row for all
    y, _ = kda.rmsnorm_fwd(one, w, EPS)
    assert torch.equal(y, kda.rmsnorm_fwd(one.contiguous(), w, EPS)[0])
    x2, r2 = x.clone(), r.clone()        # out over x, residual_out over the residual
    y, res = kda.rmsnorm_fwd(x2, w, EPS, residual=r2, out=x2, residual_out=r2)
    assert torch.equal(x2, want) and torch.equal(r2, wres)
    x3, w3, r3 = make(5, 77, F32, seed=8)  # the scalar path
    want, wres = kda.rmsnorm_fwd(x3, w3, EPS, residual=r3)
    kda.rmsnorm_fwd(x3, w3, EPS, residual=r3, out=x3, residual_out=r3)
    assert torch.equal(x3, want) and torch.equal(r3, wres)


def test_no_rows():
    x, w, r = make(4, 64, BF)
    y, res = kda.rmsnorm_fwd(x[:0], w, EPS, residual=r[:0])
    assert y.shape == (0, 64) and res.shape == (0, 64)
    q, s, _ = kda.rmsnorm_quant(x[:0], w, EPS, group=128)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    g = kda.rmsnorm_bwd(x[:0], w, EPS, x[:0])
    assert g["dx"].shape == (0, 64) and torch.equal(g["dweight"], torch.zeros(64, device="cuda"))


@pytest.mark.parametrize("D", [64, 77, 4096])
@pytest.mark.parametrize("group", [0, 128])
def test_special_values(D, group):
    """Zero rows, huge and tiny rows, and rows with a NaN or an infinity leave their neighbours alone."""
    x, w, _ = make(8, D, None, seed=11)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 3e38 / D            # squares overflow fp32: the root of infinity, outputs zero
    x[5] = 1e-30
    say("case rmsnorm special values %d group %d" % (D, group))
    y, _ = kda.rmsnorm_fwd(x, w, EPS)
    q, s, _ = kda.rmsnorm_quant(x, w, EPS, group=group)
    y, q, s = y.cpu().float(), q.cpu().float(), s.cpu()
    assert (y[1] == 0).all() and (q[1] == 0).all() and (s[1] > 0).all()
    assert y[2].isnan().all() and q[2].isnan().all() and s[2].isnan().all()
    assert y[3, 5].isnan() and (y[3, :5] == 0).all()
    assert q[3, 5].isnan() and s[3, 0].isnan()
    assert (y[4] == 0).all() and (q[4] == 0).all()
    for i in (0, 6, 7):
        check_fwd(x[i:i + 1], w, None, y[i:i + 1], None)
        check_quant(x[i:i + 1], w, None, q[i:i + 1], s[i:i + 1], group)
    ref, _ = R.rmsnorm(R.d(x[5:6]), R.d(w), EPS)
    R.check(y[5:6], ref, BF, F32_REL * 2 * ref.abs(), "tiny")


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("hd,with_res", [(BF, False), (BF, True), (F32, True), (F32, False)])
def test_bwd(rows, D, hd, with_res):
    h, w, _ = make(rows, D, None, BF if D % 3 == 0 else F32, seed=13)
    h = (2 * h.float()).to(hd)
    dy = make(rows, D, None, seed=14)[0]
    dr = make(rows, D, hd, seed=15)[2] if with_res else None
    say("case rmsnorm bwd %d x %d %s" % (rows, D, hd))
    g = kda.rmsnorm_bwd(h, w, EPS, dy, d_residual_out=dr)
    torch.cuda.synchronize()
    hh, ww, gy = R.d(h).requires_grad_(), R.d(w).requires_grad_(), R.d(dy)
    y, _ = R.rmsnorm(hh, ww, EPS)
    loss = (y * gy).sum() + (0 if dr is None else (hh * R.d(dr)).sum())
    dh, dw = R.grads(loss, [hh, ww])
    hh, ww = hh.detach(), ww.detach()
    rstd = 1 / torch.sqrt((hh * hh).mean(-1, keepdim=True) + EPS)
    n = hh * rstd
    size = rstd * ((ww * gy).abs() + n.abs() * (ww * gy * n).abs().mean(-1, keepdim=True)) + (0 if dr is None else R.d(dr).abs())
    R.check(g["dx"], dh, BF, F32_REL * size, "dx")
    if hd == F32:
        R.check(g["dresidual"], dh, F32, F32_REL * size, "dresidual")
    elif with_res:
        assert torch.equal(g["dresidual"], g["dx"])
    else:
        assert g["dresidual"] is None
    R.check(g["dweight"], dw, F32, F32_REL * (gy * n).abs().sum(0), "dweight")


def test_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, c, v = n(3, 10), n(10), n(3, 10), n(3, 10)
    f = lambda t: float((R.rmsnorm(t, w, EPS)[0] * c).sum())  # noqa: E731
    leaf = x.clone().requires_grad_()
    g = torch.autograd.grad((R.rmsnorm(leaf, w, EPS)[0] * c).sum(), leaf)[0]
    want = R.difference(f, x, v)
    assert abs(float((g * v).sum()) - want) <= 1e-7 * (1 + abs(want))


def test_bwd_strides():
    h, w, _ = make(6, 128, None, wide=64, off=64, seed=17)
    dy = make(6, 128, None, wide=8, off=8, seed=18)[0]
    a = kda.rmsnorm_bwd(h, w, EPS, dy)
    b = kda.rmsnorm_bwd(h.contiguous(), w, EPS, dy.contiguous())
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    h, dy = h[:, 1:100], dy[:, 3:102]    # odd addresses
    a = kda.rmsnorm_bwd(h, w[:99].contiguous(), EPS, dy)
    b = kda.rmsnorm_bwd(h.contiguous(), w[:99].contiguous(), EPS, dy.contiguous())
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


def test_autograd():
    for res in (None, BF, F32):
        x, w, r = make(10, 192, res, seed=19)
        x.requires_grad_(), w.requires_grad_()
        if r is not None:
            r.requires_grad_()
        y, h = kda.rms_norm(x, w, EPS, residual=r)
        dy = make(10, 192, None, seed=20)[0]
        loss = (y * dy).sum() if r is None else (y * dy).sum() + (h * 0.5).sum()
        loss.backward()
        if r is None:
            g = kda.rmsnorm_bwd(x.detach(), w.detach(), EPS, dy)
        else:
            g = kda.rmsnorm_bwd(h.detach(), w.detach(), EPS, dy, d_residual_out=torch.full_like(h, 0.5))
            assert r.grad.dtype == r.dtype and torch.equal(r.grad, g["dresidual"])
        assert torch.equal(x.grad, g["dx"]) and torch.equal(w.grad, g["dweight"])
    x, w, r = make(4, 64, F32, seed=21)   # only the normalised output is used: no gradient of h
    r.requires_grad_()
    kda.rms_norm(x, w, EPS, residual=r)[0].sum().backward()
    assert torch.isfinite(r.grad).all() and float(r.grad.abs().max()) > 0


def test_graph_and_streams():
    x, w, r = make(33, 512, BF, seed=23)
    dy = make(33, 512, None, seed=24)[0]
    want = kda.rmsnorm_quant(x, w, EPS, residual=r, group=128)
    wantg = kda.rmsnorm_bwd(x, w, EPS, dy)
    out, sc, ro = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(r)
    outs = {k: torch.empty_like(v) for k, v in wantg.items() if v is not None}
    ws = torch.empty(kda.rmsnorm_bwd_workspace_size(33, 512), dtype=torch.uint8, device="cuda")

    def call():
        kda.rmsnorm_quant(x, w, EPS, residual=r, group=128, out=out, scales=sc, residual_out=ro)
        kda.rmsnorm_bwd(x, w, EPS, dy, workspace=ws, outputs=outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        sc.fill_(float("nan")), ro.fill_(float("nan")), ws.fill_(255), out.view(torch.uint8).fill_(1)
        for t in outs.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(sc, want[1])
        assert torch.equal(ro, want[2])
        for k, v in outs.items():
            assert torch.equal(v, wantg[k]), (rep, k)


def test_refusals():
    x, w, r = make(4, 64, BF)
    for bad in (lambda: kda.rmsnorm_fwd(x.float(), w, EPS), lambda: kda.rmsnorm_fwd(x, w[:63], EPS),
                lambda: kda.rmsnorm_fwd(x, w.half(), EPS), lambda: kda.rmsnorm_fwd(x, w, 0.0),
                lambda: kda.rmsnorm_fwd(x, w, float("nan")), lambda: kda.rmsnorm_fwd(x.t(), w[:4], EPS),
                lambda: kda.rmsnorm_fwd(x, w, EPS, residual=r[:3]), lambda: kda.rmsnorm_fwd(x, w, EPS, residual_out=r),
                lambda: kda.rmsnorm_fwd(x, w, EPS, residual=r, out=r), lambda: kda.rmsnorm_fwd(x, w.cpu(), EPS),
                lambda: kda.rmsnorm_quant(x, w, EPS, group=64), lambda: kda.rmsnorm_quant(x, w, EPS, out=x),
                lambda: kda.rmsnorm_bwd(x, w, EPS, x, d_residual_out=x.float()),
                lambda: kda.rmsnorm_bwd(x, w, EPS, x[:3]),
                lambda: kda.rmsnorm_bwd(x, w, EPS, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: kda.rmsnorm_bwd(x, w, EPS, r, outputs={"dx": x})):
        with pytest.raises(ValueError):
            bad()
