"""How the layer operators may be called: on two streams at once, from two graphs that share a
workspace, with broadcast inputs, and through autograd with some outputs unused."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say
from tests.test_gpu_ssm import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def layer(T, seed):
    """Every operator once, forwards and backwards: a function that returns all their outputs."""
    D, H, P, S = 256, 4, 64, 64
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u, h, w = n(T, D).to(BF).cuda(), n(T, D).cuda(), n(D).cuda()
    x, cw, cb = n(2, T, D).to(BF).cuda(), n(D, 4).cuda(), n(D).cuda()
    a, s = make(2, T, H, P, 1, S, 2, F32, seed=seed)
    dy, dx = n(2, T, H, P).to(BF).cuda(), n(2, T, D).to(BF).cuda()

    def run():
        fin = torch.empty(2, H, P, S, dtype=F32, device="cuda")
        out = list(kda.rmsnorm_fwd(u, w, 1e-5, residual=h))
        out += kda.rmsnorm_quant(u, w, 1e-5, residual=h)
        out += kda.rmsnorm_bwd(h, w, 1e-5, u).values()
        out += kda.conv_fwd(x, cw, cb, "silu")
        out += kda.conv_bwd(x, cw, cb, "silu", dx).values()
        out += kda.ssm_fwd(*a.values(), initial_state=s, final_state=fin)
        out += kda.ssm_bwd(*a.values(), dy, initial_state=s).values()
        return [t.clone() for t in out if t is not None]
    return run


def same(a, b):
    assert len(a) == len(b)
    for i, (p, q) in enumerate(zip(a, b)):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), i


def test_two_streams_at_once():
    runs = [layer(333, 1), layer(1500, 2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for r, st in zip(runs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(r())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        say("case two streams, call %d" % i)
        same(g, want[i % 2])


def test_two_graphs_share_a_workspace():
    sets = [make(1, T, 4, 64, 2, 128, 1, F32, seed=T) for T in (130, 700)]
    size = max(max(kda.ssm_workspace_size(1, T, 4, 64, 2, 128), kda.ssm_bwd_workspace_size(1, T, 4, 64, 2, 128))
               for T in (130, 700))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dys = [torch.randn(a["x"].shape, device="cuda").to(BF) for a, _ in sets]
    outs = [{"dx": torch.empty(a["x"].shape, dtype=BF, device="cuda"),
             "dA_log": torch.empty(4, device="cuda")} for a, _ in sets]
    ys = [torch.empty(a["x"].shape, dtype=BF, device="cuda") for a, _ in sets]

    def call(i):
        a, s = sets[i]
        kda.ssm_fwd(*a.values(), initial_state=s, out=ys[i], workspace=ws)
        kda.ssm_bwd(*a.values(), dys[i], initial_state=s, workspace=ws, outputs=outs[i])
    want = []
    for i in range(2):
        call(i)
        want.append([t.clone() for t in (ys[i], *outs[i].values())])
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        for t in (ys[0], ys[1], *outs[0].values(), *outs[1].values()):
            t.zero_()
        for i in (rep % 2, 1 - rep % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            same([ys[i], *outs[i].values()], want[i])


def test_broadcast_inputs():
    """Inputs expanded over the batch or over the tokens (stride 0) give what their copies give; autograd
    sums their gradients."""
    a, _ = make(3, 70, 2, 64, 1, 64, 3, None, seed=4)
    for dim in (0, 1):
        e = {k: v.narrow(dim, 0, 1).expand(v.shape) if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
        c = {k: v.contiguous() for k, v in e.items()}
        dy = torch.randn(a["x"].shape, device="cuda").to(BF)
        same([kda.ssm_fwd(*e.values())[0]], [kda.ssm_fwd(*c.values())[0]])
        same([v for v in kda.ssm_bwd(*e.values(), dy).values() if v is not None],
             [v for v in kda.ssm_bwd(*c.values(), dy).values() if v is not None])
        same([kda.ssm_bwd(*a.values(), dy[:1, :1].expand(dy.shape))["dx"]],
             [kda.ssm_bwd(*a.values(), dy[:1, :1].expand(dy.shape).contiguous())["dx"]])
        x = a["x"].flatten(2)
        xe = x.narrow(dim, 0, 1).expand(x.shape)
        w = torch.randn(x.shape[2], 4, device="cuda")
        same([kda.conv_fwd(xe, w)[0]], [kda.conv_fwd(xe.contiguous(), w)[0]])
        same([v for v in kda.conv_bwd(xe, w, None, "silu", xe).values() if v is not None],
             [v for v in kda.conv_bwd(xe.contiguous(), w, None, "silu", xe.contiguous()).values() if v is not None])
        row = x[0].narrow(0, 0, 1).expand(x.shape[1:])
        wn = torch.randn(x.shape[2], device="cuda")
        same([kda.rmsnorm_fwd(row, wn, 1e-5)[0]], [kda.rmsnorm_fwd(row.contiguous(), wn, 1e-5)[0]])
    small = a["B"][:1].contiguous().requires_grad_()
    y, _ = kda.ssm_scan(a["x"], a["dt"], small.expand(a["B"].shape), *list(a.values())[3:])
    (y.float() * dy).sum().backward()
    each = kda.ssm_bwd(a["x"], a["dt"], small.detach().expand(a["B"].shape).contiguous(), *list(a.values())[3:], dy)["dB"]
    # three bf16 gradients summed in bf16: two roundings of partial sums
    bound = 2 * 2.0 ** -8 * each.double().abs().sum(0, keepdim=True)
    assert ((small.grad.double() - each.double().sum(0, keepdim=True)).abs() <= bound).all()


def test_autograd_with_unused_outputs_and_twice():
    a, s = make(1, 90, 2, 64, 1, 64, 1, F32, seed=5)
    leaf = {k: v.detach().clone().requires_grad_() for k, v in a.items()}
    _, fin = kda.ssm_scan(*leaf.values(), initial_state=s, final_state_dtype=F32)
    fin.sum().backward()
    want = kda.ssm_bwd(*a.values(), torch.zeros(a["x"].shape, dtype=BF, device="cuda"),
                       d_final_state=torch.ones_like(fin), initial_state=s)
    same([leaf["x"].grad, leaf["A_log"].grad, leaf["C"].grad], [want["dx"], want["dA_log"], want["dC"]])
    assert float(want["dC"].abs().max()) == 0
    x, w = torch.randn(9, 64, device="cuda").to(BF).requires_grad_(), torch.randn(64, device="cuda").requires_grad_()
    r = torch.randn(9, 64, device="cuda", requires_grad=True)
    _, h = kda.rms_norm(x, w, 1e-5, residual=r)
    h.sum().backward()  # only the sum: its gradient passes through, the weight's is zero
    assert (x.grad == 1).all() and (r.grad == 1).all() and (w.grad == 0).all()
    c = torch.randn(1, 9, 64, device="cuda").to(BF).requires_grad_()
    wc = torch.randn(64, 4, device="cuda")
    _, last = kda.short_conv(c, wc, final_state_dtype=F32)
    last.sum().backward()
    assert (c.grad[:, :6] == 0).all() and (c.grad[:, 6:] == 1).all()
    for y, leaf1 in ((kda.rms_norm(x, w)[0], x), (kda.short_conv(c, wc)[0], c),
                     (kda.ssm_scan(*leaf.values())[0], leaf["x"])):
        g = torch.autograd.grad(y.float().square().sum(), leaf1, create_graph=True)[0]
        with pytest.raises(RuntimeError):
            g.float().sum().backward()


def packed_calls(cu, T=100):
    """Each call that takes cu_seqlens, with its outputs the middle one of three in a buffer of zeros."""
    a, _ = make(1, T, 2, 64, 1, 64, 1, None, seed=6)
    x = a["x"].flatten(2).contiguous()
    w = torch.ones(x.shape[2], 4, device="cuda")
    dy = torch.randn(a["x"].shape, device="cuda").to(BF)

    def guarded(*names):
        outs = {n: torch.zeros(3, *s[1:], dtype=BF, device="cuda") for n, s in names}
        return outs, {n: t[1:2] for n, t in outs.items()}
    conv, ssm = [("dx", x.shape)], [("dx", a["x"].shape), ("ddt", a["dt"].shape), ("dB", a["B"].shape), ("dC", a["C"].shape)]
    for fn, names in ((lambda o: kda.conv_fwd(x, w, cu_seqlens=cu, out=o["dx"]), conv),
                      (lambda o: kda.conv_bwd(x, w, None, "silu", x, cu_seqlens=cu, outputs=o), conv),
                      (lambda o: kda.ssm_fwd(*a.values(), cu_seqlens=cu, out=o["dx"], piece_chunks=1), ssm),
                      (lambda o: kda.ssm_bwd(*a.values(), dy, cu_seqlens=cu, outputs=o, piece_chunks=1), ssm)):
        whole, outs = guarded(*names)
        yield lambda: fn(outs), whole


def test_wrong_lengths_stay_inside():
    """Contents of cu_seqlens that no batch has are clamped on the device: nothing outside the outputs is written."""
    for cu in ([0, -5, 1000, 50], [70, 20, 90, 30], [0, 1 << 40, 5, 1 << 50], [0, 100] * 20, [100, 0] * 20):
        for i, (call, whole) in enumerate(packed_calls(torch.tensor(cu, device="cuda"))):
            say("case lengths %s, call %d" % (cu[:4], i))
            call()
            torch.cuda.synchronize()
            for t in whole.values():
                assert (t[0] == 0).all() and (t[2] == 0).all()


def test_validated_lengths(monkeypatch):
    """KDA_VALIDATE=1 refuses such contents before anything is launched; a batch's rows may go on behind its
    last sequence."""
    monkeypatch.setenv("KDA_VALIDATE", "1")
    for cu in ([3, 20, 100], [0, 60, 20], [0, 50, 101]):
        for call, whole in packed_calls(torch.tensor(cu, device="cuda")):
            with pytest.raises(RuntimeError):
                call()
            torch.cuda.synchronize()
            assert all((t == 0).all() for t in whole.values())
    for call, whole in packed_calls(torch.tensor([0, 0, 77], device="cuda")):
        call()
        assert all(float(t[1, :77].abs().max()) > 0 and (t[1, 77:] == 0).all() for t in whole.values() if t.any())


def test_more_than_32_bits_of_entries():
    """Tensors of more than 2^31 entries: their last rows come out as those of a small batch."""
    rows, D, tail = 530000, 4096, 200
    assert rows * D > 1 << 31
    x = torch.zeros(1, rows, D, dtype=BF, device="cuda")
    x[:, -tail:].normal_()
    last = x[:, -tail:].contiguous()
    w, wc = torch.rand(D, device="cuda"), torch.randn(D, 4, device="cuda")
    say("case 2^31 entries: norm")
    same([kda.rmsnorm_fwd(x, w, 1e-5)[0][0, -tail:]], [kda.rmsnorm_fwd(last, w, 1e-5)[0][0]])
    q, s, _ = kda.rmsnorm_quant(x, w, 1e-5)
    ql, sl, _ = kda.rmsnorm_quant(last, w, 1e-5)
    same([q[0, -tail:], s[0, -tail:]], [ql[0], sl[0]])
    same([kda.rmsnorm_bwd(x, w, 1e-5, x)["dx"][0, -tail:]], [kda.rmsnorm_bwd(last, w, 1e-5, last)["dx"][0]])
    say("case 2^31 entries: convolution")
    same([kda.conv_fwd(x, wc)[0][0, -tail:]], [kda.conv_fwd(last, wc)[0][0]])
    same([kda.conv_bwd(x, wc, None, "silu", x)["dx"][0, -tail:]], [kda.conv_bwd(last, wc, None, "silu", last)["dx"][0]])
    # the scan: zeros leave no state behind, so the tail starts from none in both
    H, P, S = D // 64, 64, 64
    g = {"dt": torch.zeros(1, rows, H, dtype=BF, device="cuda"), "B": torch.zeros(1, rows, 1, S, dtype=BF, device="cuda"),
         "C": torch.zeros(1, rows, 1, S, dtype=BF, device="cuda")}
    for t in g.values():
        t[:, -tail:].normal_()
    A, bias = torch.zeros(H, device="cuda"), torch.full((H,), -3.0, device="cuda")
    big = [x.unflatten(2, (H, P)), *g.values(), A, bias]
    small = [t[:, -tail:].contiguous() for t in big[:4]] + [A, bias]
    say("case 2^31 entries: scan")
    y, yl = kda.ssm_fwd(*big)[0][0, -tail:].float(), kda.ssm_fwd(*small)[0][0].float()
    # the chunks begin at other tokens: two roundings to bf16 of sums that agree to 2^-16 of their size
    assert float((y - yl).abs().max()) <= (2.0 ** -7 + 2.0 ** -15) * float(yl.abs().max())
    say("case 2^31 entries: scan's gradient")
    d, dl = kda.ssm_bwd(*big, None, big[0])["dx"][0, -tail:].float(), kda.ssm_bwd(*small, None, small[0])["dx"][0].float()
    assert float((d - dl).abs().max()) <= (2.0 ** -7 + 2.0 ** -15) * float(dl.abs().max())


def test_the_library_takes_its_own_workspace(monkeypatch):
    """Through the C ABI without a workspace: taken and given back on the stream, with the same results."""
    from gated_delta_rule_110_amd import layer as L

    lens = [300, 0, 5, 129]
    a, s = make(1, sum(lens), 4, 64, 1, 128, len(lens), F32, seed=7)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    dy = torch.randn(a["x"].shape, device="cuda").to(BF)
    x, w, wc = torch.randn(1, 434, 256, device="cuda").to(BF), torch.randn(256, device="cuda"), torch.randn(256, 4, device="cuda")
    u, odd = torch.randn(70, 256, device="cuda").to(BF), torch.randn(70, 77, device="cuda").to(BF)

    def run():
        return [t.clone() for t in (*kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), cu_seqlens=cu, piece_chunks=1),
                                    *kda.ssm_bwd(*a.values(), dy, initial_state=s, cu_seqlens=cu, piece_chunks=1).values(),
                                    *kda.conv_bwd(x, wc, None, "silu", x, cu_seqlens=cu).values(),
                                    *kda.rmsnorm_bwd(u, w, 1e-5, u).values(), *kda.rmsnorm_bwd(odd, w[:77].clone(), 1e-5, odd).values())
                if t is not None]
    want = run()
    none = []
    monkeypatch.setattr(L, "_workspace", lambda t, need, dev, d: none.append(need))
    for rep in range(3):
        same(run(), want)
    torch.cuda.synchronize()
    assert len(none) == 15 and all(n > 0 for n in none)
