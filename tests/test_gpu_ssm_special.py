"""The scan where calls are out of the ordinary.  NaN and infinities in its inputs: a prompt's
outputs are those of its tokens taken one by one, so one in a token reaches that token and those
behind it, never those before.  Packed batches of very short sequences and their workspaces."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R
from tests.parity import say
from tests.test_gpu_ssm import check as check_scan, check_bwd, make

pytestmark = pytest.mark.gpu
F32 = torch.float32
NAN, INF = float("nan"), float("inf")


def step_by_step(a, s):
    st, ys = s.clone(), []
    for t in range(a["x"].shape[1]):
        one = [v[:, t:t + 1] if k in ("x", "dt", "B", "C") else v for k, v in a.items()]
        ys.append(kda.ssm_decode(*one, initial_state=st, final_state=st)[0])
    return torch.cat(ys, 1), st


def check(a, clean, s, label, pc=0):
    y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), piece_chunks=pc)
    want, last = step_by_step(a, s)
    was, _ = kda.ssm_fwd(*clean.values(), initial_state=s, piece_chunks=pc)
    ok = want.isfinite()
    assert torch.equal(y.isfinite(), ok), (label, (y.isfinite() != ok).nonzero()[:5].tolist())
    assert torch.equal(fin.isfinite(), last.isfinite()), label
    assert torch.equal(y[ok], was[ok]), label


@pytest.mark.parametrize("H,P,G,S", [(2, 64, 1, 64), (4, 128, 2, 128)])
@pytest.mark.parametrize("t", [0, 5, 15, 16, 40, 63, 64, 100, 129])
def test_nothing_reaches_the_tokens_before(H, P, G, S, t):
    clean, s = make(1, 130, H, P, G, S, 1, F32, seed=t)
    for name, at, value in (("x", (0, t, 1, 7), NAN), ("x", (0, t, 0, P - 1), INF), ("x", (0, t, 1, 16), -INF), ("B", (0, t, 0, 3), NAN),
                            ("B", (0, t, 0, S - 1), INF), ("C", (0, t, G - 1, 9), NAN), ("C", (0, t, 0, 0), -INF), ("dt", (0, t, 1), NAN),
                            ("dt", (0, t, 0), INF)):
        say("case %s = %s at token %d" % (name, value, t))
        a = {k: v.clone() if k == name else v for k, v in clean.items()}
        a[name][at] = value
        check(a, clean, s, (name, value, t), pc=t % 2)


def test_several_at_once():
    clean, s = make(1, 200, 3, 64, 1, 128, 1, F32, seed=3)
    a = {k: v.clone() if k == "x" else v for k, v in clean.items()}
    for t, p, v in ((3, 0, INF), (9, 0, -INF), (20, 1, NAN), (20, 2, INF), (63, 3, NAN), (64, 3, NAN), (150, 40, INF), (199, 63, NAN)):
        a["x"][0, t, t % 3, p] = v
    check(a, clean, s, "several")


def test_padding_that_holds_nan():
    """A padded batch: what stands behind a row's tokens, in every tensor, leaves their outputs as they are."""
    lens = [1, 40, 65, 100]
    a, _ = make(4, 100, 2, 64, 1, 64, 4, None, seed=4)
    was, _ = kda.ssm_fwd(*a.values())
    for k in ("x", "dt", "B", "C"):
        a[k] = a[k].clone()
        for n, m in enumerate(lens):
            a[k][n, m:] = NAN
    y, _ = kda.ssm_fwd(*a.values())
    for n, m in enumerate(lens):
        assert torch.equal(y[n, :m], was[n, :m]) and y[n, m:].isnan().all(), n


def test_no_step_leaves_everything():
    """A raw step size of -inf or of the type's lowest value takes no step: the token leaves the state as it was."""
    a, s = make(1, 70, 2, 64, 1, 64, 1, F32, seed=5)
    a["dt"][0, 10:20] = -INF
    a["dt"][0, 30:] = torch.finfo(torch.bfloat16).min
    check(a, a, s, "no step")
    keep = {k: v[:, :30] if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
    _, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s))
    _, last = kda.ssm_fwd(*keep.values(), initial_state=s, final_state=torch.empty_like(s))
    assert torch.equal(fin, last)


@pytest.mark.parametrize("lens,pc", [([65] * 10, 1), ([129, 3, 0, 129, 64, 1, 129], 2), ([1] * 70 + [700] + [2] * 70, 4),
                                     ([7, 64, 5], 1), ([0, 0], 1)])
def test_a_workspace_of_exactly_the_size(lens, pc):
    """Sequences of one and of several pieces among each other, in a workspace that ends where its size says."""
    a, s = make(1, sum(lens), 2, 64, 1, 128, len(lens), F32, seed=7)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    dy = torch.randn(a["x"].shape, device="cuda").to(torch.bfloat16)
    for bwd in (False, True):
        size = kda.ssm_bwd_workspace_size if bwd else kda.ssm_workspace_size
        need = size(1, sum(lens), 2, 64, 1, 128, num_seqs=len(lens), piece_chunks=pc)
        ws = torch.full((need + 65536,), 0xa5, dtype=torch.uint8, device="cuda")
        say("case workspace %s pieces of %d backwards %s" % (lens[:4], pc, bwd))
        if bwd:
            g = kda.ssm_bwd(*a.values(), dy, initial_state=s, cu_seqlens=cu, workspace=ws, piece_chunks=pc)
            check_bwd(a, s, lens, dy, None, g)
        else:
            y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), cu_seqlens=cu, workspace=ws,
                                 piece_chunks=pc)
            check_scan(a, s, lens, y, fin, "exact workspace")
        assert (ws[need:] == 0xa5).all()


@pytest.mark.parametrize("H,P,G", [(3, 64, 1), (8, 128, 2)])
def test_launches_in_pieces(H, P, G):
    """launch_piece splits every kernel's grid as a very large batch does: the same results, bit for bit."""
    lens = [70, 3, 300, 0, 129]
    a, s = make(1, sum(lens), H, P, G, 64, len(lens), F32, seed=8)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    dy = torch.randn(a["x"].shape, device="cuda").to(torch.bfloat16)
    one, st = make(20, 1, H, P, G, 64, 20, F32, seed=9)

    def run(cap):
        y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), cu_seqlens=cu, piece_chunks=1,
                             launch_piece=cap)
        g = kda.ssm_bwd(*a.values(), dy, initial_state=s, cu_seqlens=cu, piece_chunks=1, launch_piece=cap)
        return [y, fin, *g.values(), *kda.ssm_decode(*one.values(), initial_state=st, final_state=torch.empty_like(st), launch_piece=cap)]
    want = run(0)
    for cap in (1, 16, 40):
        say("case launches of at most %d" % cap)
        for i, (t, u) in enumerate(zip(run(cap), want)):
            assert torch.equal(t, u), (cap, i)


def test_more_sequences_than_a_launch_holds():
    """131073 sequences of one token, 64 heads: more than 2^23 workgroups, packed and as a batch."""
    n, H, P, S = 131073, 64, 64, 64
    small, _ = make(1, 64, H, P, 1, S, 64, None, seed=10)
    args = {k: v.repeat(1, n // 64 + 1, *[1] * (v.dim() - 2))[:, :n] if k in ("x", "dt", "B", "C") else v for k, v in small.items()}
    cu = torch.arange(n + 1, device="cuda")
    want, _ = kda.ssm_fwd(*small.values(), cu_seqlens=cu[:65].contiguous())
    say("case 131073 packed sequences")
    y, _ = kda.ssm_fwd(*args.values(), cu_seqlens=cu)
    assert torch.equal(y[0, :64], want[0]) and torch.equal(y[0, n - 1], want[0, (n - 1) % 64])
    assert torch.equal(y[0, n - 65:n - 1], want[0].roll(-((n - 65) % 64), 0))
    say("case 131073 batch rows")
    rows = {k: v.transpose(0, 1) if k in ("x", "dt", "B", "C") else v for k, v in args.items()}
    assert torch.equal(kda.ssm_fwd(*rows.values())[0][:, 0], y[0])


@pytest.mark.parametrize("dtype,N", [(F32, 200), (torch.bfloat16, 400)])
@pytest.mark.parametrize("in_place", [False, True])
def test_states_larger_than_the_cache(dtype, N, in_place):
    """A step over states of more than 384 MiB, which are read past the caches: the first and last sequences as
    those of a small batch."""
    H, P, S = 64, 64, 128
    a, _ = make(N, 1, H, P, 1, S, N, None, seed=11)
    s = torch.randn(N, H, P, S, device="cuda").to(dtype)
    assert s.numel() * s.element_size() > 384 << 20
    picks = [0, 1, N // 2, N - 1]
    few = {k: v[picks].contiguous() if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
    y, fin = kda.ssm_decode(*few.values(), initial_state=s[picks], final_state=torch.empty_like(s[picks]))
    say("case %d sequences, %s, in place %s" % (N, dtype, in_place))
    z, last = kda.ssm_decode(*a.values(), initial_state=s, final_state=s if in_place else torch.empty_like(s))
    assert torch.equal(z[picks], y) and torch.equal(last[picks], fin)
    assert last.isfinite().all()


def test_a_step_over_more_than_32_bits_of_entries():
    """A state of more than 2^31 entries: the last sequences as those of a small batch."""
    H, P, S, N = 64, 128, 128, 2050
    assert N * H * P * S > 1 << 31
    a, _ = make(N, 1, H, P, 1, S, N, None, seed=12)
    s = torch.zeros(N, H, P, S, dtype=torch.bfloat16, device="cuda")
    s[-2:].normal_()
    few = {k: v[-2:].contiguous() if k in ("x", "dt", "B", "C") else v for k, v in a.items()}
    y, fin = kda.ssm_decode(*few.values(), initial_state=s[-2:].clone(), final_state=torch.empty_like(s[-2:]))
    z, _ = kda.ssm_decode(*a.values(), initial_state=s, final_state=s)
    assert torch.equal(z[-2:], y) and torch.equal(s[-2:], fin)


@pytest.mark.parametrize("T,H", [(8192, 64), (5000, 4)])
def test_pieces_as_the_query_says(T, H):
    """Of a batch row and of a packed batch of one sequence: the pieces that ssm_piece_chunks tells, so that asking for
    them changes no bit."""
    a, s = make(1, T, H, 64, 1, 128, 1, F32, seed=13)
    pc = kda.ssm_piece_chunks(1, T, H, 64, 1, 128)
    assert kda.ssm_piece_chunks(1, T, H, 64, 1, 128, num_seqs=1) == pc < T // 64
    cu = torch.tensor([0, T], device="cuda")
    want = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), piece_chunks=pc)
    for lens in (None, cu):
        for n in (0, pc):
            got = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s), cu_seqlens=lens, piece_chunks=n)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (n, lens)


@pytest.mark.parametrize("A_log", [20.0, 80.0, 88.0, 100.0, 3e38, INF])
def test_decay_rates_that_leave_nothing(A_log):
    """e^A_log far above one, or above fp32: a step leaves nothing of the state before it, prompts as well as
    single tokens; where there is no step (dt = 0) nothing decays.  The gradients are those of that."""
    a, s = make(1, 100, 3, 64, 1, 64, 1, F32, seed=14)
    a["A_log"][1] = A_log
    a["dt"][0, 50:60] = -INF
    check(a, a, s, "A_log = %g" % A_log)
    y, fin = kda.ssm_fwd(*a.values(), initial_state=s, final_state=torch.empty_like(s))
    want, last = step_by_step(a, s)
    assert y.isfinite().all() and fin.isfinite().all()
    # no state of that head outlives a token: y = (dt C.B + D) x, as the one-token step has it, once more rounded
    R.check(y[0, :, 1], R.d(want[0, :, 1]), torch.bfloat16, 2.0 ** -8 * R.d(want[0, :, 1]).abs() + 1e-30, "y")
    R.check(fin[0, 1], R.d(last[0, 1]), F32, 64 * R.U * R.d(last[0, 1]).abs() + 1e-30, "state")
    dy = torch.randn(a["x"].shape, device="cuda").to(torch.bfloat16)
    g = kda.ssm_bwd(*a.values(), dy, d_final_state=torch.randn_like(s), initial_state=s)
    for k, v in g.items():
        assert v.isfinite().all(), k
    assert (g["dA_log"][1] == 0) and (g["d_initial_state"][0, 1] == 0).all()


def test_special_values_in_place_and_captured():
    """Pieces that are walked through twice: with the state updated in place, and in a graph whose inputs change
    between replays."""
    lens = [200, 0, 65, 300]
    a, s = make(1, sum(lens), 4, 128, 2, 64, len(lens), F32, seed=15)
    cu = torch.tensor(R.bounds(lens), dtype=torch.int64, device="cuda")
    b = {k: v.clone() for k, v in a.items()}
    b["x"][0, 100, 1, 5], b["x"][0, 400, 3, 70] = NAN, INF
    bits = lambda y, f: (y.view(torch.int16).clone(), f.view(torch.int32).clone())  # noqa: E731
    want = {i: bits(*kda.ssm_fwd(*v.values(), initial_state=s, final_state=torch.empty_like(s), cu_seqlens=cu))
            for i, v in enumerate((a, b))}
    st = s.clone()
    got = bits(*kda.ssm_fwd(*b.values(), initial_state=st, final_state=st, cu_seqlens=cu))
    assert all(torch.equal(g, w) for g, w in zip(got, want[1]))
    c = {k: v.clone() for k, v in a.items()}
    out, fin = torch.empty(a["x"].shape, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s)
    ws = torch.empty(kda.ssm_workspace_size(1, sum(lens), 4, 128, 2, 64, num_seqs=len(lens)), dtype=torch.uint8, device="cuda")

    def call():
        kda.ssm_fwd(*c.values(), initial_state=s, final_state=fin, cu_seqlens=cu, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in (1, 0, 1, 0):
        c["x"].copy_((a, b)[i]["x"])
        out.zero_(), fin.zero_(), ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(bits(out, fin), want[i])), i
