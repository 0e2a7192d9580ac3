"""Latent attention in its expanded form against the 64-bit oracle: lengths around
the tiles' sizes, masks that leave rows empty, packed batches, strides, special
values in hidden places, large offsets, and how the calls may be made."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import latent_ref as R
from tests.layer_ref import d
from tests.parity import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SCALE = 192 ** -0.5


def make(B, T, Tk, H, seed=0, std=1.5):
    g = torch.Generator().manual_seed(1000 * seed + 7 * T + Tk + H)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"q": (n(B, T, H, 192) * std).to(BF).cuda(), "kv": n(B, Tk, H, 256).to(BF).cuda(), "k_pe": n(B, Tk, 64).to(BF).cuda(),
            "dy": n(B, T, H, 128).to(BF).cuda()}


def cu_of(lens):
    return torch.tensor(R.bounds(lens), dtype=torch.int64).cuda()


def run(a, causal, cu=None, cu_k=None, **kw):
    """The forward and its gradient: a dict of all outputs."""
    out, lse = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, causal, cu, cu_k, **kw)
    g = kda.latent_bwd(a["q"], a["kv"], a["k_pe"], SCALE, out, lse, a["dy"], causal, cu, cu_k, **kw)
    return {"out": out, "lse": lse} | g


def reference(a, res, causal, lens, lens_k):
    f = lambda t: d(t).reshape(-1, *t.shape[2:])  # noqa: E731
    ref = R.attention(f(a["q"]), f(a["kv"]), f(a["k_pe"]), SCALE, causal, lens, lens_k)
    return ref | R.attention_bwd(f(a["q"]), f(a["kv"]), f(a["k_pe"]), SCALE, causal, lens, lens_k, f(res["out"]), f(res["lse"]), f(a["dy"]))


def check(a, res, causal, lens, lens_k, label):
    ref = reference(a, res, causal, lens, lens_k)
    for k in ("out", "lse", "dq", "dkv", "dk_pe"):
        R.within(res[k].reshape(ref[k].shape), ref[k], ref["tol_" + k], "%s %s" % (label, k))


def same(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,T,Tk,H", [(1, 1, 1, 1), (2, 1, 5, 3), (1, 31, 31, 2), (1, 32, 33, 1), (2, 63, 63, 1), (1, 64, 64, 5),
                                      (1, 65, 66, 1), (1, 127, 127, 2), (1, 128, 128, 1), (1, 129, 129, 8), (2, 200, 333, 3),
                                      (1, 300, 300, 1), (1, 5, 700, 2), (1, 257, 40, 2), (3, 70, 1, 2), (1, 33, 0, 2)])
def test_lengths(B, T, Tk, H, causal):
    say("case latent %s causal=%s" % ((B, T, Tk, H), causal))
    a = make(B, T, Tk, H)
    res = run(a, causal)
    check(a, res, causal, [T] * B, [Tk] * B, "latent")
    if causal and T > Tk:  # queries ahead of the first key
        assert (res["out"][:, :T - Tk] == 0).all() and (res["lse"][:, :T - Tk] == float("-inf")).all()
        assert (res["dq"][:, :T - Tk] == 0).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,extra", [([1], [0]), ([70, 0, 1, 130, 64], [0] * 5), ([5, 200, 0, 3], [100, 0, 7, 65]),
                                        ([128, 128, 256], [0, 64, 0]), ([0, 0], [0, 0]), ([1] * 70, [0] * 70),
                                        ([10, 20], [-4, -20])])
def test_packed(lens, extra, causal):
    say("case latent packed %s + %s causal=%s" % (lens, extra, causal))
    lens_k = [p + e for p, e in zip(lens, extra)]
    H, tail = 3, 9
    a = make(1, sum(lens) + tail, sum(lens_k) + tail, H, seed=1)
    cu, cu_k = cu_of(lens), None if lens == lens_k else cu_of(lens_k)
    outs = {"dq": torch.full_like(a["q"], 7.0), "dkv": torch.full_like(a["kv"], 7.0), "dk_pe": torch.full_like(a["k_pe"], 7.0)}
    out = torch.full((1, sum(lens) + tail, H, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((1, sum(lens) + tail, H), 7.0, device="cuda")
    kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, causal, cu, cu_k, out=out, lse=lse)
    res = {"out": out, "lse": lse} | kda.latent_bwd(a["q"], a["kv"], a["k_pe"], SCALE, out, lse, a["dy"], causal, cu, cu_k, outputs=outs)
    for k, v in res.items():  # rows behind the last sequence stay
        assert (v[:, (sum(lens_k) if k in ("dkv", "dk_pe") else sum(lens)):] == 7.0).all(), k
    cut = {k: v[:, :sum(lens_k) if k in ("kv", "k_pe") else sum(lens)] for k, v in a.items()}
    res = {k: v[:, :sum(lens_k) if k in ("dkv", "dk_pe") else sum(lens)] for k, v in res.items()}
    check(cut, res, causal, lens, lens_k, "packed")


def test_packed_is_the_sequences_one_by_one():
    lens, ctx = [300, 1, 0, 129, 64], [0, 50, 3, 200, 0]
    lens_k = [p + c for p, c in zip(lens, ctx)]
    a = make(1, sum(lens), sum(lens_k), 4, seed=2)
    whole = run(a, True, cu_of(lens), cu_of(lens_k))
    q0 = k0 = 0
    for p, k in zip(lens, lens_k):
        one = {n: (v[:, k0:k0 + k] if n in ("kv", "k_pe") else v[:, q0:q0 + p]) for n, v in a.items()}
        res = run(one, True)
        for n, v in res.items():
            w = whole[n][:, k0:k0 + k] if n in ("dkv", "dk_pe") else whole[n][:, q0:q0 + p]
            assert torch.equal(v, w), n
        q0, k0 = q0 + p, k0 + k


def test_gradient_of_the_definition():
    """The kernels' gradient is that of the formulas in 64 bits by autograd, which central differences pin; the
    stored output's rounding (2^-8) enters by way of delta."""
    T, Tk, H = 70, 90, 2
    a = make(1, T, Tk, H, seed=3, std=0.7)
    res = run(a, True)
    leaves = {k: d(a[k])[0].clone().requires_grad_() for k in ("q", "kv", "k_pe")}

    def loss(**over):
        x = {k: v.detach() for k, v in leaves.items()} | over
        see = R.visible(T, Tk, True)
        p, _ = R.softmax(x["q"].transpose(0, 1) @ R.keys_of(x["kv"], x["k_pe"]).transpose(0, 1).transpose(1, 2) * SCALE, see)
        return ((p @ x["kv"][..., 128:].transpose(0, 1)).transpose(0, 1) * d(a["dy"])[0]).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss(**leaves), list(leaves.values()))))
    for k, v in leaves.items():
        step = torch.randn(v.shape, dtype=torch.float64)
        diff = (loss(**{k: v.detach() + 1e-5 * step}) - loss(**{k: v.detach() - 1e-5 * step})) / 2e-5
        assert abs(float(diff - (grads[k] * step).sum())) <= 1e-6 * float((grads[k] * step).abs().sum())
    ref = reference(a, res, True, [T], [Tk])
    f = lambda t: d(t)[0]  # noqa: E731
    p, _ = R.softmax(f(a["q"]).transpose(0, 1) @ R.keys_of(f(a["kv"]), f(a["k_pe"])).transpose(0, 1).transpose(1, 2) * SCALE, R.visible(T, Tk, True))
    # delta's error from the rounding of out, over p, times k (or q)
    e = p * SCALE * R.HALF * (f(a["dy"]).abs() * f(res["out"]).abs()).sum(-1).transpose(0, 1)[..., None] * 1.01
    ks, qs = R.keys_of(f(a["kv"]), f(a["k_pe"])).transpose(0, 1).abs(), f(a["q"]).transpose(0, 1).abs()
    more = {"dq": (e @ ks).transpose(0, 1), "dkv": torch.cat([(e.transpose(1, 2) @ qs)[..., :128], torch.zeros(H, Tk, 128)], -1).transpose(0, 1),
            "dk_pe": (e.transpose(1, 2) @ qs)[..., 128:].sum(0)}
    for k, g in zip(("dq", "dkv", "dk_pe"), (grads["q"], grads["kv"], grads["k_pe"])):
        # (tolerances of the formula's test, which take the values' own rounding from values off by `more`)
        R.within(res[k][0], g, ref["tol_" + k] + more[k] * (1 + R.HALF) + R.HALF * 0.02 * g.abs(), k)


def test_strides_and_broadcasts():
    B, T, H = 2, 150, 3
    a = make(B, T, T, H, seed=4)
    want = run(a, True)
    wide = {"q": torch.randn(B, T, H * 192 + 64, device="cuda").to(BF), "kv": torch.randn(B, T + 5, H * 256 + 8, device="cuda").to(BF),
            "k_pe": torch.randn(B, T, 576, device="cuda").to(BF), "dy": torch.randn(B, T, H * 128 + 16, device="cuda").to(BF)}
    s = {"q": wide["q"][..., 64:].unflatten(-1, (H, 192)), "kv": wide["kv"][:, 5:, 8:].unflatten(-1, (H, 256)),
         "k_pe": wide["k_pe"][..., 512:], "dy": wide["dy"][..., :H * 128].unflatten(-1, (H, 128))}
    for k, v in s.items():
        v.copy_(a[k])
    same(run(s, True), want)
    same(run({k: v.transpose(0, 1).contiguous().transpose(0, 1) for k, v in a.items()}, True), want)  # batch inside
    for dim in (0, 1):
        e = {k: v.narrow(dim, 0, 1).expand(v.shape) for k, v in a.items()}
        same(run(e, True), run({k: v.contiguous() for k, v in e.items()}, True))
    small = a["kv"][:1].clone().requires_grad_()
    kda.latent_attention(a["q"], small.expand(a["kv"].shape), a["k_pe"], SCALE).backward(a["dy"])
    each = run(a | {"kv": a["kv"][:1].expand(a["kv"].shape).contiguous()}, True)["dkv"]
    # autograd adds the bf16 gradients of the batch's rows: one rounding more
    R.within(small.grad, d(each).sum(0, keepdim=True), R.HALF * d(each).sum(0, keepdim=True).abs() + 1e-30, "broadcast kv")


@pytest.mark.parametrize("packed", [False, True])
def test_long_sequences(packed):
    """Sizes at which a workgroup takes 256 queries: the heads' bits are those of fewer heads, which take 128, and
    hidden values that are not finite stay where they are."""
    T, H = 2100, 64
    lens = [T + 30, T - 30] if packed else [T]
    say("case latent long packed=%s" % packed)
    a = make(1, sum(lens), sum(lens), H, seed=17)
    cu = cu_of(lens) if packed else None
    a["kv"][0, T - 60, 5, 130] = float("nan")
    a["kv"][0, T - 70, 63, 3] = float("inf")
    out, lse = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, True, cu)
    for h in (0, 24, 48):
        q, kv = a["q"][:, :, h:h + 16].contiguous(), a["kv"][:, :, h:h + 16].contiguous()
        few = kda.latent_fwd(q, kv, a["k_pe"], SCALE, True, cu)
        same({"out": out[:, :, h:h + 16].contiguous(), "lse": lse[:, :, h:h + 16].contiguous()}, {"out": few[0], "lse": few[1]})
    assert out[0, :, 5, 2].isnan().nonzero().flatten().tolist() == list(range(T - 60, lens[0]))
    f = lambda t: d(t)[0]  # noqa: E731
    ref = R.attention(f(a["q"][:, :, 31:32]), f(a["kv"][:, :, 31:32]), f(a["k_pe"]), SCALE, True, lens, lens)
    R.within(out[0, :, 31:32], ref["out"], ref["tol_out"], "out")
    R.within(lse[0, :, 31:32], ref["lse"], ref["tol_lse"], "lse")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v", "pe"])
def test_hidden_special_values(where, bad):
    """A value that is not finite reaches the queries that see its key, and leaves the others' bits alone."""
    T, Tk, H, j = 210, 230, 2, 150
    a = make(1, T, Tk, H, seed=5)
    want, lse = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE)
    b = {k: v.clone() for k, v in a.items()}
    if where == "pe":
        b["k_pe"][0, j, 3] = bad
    else:
        b["kv"][0, j, 1, 17 + (128 if where == "v" else 0)] = bad
    out, lse2 = kda.latent_fwd(b["q"], b["kv"], b["k_pe"], SCALE)
    first = j - (Tk - T)  # the first query that sees key j
    assert torch.equal(out[:, :first], want[:, :first]) and torch.equal(lse[:, :first], lse2[:, :first])
    if where != "pe":
        assert torch.equal(out[:, :, 0], want[:, :, 0])  # the other head
    seen = out[0, first:, 1]
    if where == "v":
        keep = torch.arange(128, device="cuda") != 17
        assert torch.equal(seen[:, keep], want[0, first:, 1][:, keep]) and torch.equal(lse, lse2)
        assert (seen[:, 17].isnan() if bad != bad else seen[:, 17] == bad).all()
    elif bad != bad:
        assert seen.isnan().all()


def test_special_values_in_another_sequence():
    lens = [70, 90, 33]
    a = make(1, sum(lens), sum(lens), 2, seed=6)
    want = run(a, True, cu_of(lens))
    for k in a:
        a[k][:, 70:160] = float("nan")
    got = run(a, True, cu_of(lens))
    for k in want:
        assert torch.equal(got[k][:, :70], want[k][:, :70]) and torch.equal(got[k][:, 160:], want[k][:, 160:]), k
        assert got[k][:, 70:160].isnan().all()


def test_large_scores_and_equal_scores():
    """Scores of some hundreds (one key takes all) and all the same (every key as much)."""
    a = make(1, 100, 100, 2, seed=7, std=40.0)
    check(a, run(a, True), True, [100], [100], "large")
    a["q"].zero_()
    res = run(a, False)
    check(a, res, False, [100], [100], "equal")
    assert torch.allclose(res["lse"], torch.full_like(res["lse"], 100.0).log(), atol=1e-5)


def test_offsets_beyond_32_bits():
    """Keys and values of more than 2^32 bytes and 2^31 entries: the last queries of a long context, heads apart."""
    T, Tk, H = 70, 70000, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(1, T, H, 192, generator=g, device="cuda").to(BF)
    kv = torch.empty(1, Tk, H, 256, dtype=BF, device="cuda").normal_(generator=g)
    pe = torch.randn(1, Tk, 64, generator=g, device="cuda").to(BF)
    dy = torch.randn(1, T, H, 128, generator=g, device="cuda").to(BF)
    assert kv.numel() > 1 << 31
    say("case latent 2^31 entries")
    res = run({"q": q, "kv": kv, "k_pe": pe, "dy": dy}, True)
    for h in (0, 77, 127):
        one = {"q": q[:, :, h:h + 1], "kv": kv[:, :, h:h + 1], "k_pe": pe, "dy": dy[:, :, h:h + 1]}
        one = {k: v.contiguous() for k, v in one.items()}
        got = kda.latent_bwd(one["q"], one["kv"], pe, SCALE, res["out"][:, :, h:h + 1], res["lse"][:, :, h:h + 1].contiguous(), one["dy"])
        for k in ("dq", "dkv"):
            assert torch.equal(got[k][:, :, 0], res[k][:, :, h]), (h, k)
        f = lambda t: d(t)[0]  # noqa: E731
        ref = R.attention(f(one["q"]), f(one["kv"]), f(pe), SCALE, True, [T], [Tk])
        for out, lse in ((res["out"][0, :, h:h + 1], res["lse"][0, :, h:h + 1]), [t[0] for t in kda.latent_fwd(one["q"], one["kv"], pe, SCALE)]):
            R.within(out, ref["out"], ref["tol_out"], "out")
            R.within(lse, ref["lse"], ref["tol_lse"], "lse")


def test_launch_pieces_and_repeats():
    a = make(2, 300, 300, 5, seed=8)
    want = run(a, True)
    same(run(a, True), want)
    same(run(a, True, launch_piece=8), want)
    lens = [150, 0, 400, 50]
    b = {k: v.reshape(1, -1, *v.shape[2:]) for k, v in a.items()}
    want = run(b, True, cu_of(lens))
    for _ in range(3):
        same(run(b, True, cu_of(lens)), want)
    same(run(b, True, cu_of(lens), launch_piece=1), want)


@pytest.mark.parametrize("lens", [[1300], [900, 0, 1, 399]])
def test_gradient_in_one_and_in_two_launches(lens):
    """Many blocks take a launch of queries and one of keys, few of them one launch for both, or for parts of both."""
    H = 16
    say("case latent gradient of %s x %d heads" % (lens, H))
    a = make(1, sum(lens), sum(lens), H, seed=18)
    cu = cu_of(lens) if len(lens) > 1 else None
    res = run(a, True, cu)
    check(a, res, True, lens, lens, "many")
    for h, n in ((0, 8), (8, 8), (15, 1)):
        few = {k: (v if k == "k_pe" else v[:, :, h:h + n].contiguous()) for k, v in a.items()}
        out, lse = res["out"][:, :, h:h + n].contiguous(), res["lse"][:, :, h:h + n].contiguous()
        got = kda.latent_bwd(few["q"], few["kv"], few["k_pe"], SCALE, out, lse, few["dy"], True, cu)
        if n == 8:  # not in parts
            same({k: got[k] for k in ("dq", "dkv")}, {k: res[k][:, :, h:h + n].contiguous() for k in ("dq", "dkv")})
        check(few, {"out": out, "lse": lse} | got, True, lens, lens, "few")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,T,Tk,H", [(1, 1, 5000, 1), (1, 64, 4097, 2), (2, 130, 2500, 3), (1, 1500, 1500, 1), (1, 1000, 900, 2)])
def test_few_queries_with_many_keys(B, T, Tk, H, causal):
    """Keys in parts, which are joined: also where the first blocks see one part or no key, and a NaN that some see."""
    say("case latent parts %s causal=%s" % ((B, T, Tk, H), causal))
    a = make(B, T, Tk, H, seed=19)
    want = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, causal)
    res = run(a, causal)
    check(a, res, causal, [T] * B, [Tk] * B, "parts")
    for piece in (0, 8):
        same(run(a, causal, launch_piece=piece), res)
    j = Tk - 1 - min(T, Tk) // 2  # seen by the last queries
    a["kv"][0, j, 0, 200] = float("nan")
    out, lse = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, causal)
    first = max(0, j - (Tk - T)) if causal else 0
    assert torch.equal(lse, want[1]) and out[0, first:, 0, 72].isnan().all()
    out[0, first:, 0, 72] = want[0][0, first:, 0, 72]
    assert torch.equal(out, want[0])


def test_packed_parts_in_a_graph():
    lens, ctx = [5, 200, 0, 3, 129], [2000, 0, 7, 900, 1300]
    lens_k = [p + c for p, c in zip(lens, ctx)]
    H, tail = 2, 6
    a = make(1, sum(lens) + tail, sum(lens_k) + tail, H, seed=20)
    cu, cu_k = cu_of(lens), cu_of(lens_k)
    need = kda.latent_workspace_size(1, sum(lens) + tail, sum(lens_k) + tail, H, num_seqs=5)
    assert need > 1 << 20
    need = max(need, kda.latent_bwd_workspace_size(1, sum(lens) + tail, sum(lens_k) + tail, H, num_seqs=5))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.full((1, sum(lens) + tail, H, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((1, sum(lens) + tail, H), 7.0, device="cuda")
    grads = {"dq": torch.full_like(a["q"], 7.0), "dkv": torch.full_like(a["kv"], 7.0), "dk_pe": torch.full_like(a["k_pe"], 7.0)}
    res = {"out": out, "lse": lse} | grads

    def call(cu, cu_k):
        kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, True, cu, cu_k, out=out, lse=lse, workspace=ws)
        kda.latent_bwd(a["q"], a["kv"], a["k_pe"], SCALE, out, lse, a["dy"], True, cu, cu_k, workspace=ws, outputs=grads)

    def compare(lens, lens_k):
        n = {k: sum(lens_k) if k in ("kv", "k_pe", "dkv", "dk_pe") else sum(lens) for k in list(a) + list(res)}
        check({k: v[:, :n[k]] for k, v in a.items()}, {k: v[:, :n[k]] for k, v in res.items()}, True, lens, lens_k, "parts")
        for k, v in res.items():
            assert (v[:, n[k]:] == 7.0).all(), k
    call(cu, cu_k)
    compare(lens, lens_k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(cu, cu_k)
    for p, k in (([5, 200, 0, 3, 129], lens_k), ([100, 1, 1, 35, 200], [100, 1, 4000, 35, 200]), ([0, 0, 0, 337, 0], [1, 2, 3, 4300, 0])):
        cu.copy_(cu_of(p))
        cu_k.copy_(cu_of(k))
        for v in res.values():
            v.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        compare(p, k)


def test_many_short_sequences():
    n = 3000
    lens = [(7 * i) % 5 for i in range(n)]
    a = make(1, sum(lens), sum(lens), 1, seed=9)
    res = run(a, True, cu_of(lens))
    check(a, res, True, lens, lens, "short")


def test_wrong_offsets_stay_inside():
    a = make(1, 200, 200, 2, seed=10)
    for bad in ([0, 300, 100, 200], [-5, 50, 1 << 40, 200], [0, 1 << 62, -(1 << 62), 7]):
        cu = torch.tensor(bad, dtype=torch.int64).cuda()
        res = run(a, True, cu)
        torch.cuda.synchronize()
        assert res["out"].shape == (1, 200, 2, 128)


def test_autograd():
    a = make(2, 90, 90, 3, seed=11)
    leaves = [a[k].clone().requires_grad_() for k in ("q", "kv", "k_pe")]
    out = kda.latent_attention(*leaves, SCALE)
    out.backward(a["dy"])
    want = run(a, True)
    assert torch.equal(out, want["out"])
    for t, k in zip(leaves, ("dq", "dkv", "dk_pe")):
        assert torch.equal(t.grad, want[k]), k
    lens = [100, 0, 60]
    flat = [t.detach().reshape(1, -1, *t.shape[2:]).clone().requires_grad_() for t in leaves]
    y = kda.latent_attention(*flat, SCALE, True, cu_of(lens))
    y.backward(a["dy"].reshape(1, -1, 3, 128))
    assert (y[:, 160:] == 0).all()
    for t in flat:
        assert (t.grad[:, 160:] == 0).all() and t.grad[:, :160].abs().sum() > 0


def test_graph_with_a_shared_workspace():
    sets = [make(1, T, T, 2, seed=12) for T in (140, 520)]
    lens = [[100, 40], [1, 519]]
    cus = [cu_of(v) for v in lens]
    ws = torch.empty(max(kda.latent_bwd_workspace_size(1, T, T, 2, 2) for T in (140, 520)), dtype=torch.uint8, device="cuda")
    want = [run(a, True, c) for a, c in zip(sets, cus)]
    outs = [{k: torch.empty_like(v) for k, v in w.items()} for w in want]

    def call(i):
        a, o = sets[i], outs[i]
        kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, True, cus[i], out=o["out"], lse=o["lse"], workspace=ws)
        kda.latent_bwd(a["q"], a["kv"], a["k_pe"], SCALE, o["out"], o["lse"], a["dy"], True, cus[i], workspace=ws, outputs=o)
    graphs = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        for o in outs:
            for t in o.values():
                t.zero_()
        for i in (rep % 2, 1 - rep % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            same(o, w)
    # a replay goes by the offsets that stand there then
    new = cu_of([40, 100])
    cus[0].copy_(new)
    fresh = run(sets[0], True, new)
    graphs[0].replay()
    torch.cuda.synchronize()
    same(outs[0], fresh)


def test_backward_in_a_graph():
    a = make(1, 130, 130, 2, seed=13)
    want = run(a, True)
    leaves = [a[k].clone().requires_grad_() for k in ("q", "kv", "k_pe")]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = kda.latent_attention(*leaves, SCALE)
        y.backward(a["dy"])
        del y
        for t in leaves:
            t.grad = None
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = kda.latent_attention(*leaves, SCALE)
        y.backward(a["dy"])
    for _ in range(3):
        for t in leaves:
            t.grad.zero_()
        g.replay()
        torch.cuda.synchronize()
        for t, k in zip(leaves, ("dq", "dkv", "dk_pe")):
            assert torch.equal(t.grad, want[k]), k


def test_two_streams():
    sets = [make(1, T, T, 3, seed=14) for T in (300, 700)]
    want = [run(a, True) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for a, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(a, True))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        same(g, want[i % 2])


def test_without_a_workspace():
    """The C ABI takes its workspace on the stream when it is given none."""
    from gated_delta_rule_110_amd import latent as L
    a = make(1, 200, 200, 2, seed=15)
    cu = cu_of([70, 130])
    want = run(a, True, cu)
    got = {k: torch.empty_like(v) for k, v in want.items()}
    dsc, dev = L._latent_args(a["q"], a["kv"], a["k_pe"], SCALE, True, cu, None)
    dsc.out_stride_b = dsc.d_out_stride_b = 0
    dsc.out_stride_t = dsc.d_out_stride_t = 2 * 128
    lib, st = kda.library(), torch.cuda.current_stream().cuda_stream
    ptr = lambda *n: [x.data_ptr() for x in n]  # noqa: E731
    assert lib.kda_latent_fwd(*ptr(a["q"], a["kv"], a["k_pe"], cu), None, *ptr(got["out"], got["lse"]), dsc, st) == 0
    assert lib.kda_latent_bwd(*ptr(a["q"], a["kv"], a["k_pe"], cu), None, *ptr(got["out"], got["lse"], a["dy"]),
                              *ptr(got["dq"], got["dkv"], got["dk_pe"]), dsc, st) == 0
    torch.cuda.synchronize()
    same(got, want)


def test_validated_offsets(monkeypatch):
    monkeypatch.setenv("KDA_VALIDATE", "1")
    a = make(1, 50, 50, 1, seed=16)
    run(a, True, cu_of([20, 30]))
    for bad in ([0, 60], [0, 30, 20], [1, 50]):
        with pytest.raises(ValueError):
            run(a, True, torch.tensor(bad, dtype=torch.int64).cuda())
    with pytest.raises(ValueError):
        run(a, True, cu_of([50]), torch.tensor([0, 51], dtype=torch.int64).cuda())
