"""Latent attention's C ABI on the host: exported symbols, argument checks that
return before any device work, workspace sizes, refusals of the binding; and the
oracle's own pins."""
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_110_amd as kda
from gated_delta_rule_110_amd import latent as L
from tests import latent_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, UNSUPPORTED, PARAM, DTYPE, ALIGN, WORKSPACE, OVERLAP = 1, 2, 3, 4, 5, 6, 7, 10


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        kda.build()
    return kda.library()


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "kda_latent.h")) as f:
        names = sorted(set(re.findall(r"^\S.*?\b(kda_\w+)\s*\(", f.read(), flags=re.M)))
    assert len(names) == 9
    dyn = subprocess.run(["nm", "-D", "--defined-only", kda.LIB_PATH], capture_output=True, text=True).stdout
    for n in names:
        assert re.search(r"\bT %s$" % n, dyn, flags=re.M), n


def p(i, off=0):
    """The i-th of some addresses far apart; never dereferenced: every call below is refused on the host."""
    return (i + 1 << 40) + off


def latent(lib, which="fwd", args=None, **kw):
    B, T, H = 2, 40, 3
    dsc = L.KdaLatentDesc(B, T, T, H, B, T * H * 192, H * 192, T * H * 256, H * 256, T * 64, 64, T * H * 128, H * 128, T * H * 128, H * 128,
                          0.1, 1, p(20), 1 << 40, 0)
    for k, v in kw.items():
        setattr(dsc, k, v)
    a = dict(q=p(0), kv=p(1), pe=p(2), cu=None, cuk=None, out=p(3), lse=p(4), dy=p(5), dq=p(6), dkv=p(7), dpe=p(8))
    a.update(args or {})
    head = [a[k] for k in ("q", "kv", "pe", "cu", "cuk", "out", "lse")]
    if which == "fwd":
        return lib.kda_latent_fwd(*head, dsc, None)
    return lib.kda_latent_bwd(*head, *[a[k] for k in ("dy", "dq", "dkv", "dpe")], dsc, None)


def test_latent_checks(lib):
    for which in ("fwd", "bwd"):
        for k in ("q", "kv", "pe", "out") + (() if which == "fwd" else ("lse", "dy", "dq", "dkv", "dpe")):
            assert latent(lib, which, {k: None}) == NULL, (which, k)
        assert latent(lib, which, {"cuk": p(9)}) == NULL
        for bad in (dict(B=0), dict(T=-1), dict(Tk=-1), dict(H=0), dict(H=1 << 16), dict(num_seqs=1), dict(T=1 << 31), dict(Tk=1 << 31),
                    dict(q_stride_t=-8), dict(kv_stride_t=1 << 24), dict(pe_stride_b=1 << 41)):
            assert latent(lib, which, **bad) == SHAPE, (which, bad)
        assert latent(lib, which, {"cu": p(9)}) == SHAPE                                  # packed: one batch row
        assert latent(lib, which, {"cu": p(9)}, B=1, num_seqs=2, Tk=41) == SHAPE          # two numbers of tokens, one table
        for bad in (dict(q_stride_t=12), dict(kv_stride_b=4), dict(pe_stride_t=65)):
            assert latent(lib, which, **bad) == ALIGN, (which, bad)
        for k in ("q", "kv", "pe", "out"):
            assert latent(lib, which, {k: p(15, 8)}) == ALIGN, (which, k)
        assert latent(lib, which, {"lse": p(4, 2)}) == ALIGN
        assert latent(lib, which, {"cu": p(9, 4)}, B=1, num_seqs=2) == ALIGN
        for e in (0.0, -1.0, float("nan"), float("inf")):
            assert latent(lib, which, scale=e) == PARAM
        assert latent(lib, which, causal=2) == PARAM and latent(lib, which, launch_piece=-1) == PARAM
    assert latent(lib, "fwd", {"out": p(0)}) == OVERLAP and latent(lib, "fwd", {"lse": p(2, 64)}) == OVERLAP
    assert latent(lib, "bwd", {"dq": p(0)}) == OVERLAP and latent(lib, "bwd", {"dpe": p(7, 16)}) == OVERLAP
    assert latent(lib, "bwd", {"dkv": p(20)}) == OVERLAP
    assert latent(lib, "bwd", out_stride_t=-8) == SHAPE and latent(lib, "bwd", d_out_stride_t=4) == ALIGN
    assert latent(lib, "bwd", workspace_bytes=256) == WORKSPACE and latent(lib, "bwd", workspace=p(20, 8)) == ALIGN
    assert latent(lib, "fwd", {"cu": p(9)}, B=1, num_seqs=2, workspace_bytes=8) == WORKSPACE
    # few queries with many keys: the parts of their keys
    assert latent(lib, "fwd", T=1, Tk=9000, H=1, workspace_bytes=256) == WORKSPACE
    assert latent(lib, "fwd", T=1, Tk=9000, H=1, workspace=p(20, 8)) == ALIGN


def test_latent_workspaces(lib):
    assert kda.latent_workspace_size(2, 100, 100, 4) == 0
    assert kda.latent_workspace_size(1, 1000, 1000, 4, num_seqs=9) > 0
    # one token of one head over many keys: accumulators and statistics of 128 rows of every part
    assert kda.latent_workspace_size(2, 1, 100000, 1) % (128 * 130 * 4) == 0 and kda.latent_workspace_size(2, 8000, 8000, 16) == 0
    assert kda.latent_bwd_workspace_size(2, 100, 300, 4) >= 2 * 300 * 4 * 64 * 4 + 2 * 100 * 4 * 8
    assert kda.latent_bwd_workspace_size(1, 200, 600, 4, num_seqs=3) > kda.latent_bwd_workspace_size(1, 200, 600, 3, num_seqs=3)
    for bad in ((0, 8, 8, 1), (1, -1, 8, 1), (1, 8, 8, 0), (2, 8, 8, 1, 3)):
        assert kda.latent_bwd_workspace_size(*bad) == 0
    assert kda.latent_decode_workspace_size(4, 1, 16) > 0 and kda.latent_decode_workspace_size(4, 0, 16) == 0
    assert kda.latent_decode_workspace_size(1 << 20, 1, 128) == 0
    # the parts of a row tile that workgroups share do not grow with the batch
    assert kda.latent_decode_workspace_size(1 << 16, 1, 32) - kda.latent_decode_workspace_size(1, 1, 32) <= 8 * (1 << 16) + 256


def decode(lib, args=None, **kw):
    dsc = L.KdaLatentDecodeDesc(2, 3, 4, 10, 16, 5, 3 * 4 * 512, 4 * 512, 512, 3 * 4 * 64, 4 * 64, 64, 0.1, p(20), 1 << 40)
    for k, v in kw.items():
        setattr(dsc, k, v)
    a = dict(ql=p(0), qp=p(1), cache=p(2), len=p(3), table=p(4), out=p(5), lse=p(6))
    a.update(args or {})
    return lib.kda_latent_decode(*a.values(), dsc, None)


def test_decode_checks(lib):
    for k in ("ql", "qp", "cache", "len", "table", "out"):
        assert decode(lib, {k: None}) == NULL, k
    for bad in (dict(N=-1), dict(T=0), dict(H=0), dict(pages=-1), dict(max_pages=-1), dict(N=1 << 24), dict(T=1 << 24), dict(H=1 << 16),
                dict(max_pages=1 << 30), dict(ql_stride_n=-8), dict(qp_stride_h=1 << 41)):
        assert decode(lib, **bad) == SHAPE, bad
    for bad in (0, 3, 24, 1 << 17, -16):
        assert decode(lib, page_size=bad) == UNSUPPORTED
    assert decode(lib, scale=0.0) == PARAM and decode(lib, scale=float("nan")) == PARAM
    assert decode(lib, ql_stride_h=12) == ALIGN and decode(lib, qp_stride_n=4) == ALIGN
    for k, off in (("ql", 8), ("qp", 8), ("cache", 8), ("out", 8), ("len", 4), ("table", 2), ("lse", 2)):
        assert decode(lib, {k: p(15, off)}) == ALIGN, k
    assert decode(lib, {"out": p(2)}) == OVERLAP and decode(lib, {"lse": p(3)}) == OVERLAP and decode(lib, {"out": p(20, 64)}) == OVERLAP
    assert decode(lib, workspace_bytes=256) == WORKSPACE and decode(lib, workspace=p(20, 16)) == ALIGN


def store(lib, args=None, **kw):
    dsc = L.KdaLatentStoreDesc(6, 32, 576, 576, 2, 1e-6)
    for k, v in kw.items():
        setattr(dsc, k, v)
    a = dict(latent=p(0), pe=p(0, 1024), w=p(1), slots=p(2), cache=p(3), normed=p(4))
    a.update(args or {})
    return lib.kda_latent_store(*a.values(), dsc, None)


def test_store_checks(lib):
    for k in ("latent", "pe", "slots", "cache"):
        assert store(lib, {k: None}) == NULL, k
    for bad in (dict(tokens=-1), dict(num_slots=-1), dict(latent_stride=-8), dict(pe_stride=1 << 41), dict(tokens=1 << 41)):
        assert store(lib, **bad) == SHAPE, bad
    assert store(lib, weight_dtype=0) == DTYPE
    for e in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -127):
        assert store(lib, eps=e) == PARAM
    assert store(lib, latent_stride=513) == ALIGN and store(lib, pe_stride=65) == ALIGN
    for k, off in (("latent", 8), ("pe", 8), ("cache", 8), ("normed", 8), ("slots", 4), ("w", 2)):
        assert store(lib, {k: p(15, off)}) == ALIGN, k
    assert store(lib, {"cache": p(0)}) == OVERLAP and store(lib, {"normed": p(3, 1152)}) == OVERLAP


def pages(lib, args=None, **kw):
    dsc = L.KdaPageDesc(4, 8, 16, 100, 50, p(20), 1 << 20)
    for k, v in kw.items():
        setattr(dsc, k, v)
    a = dict(len=p(0), add=p(1), ended=p(2), table=p(3), free=p(4), count=p(5), slots=p(6), cu=p(7), out=p(8), got=p(9), left=p(10))
    a.update(args or {})
    return lib.kda_page_assign(*a.values(), dsc, None)


def test_page_checks(lib):
    for k in ("len", "add", "table", "free", "count", "slots", "cu", "out", "got", "left"):
        assert pages(lib, {k: None}) == NULL, k
    for bad in (dict(N=-1), dict(max_pages=-1), dict(stack=-1), dict(tokens=-1), dict(N=1 << 21), dict(max_pages=1 << 30), dict(tokens=1 << 31),
                dict(stack=1 << 31)):
        assert pages(lib, **bad) == SHAPE, bad
    for bad in (0, 48, 1 << 17):
        assert pages(lib, page_size=bad) == UNSUPPORTED
    for k in ("len", "add", "count", "slots", "cu", "out", "got", "left"):
        assert pages(lib, {k: p(15, 4)}) == ALIGN, k
    assert pages(lib, {"table": p(3, 2)}) == ALIGN
    for k, at in (("slots", 0), ("out", 1), ("got", 0), ("left", 1), ("cu", 6), ("table", 4), ("out", 20)):
        assert pages(lib, {k: p(at)}) == OVERLAP, (k, at)
    assert pages(lib, {"out": p(0, 8)}) == OVERLAP
    assert pages(lib, workspace_bytes=8) == WORKSPACE and pages(lib, workspace=p(20, 8)) == ALIGN


def test_binding_refusals():
    bf = torch.bfloat16
    q, kv, pe = torch.zeros(1, 4, 2, 192, dtype=bf), torch.zeros(1, 4, 2, 256, dtype=bf), torch.zeros(1, 4, 64, dtype=bf)
    cache, lens = torch.zeros(2, 16, 576, dtype=bf), torch.zeros(1, dtype=torch.int64)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for bad in (lambda: kda.latent_fwd(q, kv, pe, 0.1), lambda: kda.latent_attention(q, kv, pe, 0.1),
                lambda: kda.latent_bwd(q, kv, pe, 0.1, q[..., :128], q[..., 0].float(), q[..., :128]),
                lambda: kda.latent_decode(torch.zeros(1, 1, 2, 512, dtype=bf), torch.zeros(1, 1, 2, 64, dtype=bf), cache, lens, table, 0.1),
                lambda: kda.latent_store(torch.zeros(3, 512, dtype=bf), torch.zeros(3, 64, dtype=bf), lens, cache),
                lambda: kda.page_assign(lens, lens, table, table[0], lens, 16, 4)):
        with pytest.raises(ValueError):
            bad()


def test_the_oracle():
    """The oracle's softmax against torch's, its gradient against autograd, its rows without keys."""
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    lens, lens_k = [5, 0, 7, 4], [5, 3, 9, 2]
    q, kv, pe, dy = n(16, 2, 192), n(19, 2, 256), n(19, 64), n(16, 2, 128)
    leaves = [t.clone().requires_grad_() for t in (q, kv, pe)]
    outs, q0, k0 = [], 0, 0
    for a, b in zip(lens, lens_k):
        x = leaves[0][q0:q0 + a].transpose(0, 1) @ R.keys_of(leaves[1][k0:k0 + b], leaves[2][k0:k0 + b]).transpose(0, 1).transpose(1, 2) * 0.1
        see = R.visible(a, b, True)
        w = torch.softmax(x.masked_fill(~see, float("-inf")), -1).masked_fill(~see.any(-1)[:, None], 0)
        outs.append((w @ leaves[1][k0:k0 + b, :, 128:].transpose(0, 1)).transpose(0, 1))
        q0, k0 = q0 + a, k0 + b
    y = torch.cat(outs)
    got = R.attention(q, kv, pe, 0.1, True, lens, lens_k)
    assert torch.allclose(got["out"], y, atol=1e-12) and (got["lse"][12:14] == float("-inf")).all() and (got["out"][12:14] == 0).all()
    live = torch.ones(16, dtype=torch.bool)
    live[12:14] = False
    grads = torch.autograd.grad((y[live] * dy[live]).sum(), leaves)
    back = R.attention_bwd(q, kv, pe, 0.1, True, lens, lens_k, got["out"], got["lse"], dy)
    for k, t in zip(("dq", "dkv", "dk_pe"), grads):
        assert torch.allclose(back[k], t.nan_to_num(0.0), atol=1e-10), k
    # the absorbed form is the expanded one with one head's keys and values for all
    cache = n(3, 4, 576)
    ql, qp = n(1, 2, 3, 512), n(1, 2, 3, 64)
    table = torch.tensor([[2, 0, -1]])
    dec = R.decode(ql, qp, cache, [7], table, 0.05)
    rows = torch.cat([cache[2], cache[0]])[:7]
    x = torch.cat([ql, qp], -1)[0, 1] @ rows.t() * 0.05
    assert torch.allclose(dec["out"][0, 1], torch.softmax(x, -1) @ rows[:, :512], atol=1e-12)
    assert torch.allclose(dec["lse"][0, 1], torch.logsumexp(x, -1), atol=1e-12)
    x = torch.cat([ql, qp], -1)[0, 0] @ rows[:6].t() * 0.05
    assert torch.allclose(dec["out"][0, 0], torch.softmax(x, -1) @ rows[:6, :512], atol=1e-12)
    got = R.pages([3, 4, 8], [2, 1, 1], [[7, -1], [8, -1], [9, 6]], [1, 2, 3, 0], 3, 4, 4, [False, False, True])
    # the third's pages 9 and 6 go back ([1, 2, 3, 9]: the stack is full), then 9, 3 and 2 are taken
    assert got["slots"] == [31, 36, 12, 8] and got["table"] == [[7, 9], [8, 3], [2, 6]] and got["free_count"] == [1]
    assert got["lengths"] == [5, 5, 1] and got["cu_seqlens"] == [0, 2, 3, 4] and got["free"] == [1, 2, 3, 9]
