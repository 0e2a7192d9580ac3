"""The layer operators' C ABI on the host: exported symbols, argument checks
that return before any device work, workspace sizes, refusals of the binding."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_110_amd as kda
from gated_delta_rule_110_amd import layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, UNSUPPORTED, PARAM, DTYPE, ALIGN, WORKSPACE, OVERLAP = 1, 2, 3, 4, 5, 6, 7, 10


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        kda.build()
    return kda.library()


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "kda_layer.h")) as f:
        names = sorted(set(re.findall(r"^\S.*?\b(kda_\w+)\s*\(", f.read(), flags=re.M)))
    assert len(names) == 14
    dyn = subprocess.run(["nm", "-D", "--defined-only", kda.LIB_PATH], capture_output=True, text=True).stdout
    for n in names:
        assert re.search(r"\bT %s$" % n, dyn, flags=re.M), n
    assert lib.kda_status_string(OVERLAP).startswith(b"a written tensor")


def p(i, off=0):
    """The i-th of some addresses far apart; never dereferenced: every call below is refused on the host."""
    return (i + 1 << 40) + off


def norm(lib, quant=False, args=None, **kw):
    d = L.KdaRmsnormDesc(4, 64, 64, 64, 2, 2, 1e-5, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    a = dict(x=p(0), res=p(1), w=p(2), res_out=p(3), out=p(4), scales=p(5))
    a.update(args or {})
    if quant:
        return lib.kda_rmsnorm_quant(a["x"], a["res"], a["w"], a["res_out"], a["out"], a["scales"], d, None)
    return lib.kda_rmsnorm_fwd(a["x"], a["res"], a["w"], a["res_out"], a["out"], d, None)


def test_rmsnorm_checks(lib):
    for q in (False, True):
        for k in ("x", "w", "out") + (("scales",) if q else ()):
            assert norm(lib, q, {k: None}) == NULL, k
        assert norm(lib, q, {"res": None}) == NULL            # residual_out without a residual
        assert norm(lib, q, rows=-1) == SHAPE and norm(lib, q, D=0) == SHAPE and norm(lib, q, x_stride=-1) == SHAPE
        assert norm(lib, q, rows=1 << 60) == SHAPE and norm(lib, q, D=1 << 40) == SHAPE
        assert norm(lib, q, residual_stride=-64) == SHAPE
        assert norm(lib, q, weight_dtype=3) == DTYPE and norm(lib, q, residual_dtype=0) == DTYPE
        for e in (0.0, -1.0, float("nan"), float("inf")):
            assert norm(lib, q, eps=e) == PARAM
        assert norm(lib, q, {"x": p(0, 1)}) == ALIGN and norm(lib, q, {"w": p(2, 2)}) == ALIGN
        assert norm(lib, q, {"res_out": p(1, 64)}) == OVERLAP and norm(lib, q, {"out": p(2, 16)}) == OVERLAP
        assert norm(lib, q, {"out": p(3)}) == OVERLAP
    assert norm(lib, True, group=64) == PARAM
    assert norm(lib, True, {"out": p(0)}) == OVERLAP          # 8-bit over 16-bit
    assert norm(lib, False, {"out": p(0)}, x_stride=128) == OVERLAP   # in place only where rows are contiguous


def norm_bwd(lib, args=None, **kw):
    d = L.KdaRmsnormDesc(4, 64, 64, 0, 2, 2, 1e-5, 0, 64, 64, p(9), 1 << 20)
    for k, v in kw.items():
        setattr(d, k, v)
    a = dict(h=p(0), w=p(1), dy=p(2), dres=p(3), dx=p(4), dr=p(5), dw=p(6))
    a.update(args or {})
    return lib.kda_rmsnorm_bwd(a["h"], a["w"], a["dy"], a["dres"], a["dx"], a["dr"], a["dw"], d, None)


def test_rmsnorm_bwd_checks(lib):
    for k in ("h", "w", "dy", "dx", "dw"):
        assert norm_bwd(lib, {k: None}) == NULL, k
    assert norm_bwd(lib, residual_dtype=1) == DTYPE           # an fp32 dresidual of a bf16 stream
    assert norm_bwd(lib, d_out_stride=-1) == SHAPE and norm_bwd(lib, d_residual_stride=-1) == SHAPE
    assert norm_bwd(lib, workspace_bytes=16) == WORKSPACE and norm_bwd(lib, workspace=p(9, 8)) == ALIGN
    assert norm_bwd(lib, {"dx": p(2)}) == OVERLAP and norm_bwd(lib, {"dw": p(9, 4)}) == OVERLAP
    assert kda.rmsnorm_bwd_workspace_size(4, 64) > 0 and kda.rmsnorm_bwd_workspace_size(-1, 64) == 0


def conv(lib, which="fwd", args=None, **kw):
    d = L.KdaConvDesc(2, 1 if which == "decode" else 10, 64, 4, 2, 640, 64, 640, 64, 1, 2, 2, 2, p(20), 1 << 30)
    for k, v in kw.items():
        setattr(d, k, v)
    a = dict(x=p(0), w=p(1), b=p(2), h0=p(3), ht=p(4), cu=None, out=p(5), dy=p(6), dht=p(7), dx=p(8), dw=p(9), db=p(10), dh0=p(11))
    a.update(args or {})
    if which == "fwd":
        return lib.kda_conv_fwd(a["x"], a["w"], a["b"], a["h0"], a["ht"], a["cu"], a["out"], d, None)
    if which == "decode":
        return lib.kda_conv_decode(a["x"], a["w"], a["b"], a["h0"], a["ht"], a["out"], d, None)
    return lib.kda_conv_bwd(a["x"], a["w"], a["b"], a["h0"], a["cu"], a["dy"], a["dht"], a["dx"], a["dw"], a["db"], a["dh0"], d, None)


def test_conv_checks(lib):
    for which in ("fwd", "decode", "bwd"):
        for k in ("x", "w") + {"fwd": ("out",), "decode": ("out", "ht"), "bwd": ("dy", "dx", "dw")}[which]:
            assert conv(lib, which, {k: None}) == NULL, (which, k)
        assert conv(lib, which, B=0) == SHAPE and conv(lib, which, T=-1) == SHAPE and conv(lib, which, num_seqs=3) == SHAPE
        assert conv(lib, which, D=0) == SHAPE and conv(lib, which, x_stride_t=-1) == SHAPE and conv(lib, which, T=1 << 50) == SHAPE
        assert conv(lib, which, W=1) == UNSUPPORTED and conv(lib, which, W=5) == UNSUPPORTED
        assert conv(lib, which, silu=2) == PARAM and conv(lib, which, weight_dtype=0) == DTYPE
        assert conv(lib, which, initial_state_dtype=0) == DTYPE and conv(lib, which, final_state_dtype=9) == DTYPE
        assert conv(lib, which, {"x": p(0, 1)}) == ALIGN and conv(lib, which, {"h0": p(3, 2)}) == ALIGN
    assert conv(lib, "decode", T=2) == SHAPE
    assert conv(lib, "fwd", {"cu": p(12)}) == SHAPE            # packed: one batch row
    assert conv(lib, "fwd", {"out": p(0, 128)}) == OVERLAP and conv(lib, "fwd", {"ht": p(3, 64)}) == OVERLAP
    assert conv(lib, "fwd", {"ht": p(3)}, final_state_dtype=1) == OVERLAP   # in place only for one type
    assert conv(lib, "decode", {"out": p(4)}) == OVERLAP
    assert conv(lib, "bwd", {"dx": p(6)}) == OVERLAP and conv(lib, "bwd", {"dw": p(20)}) == OVERLAP
    assert conv(lib, "bwd", workspace_bytes=8) == WORKSPACE and conv(lib, "bwd", workspace=p(20, 4)) == ALIGN
    assert conv(lib, "bwd", d_out_stride_t=-1) == SHAPE
    assert kda.conv_bwd_workspace_size(1, 100, 64, 4) > 0 and kda.conv_bwd_workspace_size(1, 100, 64, 5) == 0


def ssm(lib, which="fwd", args=None, **kw):
    T = 1 if which == "decode" else 10
    d = L.KdaSsmDesc(2, T, 4, 64, 2, 64, 2, T * 256, 256, T * 4, 4, T * 128, 128, T * 128, 128, T * 256, 256, 2, 2, p(30), 1 << 40, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    a = dict(x=p(0), dt=p(1), B=p(2), C=p(3), A=p(4), bias=p(5), D=p(6), h0=p(7), ht=p(8), cu=None, out=p(9), dy=p(10), dht=p(11),
             dx=p(12), ddt=p(13), dB=p(14), dC=p(15), dA=p(16), dbias=p(17), dD=p(18), dh0=p(19))
    a.update(args or {})
    head = [a[k] for k in ("x", "dt", "B", "C", "A", "bias", "D", "h0")]
    if which == "fwd":
        return lib.kda_ssm_fwd(*head, a["ht"], a["cu"], a["out"], d, None)
    if which == "decode":
        return lib.kda_ssm_decode(*head, a["ht"], a["out"], d, None)
    return lib.kda_ssm_bwd(*head, a["cu"], a["dy"], a["dht"], *[a[k] for k in ("dx", "ddt", "dB", "dC", "dA", "dbias", "dD", "dh0")], d, None)


def test_ssm_checks(lib):
    for which in ("fwd", "decode", "bwd"):
        need = {"fwd": ("out",), "decode": ("out", "ht"), "bwd": ("dy", "dx", "ddt", "dB", "dC", "dA")}[which]
        for k in ("x", "dt", "B", "C", "A") + need:
            assert ssm(lib, which, {k: None}) == NULL, (which, k)
        assert ssm(lib, which, B=0) == SHAPE and ssm(lib, which, T=-1) == SHAPE and ssm(lib, which, num_seqs=1) == SHAPE
        assert ssm(lib, which, G=3) == SHAPE and ssm(lib, which, H=0) == SHAPE and ssm(lib, which, T=1 << 33) == SHAPE
        assert ssm(lib, which, P=32) == UNSUPPORTED and ssm(lib, which, N=256) == UNSUPPORTED
        assert ssm(lib, which, x_stride_t=-8) == SHAPE and ssm(lib, which, b_stride_t=1 << 24) == SHAPE and ssm(lib, which, x_stride_t=257) == ALIGN
        assert ssm(lib, which, piece_chunks=-1) == PARAM
        assert ssm(lib, which, initial_state_dtype=0) == DTYPE and ssm(lib, which, final_state_dtype=3) == DTYPE
        for k in ("x", "B", "C", "h0") + need[:1]:
            assert ssm(lib, which, {k: p(21, 8)}) == ALIGN, (which, k)
    assert ssm(lib, "decode", T=2) == SHAPE
    assert ssm(lib, "fwd", {"cu": p(22)}) == SHAPE
    assert ssm(lib, "fwd", {"out": p(0)}) == OVERLAP and ssm(lib, "fwd", {"ht": p(7)}, final_state_dtype=1) == OVERLAP
    assert ssm(lib, "decode", {"out": p(8)}) == OVERLAP
    assert ssm(lib, "bwd", {"dx": p(10)}) == OVERLAP and ssm(lib, "bwd", {"dB": p(15)}) == OVERLAP
    assert ssm(lib, "bwd", {"dh0": p(30, 256)}) == OVERLAP
    assert ssm(lib, "bwd", workspace_bytes=256) == WORKSPACE
    assert ssm(lib, "fwd", piece_chunks=1, workspace=p(30, 16), T=200) == ALIGN
    assert ssm(lib, "fwd", piece_chunks=1, workspace_bytes=256, T=200) == WORKSPACE


def test_ssm_pieces_and_workspaces(lib):
    # a single prompt is cut into pieces, heads that fill the GPU by themselves are not
    assert kda.ssm_piece_chunks(1, 8192, 4, 64, 1, 64) < 128
    assert kda.ssm_piece_chunks(32, 2048, 64, 64, 1, 128) == 32
    assert kda.ssm_piece_chunks(1, 64, 4, 64, 1, 64) == 1
    assert kda.ssm_piece_chunks(1, 640, 4, 64, 1, 64, piece_chunks=3) == 3
    assert kda.ssm_piece_chunks(1, 640, 4, 64, 1, 64, piece_chunks=1 << 40) == 10
    with pytest.raises(ValueError):
        kda.ssm_piece_chunks(1, 640, 4, 96, 1, 64)
    assert kda.ssm_workspace_size(2, 640, 4, 64, 1, 64, piece_chunks=10) == 0
    assert kda.ssm_workspace_size(2, 640, 4, 64, 1, 64, piece_chunks=5) >= 2 * 2 * 4 * 64 * 64 * 4
    assert kda.ssm_workspace_size(1, 640, 4, 64, 1, 64, num_seqs=9) > 0
    # two fp32 states per chunk and head
    a, b = (kda.ssm_bwd_workspace_size(2, 64 * n, 4, 64, 1, 128, piece_chunks=n) for n in (600, 1200))
    assert b - a >= 2 * 2 * 600 * 4 * 64 * 128 * 4
    for bad in ((0, 64, 4, 64, 1, 64), (1, -1, 4, 64, 1, 64), (1, 64, 4, 64, 3, 64)):
        assert kda.ssm_bwd_workspace_size(*bad) == 0


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.zeros(64)
    for bad in (lambda: kda.rmsnorm_fwd(x, w, 1e-5), lambda: kda.rmsnorm_quant(x, w, 1e-5), lambda: kda.rmsnorm_bwd(x, w, 1e-5, x),
                lambda: kda.conv_fwd(x, w[:, None].expand(64, 4).contiguous()),
                lambda: kda.ssm_fwd(x[..., None], x, x[..., None], x[..., None], w)):
        with pytest.raises(ValueError):
            bad()


def test_the_library_is_published_with_its_types(monkeypatch):
    """Another thread may look while the first call declares the functions: it must not find a library whose
    functions still take anything."""
    class Function:
        restype = argtypes = None

    class Library:
        def __init__(self):
            self.functions, self.seen = {}, []

        def __getattr__(self, name):
            self.seen.append(L._lib)
            return self.functions.setdefault(name, Function())

    fake = Library()
    monkeypatch.setattr(L, "_lib", None)
    L._declare(fake)
    assert fake.seen and all(s is None for s in fake.seen)
    assert L._lib is fake and all(f.argtypes is not None for f in fake.functions.values())


def test_short_sequences_need_no_piece_states(lib):
    """Only the pieces of sequences with several have a state in the workspace: 4096 sequences of 8 tokens need
    the tables and the states of a few pieces, forwards, and two states per chunk (and head) for the gradient."""
    shape = (1, 32768, 64, 64, 1, 128)
    state = 64 * 64 * 128 * 4
    pieces = 2 * 32768 // (64 * kda.ssm_piece_chunks(*shape, num_seqs=4096))   # at most, of sequences with several
    assert kda.ssm_workspace_size(*shape, num_seqs=4096) <= pieces * state + (1 << 20)
    chunks = 32768 // 64 + 4096
    # the shares of dB and dC and the parameters' sums are small beside the states
    assert kda.ssm_bwd_workspace_size(*shape, num_seqs=4096) <= (pieces + 2 * chunks) * state * 9 // 8
    # sequences of one chunk more than a piece have two pieces each
    assert kda.ssm_workspace_size(1, 65 * 10, 4, 64, 1, 64, num_seqs=10, piece_chunks=1) >= 20 * 4 * 64 * 64 * 4


def test_many_sequences_take_several_launches(lib):
    """More pieces times heads than one launch holds workgroups is no reason to refuse a call."""
    n = 131073
    assert kda.ssm_workspace_size(1, 8 * n, 64, 64, 1, 128, num_seqs=n) > 0
    assert kda.ssm_bwd_workspace_size(1, 8 * n, 64, 64, 1, 128, num_seqs=n) > 2 * n * 64 * 64 * 128 * 4
    assert kda.ssm_piece_chunks(n, 8, 64, 64, 1, 128) == 1
    assert ssm(lib, launch_piece=-1) == PARAM and ssm(lib, "decode", launch_piece=-1) == PARAM
    assert ssm(lib, "bwd", launch_piece=-1) == PARAM


def test_rmsnorm_refuses_subnormal_eps(lib):
    """A row of zeros leaves eps by itself, and the hardware's reciprocal root takes a subnormal one as zero."""
    for q in (False, True):
        assert norm(lib, q, eps=1e-40) == PARAM and norm(lib, q, eps=2.0 ** -127) == PARAM
    assert norm_bwd(lib, eps=1e-40) == PARAM
    assert norm(lib, False, {"x": None}, eps=2.0 ** -126) == NULL   # accepted: the next check answers
