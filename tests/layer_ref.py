"""The layer operators in 64 bits on the CPU, from their formulas: the oracle of
the layer tests.  Gradients come from autograd over these forms; the tests pin
them by central differences."""
from __future__ import annotations

import torch

F64 = torch.float64
# half a step of a type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def d(t):
    return None if t is None else t.detach().cpu().to(F64)


def rmsnorm(x, weight, eps, residual=None):
    """(y, h)"""
    h = x if residual is None else x + residual
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight, h


def bounds(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def conv(x, weight, bias, activation, initial, lens):
    """x [tokens, D], initial [N, W - 1, D] or None -> (y [tokens, D], final [N, W - 1, D])"""
    D, W = weight.shape
    at = bounds(lens)
    ys, fin = [], []
    for n, k in enumerate(lens):
        e = torch.cat([torch.zeros(W - 1, D, dtype=F64) if initial is None else initial[n], x[at[n]:at[n + 1]]])
        pre = torch.zeros(k, D, dtype=F64) if bias is None else bias.expand(k, D)
        for j in range(W):
            pre = pre + e[j:j + k] * weight[:, j]
        ys.append(pre * torch.sigmoid(pre) if activation else pre)
        fin.append(e[k:])
    return torch.cat(ys), torch.stack(fin)


def scan(x, dt, B, C, A_log, dt_bias, D, initial, lens):
    """x [tokens, H, P], dt [tokens, H], B, C [tokens, G, S], initial [N, H, P, S] or None -> (y, final)"""
    M, H, P = x.shape
    G, S = B.shape[1:]
    raw = dt if dt_bias is None else dt + dt_bias
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    decay = torch.exp(-torch.exp(A_log) * step)
    B, C = (t.repeat_interleave(H // G, 1) for t in (B, C))
    at = bounds(lens)
    ys, fin = [], []
    for n, k in enumerate(lens):
        st = torch.zeros(H, P, S, dtype=F64) if initial is None else initial[n]
        for t in range(at[n], at[n] + k):
            st = decay[t][:, None, None] * st + (step[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            y = (st * C[t][:, None, :]).sum(-1)
            ys.append(y if D is None else y + D[:, None] * x[t])
        fin.append(st)
    return (torch.stack(ys) if ys else torch.zeros(0, H, P, dtype=F64)), torch.stack(fin)


def check(got, ref, dtype, slack, label):
    """|got - ref| <= half a step of `dtype` relative to ref, plus `slack` (a tensor or a number)."""
    got = d(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    tol = HALF[dtype] * ref.abs() + slack
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d entries off, worst %.3g of the tolerance" % (
        label, int(bad.sum()), bad.numel(), float(((got - ref).abs() / (tol + 1e-300)).nan_to_num(float("inf")).max()))


def check_norm(got, ref, rel, label):
    """2-norm of the difference over that of ref."""
    got = d(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    n = float(ref.norm())
    off = float((got - ref).norm())
    assert off <= rel * n + 1e-30, "%s: %.3g relative, %.3g allowed" % (label, off / max(n, 1e-300), rel)


def grads(loss, leaves):
    if not loss.requires_grad:  # no token and no state reaches it
        return [None if t is None else torch.zeros_like(t) for t in leaves]
    got = torch.autograd.grad(loss, [t for t in leaves if t is not None], allow_unused=True)
    it = iter(got)
    out = []
    for t in leaves:
        g = None if t is None else next(it)
        out.append(torch.zeros_like(t) if t is not None and g is None else g)
    return out


def difference(fn, leaf, direction, h=1e-5):
    """Central difference of the scalar fn along `direction` at `leaf`."""
    return (fn(leaf + h * direction) - fn(leaf - h * direction)) / (2 * h)
