"""Latent attention, its cache and its pages in 64 bits on the CPU, from their
formulas: the oracle of the latent tests, with the bounds that the kernels'
roundings allow.

Bounds.  A probability enters the second product rounded to bf16 (2^-8 of it at
most) and comes from a score of 192 (576) products added in fp32, an exponential
and a log-sum-exp: a relative error `d` of (width + 8) 2^-24 times the largest
scaled |q| |k| of a row, plus a few units for the exponential (2^-21).  Sums of n
terms in fp32 add n 2^-24 of the terms' magnitudes.  The output's own rounding is
2^-8 of the value.  Probabilities and products below fp32's smallest normal number,
2^-126, are zeros to the kernels: sums of up to 2^20 of them, times values up to
2^6, leave out less than 2^-100."""
from __future__ import annotations

import torch

from tests.layer_ref import F64, U, bounds, d

HALF = 2.0 ** -8
UNDER = 2.0 ** -100
NEG = float("-inf")


def visible(lq, lk, causal):
    i, j = torch.arange(lq)[:, None], torch.arange(lk)[None]
    return (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)


def softmax(x, see):
    """(probabilities, log-sum-exp) of scores x where see; rows without any: zeros and -inf."""
    x = torch.where(see, x, torch.full_like(x, NEG))
    some = see.any(-1)
    top = torch.where(some, x.amax(-1) if x.shape[-1] else torch.zeros(x.shape[:-1], dtype=F64), torch.zeros(x.shape[:-1], dtype=F64))
    e = torch.where(see, torch.exp(x - top[..., None]), torch.zeros_like(x))
    z = e.sum(-1)
    return e / z.clamp_min(1e-300)[..., None], torch.where(some, top + torch.log(z.clamp_min(1e-300)), torch.full_like(z, NEG))


def score_error(q, k, scale, see):
    """[rows]: the relative error of a row's probabilities by its scores."""
    width = q.shape[-1]
    mag = torch.where(see, (q.abs() @ k.abs().transpose(-1, -2)) * scale, torch.zeros((), dtype=F64))
    top = mag.amax(-1) if mag.shape[-1] else torch.zeros(mag.shape[:-1], dtype=F64)
    return (width + 8) * U * top + 2.0 ** -21


def keys_of(kv, pe):
    return torch.cat([kv[..., :128], pe[:, None].expand(-1, kv.shape[1], -1)], -1)


def attention(q, kv, pe, scale, causal, lens, lens_k):
    """Packed [tokens, ...] in 64 bits -> dict of out, lse and their tolerances tol_out, tol_lse."""
    H = q.shape[1]
    out, lse = torch.zeros(q.shape[0], H, 128, dtype=F64), torch.full((q.shape[0], H), NEG, dtype=F64)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    at, ak = bounds(lens), bounds(lens_k)
    for n, (lq, lk) in enumerate(zip(lens, lens_k)):
        if lq == 0 or lk == 0:
            continue
        r, c = slice(at[n], at[n + 1]), slice(ak[n], ak[n + 1])
        see = visible(lq, lk, causal)
        qs, ks, vs = q[r].transpose(0, 1), keys_of(kv[c], pe[c]).transpose(0, 1), kv[c][..., 128:].transpose(0, 1)
        p, z = softmax(qs @ ks.transpose(1, 2) * scale, see)
        err = score_error(qs, ks, scale, see)
        o = p @ vs
        out[r], lse[r] = o.transpose(0, 1), z.transpose(0, 1)
        size = p @ vs.abs()
        to[r] = (size * (HALF + 2 * err + 2 * lk * U)[..., None] + HALF * o.abs()).transpose(0, 1)
        tl[r] = (err + lk * U + 4 * U * z.abs().nan_to_num(0, 0, 0) + 4 * U).transpose(0, 1)
    return {"out": out, "lse": lse, "tol_out": to, "tol_lse": tl}


def attention_bwd(q, kv, pe, scale, causal, lens, lens_k, out, lse, dy):
    """The gradient by its formula from the forward's stored out and lse -> dict of dq, dkv, dk_pe and tolerances tol_*."""
    res = {"dq": torch.zeros_like(q), "dkv": torch.zeros_like(kv), "dk_pe": torch.zeros_like(pe)}
    tol = {k: torch.zeros_like(v) for k, v in res.items()}
    at, ak = bounds(lens), bounds(lens_k)
    for n, (lq, lk) in enumerate(zip(lens, lens_k)):
        if lq == 0 or lk == 0:
            continue
        r, c = slice(at[n], at[n + 1]), slice(ak[n], ak[n + 1])
        see = visible(lq, lk, causal)
        qs, ks, vs = q[r].transpose(0, 1), keys_of(kv[c], pe[c]).transpose(0, 1), kv[c][..., 128:].transpose(0, 1)
        g, o, z = dy[r].transpose(0, 1), out[r].transpose(0, 1), lse[r].transpose(0, 1)
        z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
        p = torch.where(see, torch.exp(qs @ ks.transpose(1, 2) * scale - z[..., None]), torch.zeros((), dtype=F64))
        dp, delta = g @ vs.transpose(1, 2), (g * o).sum(-1, keepdim=True)
        ds = p * (dp - delta) * scale
        err = (score_error(qs, ks, scale, see) + 2 * U * z.abs())[..., None]
        # of dS: its rounding, its probability's error, and the sums that make up dP and delta
        e = ds.abs() * (HALF + 2 * err) + p * scale * 136 * U * (g.abs() @ vs.abs().transpose(1, 2) + (g * o).abs().sum(-1, keepdim=True))
        ep = p * (HALF + 2 * err)
        size = (ds.abs() + e)
        res["dq"][r] = (ds @ ks).transpose(0, 1)
        tol["dq"][r] = ((e + size * 2 * lk * U) @ ks.abs()).transpose(0, 1)
        dk = ds.transpose(1, 2) @ qs
        tk = (e + size * 2 * lq * U).transpose(1, 2) @ qs.abs()
        res["dkv"][c] = torch.cat([dk[..., :128], p.transpose(1, 2) @ g], -1).transpose(0, 1)
        tol["dkv"][c] = torch.cat([tk[..., :128], (ep + 2 * lq * U * p).transpose(1, 2) @ g.abs()], -1).transpose(0, 1)
        res["dk_pe"][c] = dk[..., 128:].sum(0)
        tol["dk_pe"][c] = tk[..., 128:].sum(0) + qs.shape[0] * U * dk[..., 128:].abs().sum(0)
    return res | {"tol_" + k: t + HALF * res[k].abs() for k, t in tol.items()}


def decode(ql, qp, cache, lengths, table, scale):
    """ql [N, T, H, 512], qp [N, T, H, 64], cache [pages, size, 576], all in 64 bits -> out, lse and tolerances."""
    N, T, H = ql.shape[:3]
    size = cache.shape[1]
    out, lse = torch.zeros(N, T, H, 512, dtype=F64), torch.full((N, T, H), NEG, dtype=F64)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    for n in range(N):
        ln = min(max(int(lengths[n]), 0), table.shape[1] * size)
        if ln == 0:
            continue
        rows = cache[table[n, :(ln + size - 1) // size].long()].reshape(-1, 576)[:ln]
        for t in range(T):
            k = rows[:max(0, ln - T + 1 + t)]
            if k.shape[0] == 0:
                continue
            q = torch.cat([ql[n, t], qp[n, t]], -1)
            see = torch.ones(H, k.shape[0], dtype=torch.bool)
            p, z = softmax(q @ k.t() * scale, see)
            err = score_error(q, k, scale, see)
            out[n, t], lse[n, t] = p @ k[:, :512], z
            to[n, t] = (p @ k[:, :512].abs()) * (HALF + 2 * err + 2 * k.shape[0] * U)[:, None] + HALF * out[n, t].abs()
            tl[n, t] = err + k.shape[0] * U + 4 * U * z.abs() + 4 * U
    return {"out": out, "lse": lse, "tol_out": to, "tol_lse": tl}


def within(got, ref, tol, label):
    got = d(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    same = (got == ref) | ((got - ref).abs() <= tol + UNDER)
    assert same.all(), "%s: %d of %d entries off, worst %.3g of the tolerance" % (
        label, int((~same).sum()), same.numel(), float(((got - ref).abs() / (tol + 1e-300)).nan_to_num(float("inf"))[~same].max()))


def pages(lengths, new, table, free, count, size, tokens, ended=None):
    """One serving step, request by request.  Lists and nested lists of whole numbers; returns a dict with the new
    table and stack among the rest."""
    N, mp = len(lengths), len(table[0]) if table else 0
    table, free = [list(r) for r in table], list(free)
    new = [max(0, k) for k in new]
    length = [min(max(0, k), mp * size) for k in lengths]
    ceil = lambda v: -(-v // size)  # noqa: E731
    count = min(max(0, count), len(free))
    for n in range(N):
        if ended is not None and ended[n]:
            for i in range(ceil(length[n])):
                if count < len(free):
                    free[count] = table[n][i]
                    count += 1
            length[n] = 0
    cu, out, granted, slots = [0], [], [], [-1] * tokens
    upto = used = 0
    for n in range(N):
        first, k = cu[-1], new[n]
        cu.append(first + k)
        fits = length[n] + k <= mp * size and first + k <= tokens
        need = ceil(length[n] + k) - ceil(length[n]) if fits else 0
        upto += need
        ok = fits and (need == 0 or upto <= count)
        if ok:
            held = ceil(length[n])
            for i in range(need):
                table[n][held + i] = free[count - 1 - (upto - need) - i]
            for j in range(k):
                p = length[n] + j
                slots[first + j] = table[n][p // size] * size + p % size
            used += need
        granted.append(k if ok else 0)
        out.append(length[n] + granted[-1])
    return {"slots": slots, "cu_seqlens": [min(c, tokens) for c in cu], "lengths": out, "granted": granted,
            "free_count": [count - used], "table": table, "free": free}
