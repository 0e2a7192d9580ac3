"""The recurrent layer's operators around the state recurrence, as they are measured: RMS normalisation with the
residual's addition (bf16 output, or 8-bit output with scales), the short causal convolution, and the selective
state-space scan, each for prompts, for single tokens where generation has them, and backwards.

``run`` computes a pass in plain torch operations, or with ``own`` set through ``gated_delta_rule_110_amd``."""
import math
import random

import torch

own = False

L = 64            # tokens per chunk of the plain scan
E4M3_MAX = 448.0
EPS = 1e-5
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one generation step of 64 sequences: the norm ahead of an 8-bit projection, one scale per token
        {"name": "norm_q8_step", "op": "norm", "rows": 64, "D": 4096, "residual": "bf16", "quant": True, "group": 0},
        # a prompt's norm on an fp32 residual stream, a ragged number of rows
        {"name": "norm_prompt", "op": "norm", "rows": 8191, "D": 4096, "residual": "fp32", "quant": False, "group": 0},
        # the same norm in training: gradients of the sum and of the weight
        {"name": "norm_train", "op": "norm_bwd", "rows": 8192, "D": 4096, "residual": "bf16"},
        # one generation step of 64 sequences: the q, k and v streams of 32 heads of 128
        {"name": "conv_step", "op": "conv_step", "N": 64, "D": 12288, "W": 4, "silu": True, "bias": False, "state": "bf16"},
        # four prompts of 2048 tokens, the same streams
        {"name": "conv_prompt", "op": "conv", "T": 2048, "n": 4, "packed": False, "D": 12288, "W": 4, "silu": True,
         "bias": False, "state": "bf16", "slice": False},
        # a packed batch that continues cached sequences; x is a slice of a wider projection
        {"name": "conv_packed", "op": "conv", "T": 32768, "n": 17, "packed": True, "D": 4352, "W": 4, "silu": True,
         "bias": True, "state": "fp32", "slice": True},
        # the convolution in training
        {"name": "conv_train", "op": "conv_bwd", "T": 8192, "n": 1, "packed": False, "D": 4352, "W": 4, "silu": True,
         "bias": True, "state": "none", "slice": False},
        # one generation step of 64 sequences, fp32 states updated in place
        {"name": "scan_step", "op": "scan_step", "N": 64, "H": 64, "P": 64, "S": 128, "G": 1, "state": "fp32"},
        # one prompt
        {"name": "scan_prompt", "op": "scan", "T": 8192, "n": 1, "packed": False, "H": 64, "P": 64, "S": 128, "G": 1,
         "state": "none"},
        # a packed batch that continues cached sequences, wide heads in groups
        {"name": "scan_packed", "op": "scan", "T": 32768, "n": 17, "packed": True, "H": 32, "P": 128, "S": 128, "G": 8,
         "state": "fp32"},
        # one long document with few heads: the state chain alone would leave the GPU idle
        {"name": "scan_long", "op": "scan", "T": 131072, "n": 1, "packed": False, "H": 4, "P": 64, "S": 64, "G": 1,
         "state": "fp32"},
        # the scan in training
        {"name": "scan_train", "op": "scan_bwd", "T": 8192, "n": 1, "packed": False, "H": 64, "P": 64, "S": 128, "G": 1,
         "state": "none"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "conv_step", "conv", "conv", "conv_bwd", "scan_step", "scan", "scan",
                     "scan", "scan_bwd", "scan_bwd"])
    if op in ("norm", "norm_bwd"):
        D = rng.choice([64, 128, 1000, 2048, 2560, 4096, 5120, 8192, _log(rng, 33, 16384)])
        c = {"op": op, "rows": _log(rng, 1, max(1, (1 << 25) // D)), "D": D,
             "residual": rng.choice(["none", "bf16", "fp32"])}
        if op == "norm":
            c["quant"] = rng.random() < 0.5
            c["group"] = rng.choice([0, 128]) if c["quant"] else 0
        return c
    state = rng.choice(["none", "bf16", "fp32"])
    if op == "conv_step":
        return {"op": op, "N": _log(rng, 1, 512), "D": rng.choice([768, 4352, 12288, _log(rng, 5, 16384)]),
                "W": rng.choice([2, 3, 4]), "silu": rng.random() < 0.8, "bias": rng.random() < 0.5,
                "state": rng.choice(["bf16", "fp32"])}
    packed = rng.random() < 0.5
    if op in ("conv", "conv_bwd"):
        D = rng.choice([768, 2304, 4352, 12288, _log(rng, 5, 16384)])
        T = _log(rng, 1, max(2, min(65536, (1 << (27 if op == "conv" else 26)) // D)))
        n = _log(rng, 1, 24) if packed else rng.choice([1, 1, 2, 4])
        return {"op": op, "T": T if packed else max(1, T // n), "n": n, "packed": packed, "D": D,
                "W": rng.choice([2, 3, 4, 4]), "silu": rng.random() < 0.8, "bias": rng.random() < 0.5, "state": state,
                "slice": rng.random() < 0.5}
    G = rng.choice([1, 1, 2, 4])
    H = G * rng.choice([1, 2, 3, 5, 8, 16])
    P, S = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "scan_step":
        return {"op": op, "N": _log(rng, 1, 256), "H": H, "P": P, "S": S, "G": G, "state": rng.choice(["bf16", "fp32"])}
    T = _log(rng, 1, min(65536, (1 << (20 if op == "scan" else 18)) * 64 // (H * P)))
    n = _log(rng, 1, 24) if packed else rng.choice([1, 1, 2, 3])
    return {"op": op, "T": T if packed else max(1, T // n), "n": n, "packed": packed, "H": H, "P": P, "S": S, "G": G,
            "state": state}


def _lens(case):
    """Sequence lengths: equal rows, or for a packed batch uneven ones that sum to T, with an empty sequence and one
    of a single token where there are four or more."""
    n, T = case["n"], case["T"]
    if not case["packed"]:
        return [T] * n
    r = random.Random(1000 * n + T)
    w = [math.exp(r.uniform(0.0, math.log(200.0))) for _ in range(n)]
    lens = [int(T * v / sum(w)) for v in w]
    if n >= 4:
        lens[1], lens[2] = min(1, T), 0
    lens[-1] = 0
    lens[-1] = max(0, T - sum(lens))
    if sum(lens) != T:
        lens = [0] * (n - 1) + [T]
    return lens


# ---- inputs ------------------------------------------------------------------

class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, dtype=BF16, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=self.g, device="cuda", dtype=F32) * std + mean).to(dtype)

    def uniform(self, shape, lo, hi):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=F32) * (hi - lo) + lo


def _dtype(name):
    return {"bf16": BF16, "fp32": F32}[name]


def _plan(lens, W=None):
    """Where a batch's tokens stand, from its lengths: what a serving loop's scheduler holds."""
    n, M = len(lens), sum(lens)
    ln = torch.tensor(lens, dtype=torch.int64)
    first = torch.cumsum(ln, 0) - ln
    seq = torch.repeat_interleave(torch.arange(n), ln)
    pos = torch.arange(M) - first[seq]
    p = {"n": n, "M": M}
    if W is not None:  # rows of [states ; tokens] that a token's taps and a sequence's last W - 1 inputs come from
        k = torch.arange(W - 1)
        row = lambda s, q: torch.where(q >= 0, n * (W - 1) + first[s] + q, s * (W - 1) + (W - 1) + q)  # noqa: E731
        p["taps"] = torch.stack([row(seq, pos - (W - 1) + j) for j in range(W)]).cuda()
        p["last"] = row(torch.arange(n)[:, None].expand(n, W - 1), ln[:, None] - (W - 1) + k).reshape(-1).cuda()
        return p
    slots = (ln + L - 1) // L
    p["slots"] = int(slots.sum())
    begin = torch.cumsum(slots, 0) - slots
    p["at"] = (begin[seq] * L + pos).cuda()
    p["seq"] = torch.repeat_interleave(torch.arange(n), slots).cuda()
    p["begin"], p["end"] = begin.cuda(), (begin + slots).cuda()
    return p


def prepare(case, seed):
    r, op = _Draws(seed), case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        s["weight"] = r.normal((D,), F32, 0.1, 1.0)
        if op == "norm":
            s["x"] = r.normal((R, D))
            s["residual"] = None if case["residual"] == "none" else r.normal((R, D), _dtype(case["residual"]), 2.0)
        else:  # h: the stream that the forward wrote (the input itself where there was no residual)
            has = case["residual"] != "none"
            s["h"] = r.normal((R, D), _dtype(case["residual"]) if has else BF16, 2.0)
            s["d_out"] = r.normal((R, D))
            s["d_residual_out"] = r.normal((R, D), s["h"].dtype) if has else None
        return s
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        s["weight"] = r.normal((D, W), F32, 0.4)
        s["bias"] = r.normal((D,), F32, 0.2) if case["bias"] else None
        s["activation"] = "silu" if case["silu"] else None
        if op == "conv_step":
            N = case["N"]
            s["x"] = r.normal((N, 1, D))
            s["initial"] = r.normal((N, W - 1, D), _dtype(case["state"]))
            s["out"], s["final"] = torch.empty_like(s["x"]), torch.empty_like(s["initial"])
            return s
        lens = _lens(case)
        B, T = (1, case["T"]) if case["packed"] else (case["n"], case["T"])
        s["plan"] = _plan(lens, W)
        s["cu"] = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64).cuda() if case["packed"] else None
        wide = r.normal((B, T, D + (256 if case["slice"] else 0)))
        s["x"] = wide[..., 256:] if case["slice"] else wide
        s["initial"] = None if case["state"] == "none" else r.normal((len(lens), W - 1, D), _dtype(case["state"]))
        if op == "conv_bwd":
            s["d_out"] = r.normal((B, T, D))
            s["d_final"] = None if s["initial"] is None else r.normal((len(lens), W - 1, D), _dtype(case["state"]))
        return s
    H, P, S, G = case["H"], case["P"], case["S"], case["G"]
    s["A_log"] = torch.log(r.uniform((H,), 1.0, 16.0))
    step = torch.exp(r.uniform((H,), math.log(1e-3), math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # the inverse softplus of the step size
    s["D"] = r.normal((H,), F32, 0.1, 1.0)
    if op == "scan_step":
        B, T, lens = case["N"], 1, [1] * case["N"]
    else:
        lens = _lens(case)
        B, T = (1, case["T"]) if case["packed"] else (case["n"], case["T"])
        s["plan"] = _plan(lens)
        s["cu"] = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64).cuda() if case["packed"] else None
    # x, B and C leave the convolution as one tensor, the step sizes the projection
    xbc = r.normal((B, T, H * P + 2 * G * S))
    s["x"] = xbc[..., : H * P].unflatten(-1, (H, P))
    s["B"] = xbc[..., H * P: H * P + G * S].unflatten(-1, (G, S))
    s["C"] = xbc[..., H * P + G * S:].unflatten(-1, (G, S))
    s["dt"] = r.normal((B, T, H))
    s["initial"] = None if case["state"] == "none" else r.normal((len(lens), H, P, S), _dtype(case["state"]), 0.5)
    if op == "scan_step":
        s["out"], s["final"] = torch.empty((B, 1, H, P), dtype=BF16, device="cuda"), torch.empty_like(s["initial"])
    if op == "scan_bwd":
        s["d_out"] = r.normal((B, T, H, P))
        s["d_final"] = None if s["initial"] is None else r.normal((len(lens), H, P, S), _dtype(case["state"]), 0.5)
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_110_amd as kda

        if op == "norm":
            if s["case"]["quant"]:
                q, scale, res = kda.rmsnorm_quant(s["x"], s["weight"], EPS, residual=s["residual"], group=s["case"]["group"])
                return {"q": q, "scale": scale, "residual": res}
            y, res = kda.rmsnorm_fwd(s["x"], s["weight"], EPS, residual=s["residual"])
            return {"y": y, "residual": res}
        if op == "norm_bwd":
            return kda.rmsnorm_bwd(s["h"], s["weight"], EPS, s["d_out"], d_residual_out=s["d_residual_out"])
        if op == "conv_step":
            y, fin = kda.conv_decode(s["x"], s["weight"], s["bias"], s["activation"], initial_state=s["initial"],
                                     final_state=s["final"], out=s["out"])
            return {"y": y, "final": fin}
        if op == "conv":
            fin = None if s["initial"] is None else torch.empty_like(s["initial"])
            y, fin = kda.conv_fwd(s["x"], s["weight"], s["bias"], s["activation"], initial_state=s["initial"],
                                  final_state=fin, cu_seqlens=s["cu"])
            return {"y": y, "final": fin}
        if op == "conv_bwd":
            return kda.conv_bwd(s["x"], s["weight"], s["bias"], s["activation"], s["d_out"], d_final_state=s["d_final"],
                                initial_state=s["initial"], cu_seqlens=s["cu"])
        args = (s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], s["D"])
        if op == "scan_step":
            y, fin = kda.ssm_decode(*args, initial_state=s["initial"], final_state=s["final"], out=s["out"])
            return {"y": y, "final": fin}
        if op == "scan":
            fin = torch.empty(s["plan"]["n"], *s["x"].shape[2:], s["B"].shape[-1], device="cuda",
                              dtype=F32 if s["initial"] is None else s["initial"].dtype)
            y, fin = kda.ssm_fwd(*args, initial_state=s["initial"], final_state=fin, cu_seqlens=s["cu"])
            return {"y": y, "final": fin}
        return kda.ssm_bwd(*args, s["d_out"], d_final_state=s["d_final"], initial_state=s["initial"], cu_seqlens=s["cu"])
    if op == "norm":
        return _norm(s)
    if op == "norm_bwd":
        return _norm_bwd(s)
    if op == "conv_step":
        return _conv_step(s)
    if op == "conv":
        y, fin = _conv(s["x"].float(), s["weight"], s["bias"], s["activation"], s["initial"], s["plan"])
        return {"y": y.to(BF16), "final": None if s["initial"] is None else fin.to(s["initial"].dtype)}
    if op == "conv_bwd":
        return _conv_bwd(s)
    if op == "scan_step":
        return _scan_step(s)
    if op == "scan":
        y, fin = _scan(s["x"].float(), s["dt"].float(), s["B"].float(), s["C"].float(), s["A_log"], s["dt_bias"], s["D"],
                       None if s["initial"] is None else s["initial"].float(), s["plan"])
        return {"y": y.to(BF16), "final": fin.to(F32 if s["initial"] is None else s["initial"].dtype)}
    return _scan_bwd(s)


# ---- the plain forms -----------------------------------------------------------

def _norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    res = None if s["residual"] is None else h.to(s["residual"].dtype)
    if not c["quant"]:
        return {"y": y.to(BF16), "residual": res}
    R, D = y.shape
    g = c["group"] or D
    yg = torch.nn.functional.pad(y, (0, -D % g)).unflatten(-1, (-1, g))
    scale = (yg.abs().amax(-1) / E4M3_MAX).clamp_min(torch.finfo(F32).tiny)
    q = (yg / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :D].to(torch.float8_e4m3fn)
    return {"q": q, "scale": scale, "residual": res}


def _norm_bwd(s):
    h, dy, w = s["h"].float(), s["d_out"].float(), s["weight"]
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * rstd
    wdy = dy * w
    dh = rstd * (wdy - n * (wdy * n).mean(-1, keepdim=True))
    if s["d_residual_out"] is not None:
        dh = dh + s["d_residual_out"].float()
    dx = dh.to(BF16)
    return {"dx": dx, "dresidual": None if s["d_residual_out"] is None else dh if s["h"].dtype == F32 else dx,
            "dweight": (dy * n).sum(0)}


def _silu(x):
    return x / (1 + torch.exp(-x))


def _conv_step(s):
    ext = torch.cat([s["initial"].float(), s["x"].float()], 1)
    pre = (ext * s["weight"].t()).sum(1, keepdim=True)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    return {"y": (_silu(pre) if s["activation"] else pre).to(BF16), "final": ext[:, 1:].to(s["initial"].dtype)}


def _conv(x, weight, bias, activation, initial, plan):
    B, T, D = x.shape
    W = weight.shape[1]
    init = torch.zeros(plan["n"], W - 1, D, device="cuda") if initial is None else initial.float()
    ext = torch.cat([init.reshape(-1, D), x.reshape(-1, D)])
    pre = sum(ext[plan["taps"][k]] * weight[:, k] for k in range(W))
    if bias is not None:
        pre = pre + bias
    return (_silu(pre) if activation else pre).view(B, T, D), ext[plan["last"]].view(plan["n"], W - 1, D)


def _conv_bwd(s):
    leaf = {"dx": s["x"].float(), "dweight": s["weight"], "dbias": s["bias"],
            "d_initial_state": None if s["initial"] is None else s["initial"].float()}
    leaf = {k: None if v is None else v.detach().clone().requires_grad_() for k, v in leaf.items()}
    y, fin = _conv(leaf["dx"], leaf["dweight"], leaf["dbias"], s["activation"], leaf["d_initial_state"], s["plan"])
    outs, grads = [y], [s["d_out"].float()]
    if s["d_final"] is not None:
        outs, grads = outs + [fin], grads + [s["d_final"].float()]
    names = [k for k, v in leaf.items() if v is not None]
    res = dict.fromkeys(leaf) | dict(zip(names, torch.autograd.grad(outs, [leaf[k] for k in names], grads)))
    return res | {"dx": res["dx"].to(BF16)}


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_step(s):
    H, G = s["x"].shape[2], s["B"].shape[2]
    x = s["x"][:, 0].float()
    Bm = s["B"][:, 0].float().repeat_interleave(H // G, 1)
    Cm = s["C"][:, 0].float().repeat_interleave(H // G, 1)
    dt = _softplus(s["dt"][:, 0].float() + s["dt_bias"])
    decay = torch.exp(-torch.exp(s["A_log"]) * dt)
    st = decay[..., None, None] * s["initial"].float() + (dt[..., None] * x)[..., None] * Bm[..., None, :]
    y = (st * Cm[..., None, :]).sum(-1) + s["D"][:, None] * x
    return {"y": y[:, None].to(BF16), "final": st.to(s["initial"].dtype)}


def _scan(x, dt, Bm, Cm, A_log, dt_bias, D, h0, plan):
    """The chunked scan: chunks of L tokens that stay within a sequence, padded with tokens of no effect."""
    B_, T, H, P = x.shape
    G, S = Bm.shape[2:]
    n, M, nc = plan["n"], plan["M"], plan["slots"]
    step = _softplus(dt.reshape(M, H) + dt_bias)

    def chunks(t):  # [tokens, heads, ...] -> [chunk, head, L, ...]
        t = t.reshape(M, *t.shape[2:]) if t.dim() > 2 and t.shape[:2] == (B_, T) else t
        full = torch.zeros(nc * L, *t.shape[1:], device="cuda", dtype=t.dtype).index_copy(0, plan["at"], t)
        return full.view(nc, L, *t.shape[1:]).transpose(1, 2)

    xs, bs, cs, ds = chunks(x), chunks(Bm), chunks(Cm), chunks(step)
    # sums of log-decays in 64 bits: differences of far ones are exponentiated
    cum = torch.cumsum(ds.double() * -torch.exp(A_log.double())[:, None], -1)
    upper = torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1)
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(upper, -math.inf)).float()
    cb = (cs @ bs.transpose(-1, -2)).repeat_interleave(H // G, 1)
    y = (cb * decay * ds[..., None, :]) @ xs
    # every chunk's own state, and the decays from chunk to chunk of a sequence
    tail = torch.exp(cum[..., -1:] - cum).float() * ds
    local = (xs * tail[..., None]).transpose(-1, -2) @ bs.repeat_interleave(H // G, 1)
    total = torch.cat([torch.zeros(1, H, device="cuda", dtype=F64), torch.cumsum(cum[..., -1], 0)])  # [nc + 1, H]
    i = torch.arange(nc, device="cuda")
    same = (plan["seq"][:, None] == plan["seq"]) & (i[None] < i[:, None])
    link = torch.exp((total[:-1].t()[:, :, None] - total[1:].t()[:, None, :]).masked_fill(~same, -math.inf)).float()
    mine = (i[None] >= plan["begin"][:, None]) & (i[None] < plan["end"][:, None])
    close = torch.exp((total[plan["end"]].t()[:, :, None] - total[1:].t()[:, None, :]).masked_fill(~mine, -math.inf)).float()
    flat = local.transpose(0, 1).reshape(H, nc, P * S)
    enter, fin = link @ flat, close @ flat
    if h0 is not None:
        start = total[plan["begin"]]
        enter = enter + (torch.exp(total[:-1] - start[plan["seq"]]).float()[..., None] * h0.reshape(n, H, -1)[plan["seq"]]).transpose(0, 1)
        fin = fin + (torch.exp(total[plan["end"]] - start).float()[..., None] * h0.reshape(n, H, -1)).transpose(0, 1)
    enter = enter.view(H, nc, P, S).transpose(0, 1)
    y = y + torch.exp(cum).float()[..., None] * (cs.repeat_interleave(H // G, 1) @ enter.transpose(-1, -2)) + D[:, None, None] * xs
    y = y.transpose(1, 2).reshape(nc * L, H, P)[plan["at"]]
    return y.view(B_, T, H, P), fin.transpose(0, 1).reshape(n, H, P, S)


_SCAN_GRADS = ("dx", "ddt", "dB", "dC", "dA_log", "ddt_bias", "dD", "d_initial_state")


def _scan_bwd(s):
    leaf = [s["x"].float(), s["dt"].float(), s["B"].float(), s["C"].float(), s["A_log"], s["dt_bias"], s["D"]]
    leaf += [] if s["initial"] is None else [s["initial"].float()]
    leaf = [t.detach().clone().requires_grad_() for t in leaf]
    y, fin = _scan(*leaf[:7], leaf[7] if len(leaf) > 7 else None, s["plan"])
    outs, grads = [y], [s["d_out"].float()]
    if s["d_final"] is not None:
        outs, grads = outs + [fin], grads + [s["d_final"].float()]
    got = list(torch.autograd.grad(outs, leaf, grads)) + ([None] if len(leaf) == 7 else [])
    return {k: v if i > 3 else v.to(BF16) for i, (k, v) in enumerate(zip(_SCAN_GRADS, got))}


# ---- the work of one pass --------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, D = case["rows"] * case["D"], case["D"]
        res = {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
        if op == "norm":
            scales = 4 * case["rows"] * -(-D // case["group"]) if case["group"] else 4 * case["rows"] * case["quant"]
            return {"bytes": n * (2 + 2 * res + (1 if case["quant"] else 2)) + 4 * D + scales, "flops": 5 * n}
        # h, d_out and the stream's gradient in; the gradient out, in both types where the stream is fp32
        return {"bytes": n * ((res or 2) + 2 + res + 2 + (4 if res == 4 else 0)) + 8 * D, "flops": 10 * n}
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        seqs = case["N"] if op == "conv_step" else case["n"]
        M = case["N"] if op == "conv_step" else case["T"] * (1 if case["packed"] else case["n"])
        st = {"none": 0, "bf16": 2, "fp32": 4}[case["state"]] * seqs * (W - 1) * D
        par = 4 * D * (W + case["bias"])
        if op == "conv_bwd":
            return {"bytes": 6 * M * D + 2 * par + 2 * st + 4 * seqs * (W - 1) * D * (case["state"] != "none"),
                    "flops": M * D * (6 * W + 8)}
        return {"bytes": 4 * M * D + par + 2 * st, "flops": M * D * (2 * W + 4)}
    H, P, S, G = case["H"], case["P"], case["S"], case["G"]
    seqs = case["N"] if op == "scan_step" else case["n"]
    M = case["N"] if op == "scan_step" else case["T"] * (1 if case["packed"] else case["n"])
    width = {"none": 0, "bf16": 2, "fp32": 4}[case["state"]]
    act, states = M * (2 * H * P + 4 * G * S + 2 * H), seqs * H * P * S
    if op == "scan_bwd":
        return {"bytes": 2 * act + 2 * M * H * P + states * (2 * width + (4 if width else 0)) + 24 * H,
                "flops": 14 * M * H * P * S}
    return {"bytes": act + 2 * M * H * P + states * (width + (width or 4)) + 12 * H, "flops": 5 * M * H * P * S}


# ---- the definition, in 64 bits -----------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("scan", "scan_bwd") and max(_lens(case)) > (140000 if op == "scan" else 40000):
        return None  # one step per token
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if op == "norm":
        h = d(s["x"]) if s["residual"] is None else d(s["x"]) + d(s["residual"])
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["D"] + EPS) * d(s["weight"])
        res = None if s["residual"] is None else h
        if not case["quant"]:
            return {"y": y, "residual": res}
        cols = torch.split(y, case["group"] or case["D"], dim=1)
        scale = torch.stack([t.abs().max(1).values for t in cols], 1) / E4M3_MAX
        q = torch.cat([t / scale[:, j: j + 1] for j, t in enumerate(cols)], 1)
        return {"q": q, "scale": scale, "residual": res}
    if op == "norm_bwd":
        h = d(s["h"]).requires_grad_()
        w = d(s["weight"]).requires_grad_()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["D"] + EPS) * w
        dh, dw = torch.autograd.grad(y, [h, w], d(s["d_out"]))
        if s["d_residual_out"] is not None:
            dh = dh + d(s["d_residual_out"])
        return {"dx": dh, "dresidual": None if s["d_residual_out"] is None else dh, "dweight": dw}
    if op.startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s, [1] * case["N"] if op == "scan_step" else _lens(case))


def _exact_conv(s):
    """Sequence by sequence, each with its state in front of its tokens."""
    c, W = s["case"], s["case"]["W"]
    lens = [1] * c["N"] if c["op"] == "conv_step" else _lens(c)
    D, back = c["D"], c["op"] == "conv_bwd"
    x = s["x"].double().reshape(-1, D)
    w = s["weight"].double()
    b = torch.zeros(D, device="cuda", dtype=F64) if s["bias"] is None else s["bias"].double()
    init = torch.zeros(len(lens), W - 1, D, device="cuda", dtype=F64) if s["initial"] is None else s["initial"].double()
    if back:
        x, w, b, init = (t.detach().clone().requires_grad_() for t in (x, w, b, init))
    ys, last, at = [], [], 0
    for i, n in enumerate(lens):
        e = torch.cat([init[i], x[at: at + n]])
        pre = b.expand(n, D)
        for k in range(W):
            pre = pre + e[k: k + n] * w[:, k]
        ys.append(pre * torch.sigmoid(pre) if s["activation"] else pre)
        last.append(e[n:])
        at += n
    y, fin = torch.cat(ys).view(s["x"].shape), torch.stack(last)
    if not back:
        return {"y": y, "final": None if s["initial"] is None else fin}
    loss = (y * s["d_out"].double()).sum()
    if s["d_final"] is not None:
        loss = loss + (fin * s["d_final"].double()).sum()
    g = torch.autograd.grad(loss, [x, w, b, init], allow_unused=True)
    return {"dx": g[0].view(s["x"].shape), "dweight": g[1], "dbias": None if s["bias"] is None else g[2],
            "d_initial_state": None if s["initial"] is None else g[3]}


def _exact_scan(s, lens):
    """The recurrence, token by token, all sequences side by side (those that have ended stand still)."""
    op = s["case"]["op"]
    H, P = s["x"].shape[2:]
    G, S = s["B"].shape[2:]
    n, top = len(lens), max(lens)
    at = torch.full((top, n), -1, dtype=torch.int64)
    off = 0
    for i, k in enumerate(lens):
        at[:k, i] = torch.arange(off, off + k)
        off += k
    live = (at >= 0).cuda()
    at = at.clamp(min=0).cuda()
    A = -torch.exp(s["A_log"].double())
    raw = s["dt"].double().reshape(-1, H) + s["dt_bias"].double()
    dt = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    x, Bm, Cm = (s[k].double().reshape(-1, *s[k].shape[2:]) for k in ("x", "B", "C"))
    Bm, Cm = (t.repeat_interleave(H // G, 1) for t in (Bm, Cm)) if x.shape[0] * H * S < 1 << 28 else (Bm, Cm)
    wide = (lambda t: t) if Bm.shape[1] == H else (lambda t: t.repeat_interleave(H // G, 1))
    y = torch.zeros_like(x)
    st = torch.zeros(n, H, P, S, device="cuda", dtype=F64) if s["initial"] is None else s["initial"].double()

    def forward(st, t):
        i, on = at[t], live[t][:, None]
        step = dt[i] * on
        return st * torch.exp(step * A)[..., None, None] + (step[..., None] * x[i])[..., None] * wide(Bm[i])[..., None, :]

    if op != "scan_bwd":
        for t in range(top):
            st = forward(st, t)
            y.index_add_(0, at[t], torch.matmul(st, wide(Cm[at[t]])[..., None])[..., 0] * live[t][:, None, None])
        return {"y": (y + s["D"].double()[:, None] * x).view(s["x"].shape), "final": st}
    # backwards, in blocks whose states are computed again
    block, starts = 64, []
    for t in range(top):
        if t % block == 0:
            starts.append(st)
        st = forward(st, t)
    dy = s["d_out"].double().reshape(-1, H, P)
    dx = s["D"].double()[:, None] * dy
    ddt, dB, dC, da = torch.zeros_like(dt), torch.zeros_like(Bm), torch.zeros_like(Cm), torch.zeros_like(dt)
    narrow = (lambda t: t) if Bm.shape[1] == H else (lambda t: t.view(n, G, H // G, S).sum(2))
    ds = torch.zeros_like(st) if s["d_final"] is None else s["d_final"].double()
    for b in range(len(starts) - 1, -1, -1):
        states = [starts[b]]
        for t in range(b * block, min(top, (b + 1) * block)):
            states.append(forward(states[-1], t))
        for t in range(min(top, (b + 1) * block) - 1, b * block - 1, -1):
            i, on = at[t], live[t][:, None]
            g, h, before = dy[i] * on[..., None], dt[i] * on, states[t - b * block]
            dC.index_add_(0, i, narrow(torch.matmul(g[..., None, :], states[t - b * block + 1])[..., 0, :]))
            ds = ds + g[..., None] * wide(Cm[i])[..., None, :]
            u = torch.matmul(ds, wide(Bm[i])[..., None])[..., 0]
            dx.index_add_(0, i, h[..., None] * u)
            ddt.index_add_(0, i, (u * x[i]).sum(-1) * on)
            dB.index_add_(0, i, narrow((h[..., None, None] * x[i][..., None] * ds).sum(2)))
            e = torch.exp(h * A)
            da.index_add_(0, i, (ds * before).sum((-1, -2)) * e * on)
            ds = ds * e[..., None, None]
    if Bm.shape[1] == H and G != H:
        dB, dC = (t.view(-1, G, H // G, S).sum(2) for t in (dB, dC))
    draw_ = (ddt + da * A) * torch.sigmoid(raw)
    return {"dx": dx.view(s["x"].shape), "ddt": draw_.view(s["dt"].shape), "dB": dB.view(s["B"].shape), "dC": dC.view(s["C"].shape),
            "dA_log": (da * dt).sum(0) * A, "ddt_bias": draw_.sum(0), "dD": (dy * x).sum((0, 2)),
            "d_initial_state": None if s["initial"] is None else ds}
