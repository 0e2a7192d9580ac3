"""The attention layers that stand between recurrent ones in a hybrid stack, as they are measured: latent attention, whose
keys and values come from one shared vector a token, in its expanded form (prompts and training) and in its absorbed form
(generation from a paged cache), the store of a token's vector into that cache, and the page bookkeeping of a serving step.

``run`` computes a pass in plain torch operations, or with ``own`` set through ``gated_delta_rule_110_amd``."""
import math
import random

import torch

own = False

NOPE, PE, VAL, LAT = 128, 64, 128, 512   # a head's own key values, those shared by all heads, its values, the latent
SCALE = (NOPE + PE) ** -0.5
EPS = 1e-6
BF16, F32, F64, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int64


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one generation step of 64 requests: a slot for each new token, a page for the few that begin one
        {"name": "pages_step", "op": "pages", "N": 64, "tokens": 64, "page": 64, "max_len": 8192, "ended": False, "short": False},
        # a serving step that mixes generation with prompts, requests that end, and too few pages for the last ones
        {"name": "pages_mixed", "op": "pages", "N": 1024, "tokens": 131072, "page": 16, "max_len": 8192, "ended": True, "short": True},
        # the new tokens of that generation step into the cache
        {"name": "store_step", "op": "store", "tokens": 64, "page": 64, "norm": True, "normed": False},
        # a packed batch of prompts into the cache; the normed latents are kept for the expansion
        {"name": "store_prompt", "op": "store", "tokens": 32768, "page": 64, "norm": True, "normed": True},
        # a few short prompts: launch and latency count
        {"name": "prompt_short", "op": "fwd", "T": 1000, "n": 7, "packed": True, "context": 0, "H": 32, "causal": True},
        # one prompt
        {"name": "prompt_long", "op": "fwd", "T": 8192, "n": 1, "packed": False, "context": 0, "H": 32, "causal": True},
        # the next pieces of prompts whose beginnings are expanded already
        {"name": "prompt_pieces", "op": "fwd", "T": 16383, "n": 17, "packed": True, "context": 2000, "H": 16, "causal": True},
        # the same layer in training: one long sequence
        {"name": "train_long", "op": "bwd", "T": 8192, "n": 1, "packed": False, "context": 0, "H": 32, "causal": True},
        # and a packed batch of documents
        {"name": "train_packed", "op": "bwd", "T": 8191, "n": 9, "packed": True, "context": 0, "H": 16, "causal": True},
        # one generation step of 64 requests
        {"name": "decode_step", "op": "decode", "N": 64, "T": 1, "H": 32, "len": 4096, "page": 64},
        # one request with a very long cache
        {"name": "decode_long", "op": "decode", "N": 1, "T": 1, "H": 128, "len": 131072, "page": 64},
        # drafted tokens of a few requests, small pages
        {"name": "decode_draft", "op": "decode", "N": 12, "T": 4, "H": 16, "len": 9000, "page": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "store", "fwd", "fwd", "fwd", "bwd", "bwd", "decode", "decode", "decode"])
    if op == "pages":
        N, page, top = _log(rng, 1, 2048), rng.choice([16, 32, 64, 128, 256]), rng.choice([1024, 4096, 8192])
        return {"op": op, "N": N, "tokens": min(131072, _log(rng, max(N, 2), N * 256)), "page": page, "max_len": top,
                "ended": rng.random() < 0.5, "short": rng.random() < 0.3}
    if op == "store":
        norm = rng.random() < 0.7
        return {"op": op, "tokens": _log(rng, 1, 32768), "page": rng.choice([16, 32, 64, 128, 256]), "norm": norm,
                "normed": norm and rng.random() < 0.5}
    if op == "decode":
        N, T, H = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 7]), rng.choice([1, 4, 8, 16, 20, 32, 40, 64, 128])
        return {"op": op, "N": N, "T": T, "H": H, "len": _log(rng, 16, min(65536, max(32, (1 << 24) // (N * max(32, T * H))))),
                "page": rng.choice([16, 32, 64, 128, 256])}
    H = rng.choice([1, 2, 3, 4, 8, 16, 32])
    top = int(math.sqrt((1 << 29) / H))
    T = _log(rng, 40, min(16384, top))
    packed = rng.random() < 0.6
    n = _log(rng, 1, 20) if packed else rng.choice([1, 1, 2, 3])
    T = max(n * 8, T) if packed else max(40, T // n)
    return {"op": op, "T": T, "n": n, "packed": packed, "context": rng.choice([0, 0, min(2000, T // 2)]), "H": H,
            "causal": rng.random() < 0.8}


def _uneven(n, total, seed):
    """n lengths up to 30 times one another that sum to total, with an empty one and one of a single token where there
    are four or more."""
    r = random.Random(seed)
    w = [math.exp(r.uniform(0.0, math.log(30.0))) for _ in range(n)]
    lens = [int(total * v / sum(w)) for v in w]
    if n >= 4:
        lens[1], lens[2] = min(1, total), 0
    lens[-1] = 0
    lens[-1] = max(0, total - sum(lens))
    return lens


def _lens(case):
    """(queries, keys) of every sequence of a prompt or training case."""
    n, T = case["n"], case["T"]
    if not case["packed"]:
        return [T] * n, [T + case["context"]] * n
    q = _uneven(n, T, 1000 * n + T)
    before = _uneven(n, case["context"] * n, 2000 * n + T) if case["context"] else [0] * n
    return q, [a + b for a, b in zip(q, before)]


def _cached(case):
    """Tokens in the cache of every sequence of a generation case, the new ones among them."""
    N, T, L = case["N"], case["T"], case["len"]
    if N == 1:
        return [max(L, T)]
    r = random.Random(3000 * N + L)
    lens = [max(T, int(L * r.uniform(0.3, 1.7))) for _ in range(N)]
    if N >= 4:  # a request that has just begun, and an unused row of the batch
        lens[1], lens[2] = T, 0
    return lens


def _new_tokens(case):
    """New tokens of every request of a serving step: one each, or where there are more, prompts among them."""
    N, total = case["N"], case["tokens"]
    new = [1] * N
    if total > N:
        r = random.Random(4000 * N + total)
        heads = sorted(r.sample(range(N), max(1, N // 8)))
        for i, k in zip(heads, _uneven(len(heads), total - N, total)):
            new[i] += min(k, case["max_len"] // 2)
    return new


# ---- inputs ------------------------------------------------------------------

class _Draws:
    def __init__(self, seed):
        self.seed = seed
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, dtype=BF16, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=self.g, device="cuda", dtype=F32) * std + mean).to(dtype)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")


def _offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=I64).cuda()


def prepare(case, seed):
    r, op = _Draws(seed), case["op"]
    s = {"case": case}
    if op == "pages":
        N, page = case["N"], case["page"]
        mp = case["max_len"] // page
        host = random.Random(seed)
        new = _new_tokens(case)
        ended = [case["ended"] and (k > 1 or host.random() < 0.1) for k in new]
        lens = [host.randint(0, case["max_len"] - (1 if e else k)) for k, e in zip(new, ended)]
        lengths = torch.tensor(lens, dtype=I64).cuda()
        held = (lengths + page - 1) // page
        pool = r.order(2 * N * mp).to(torch.int32)
        table = pool[: N * mp].view(N, mp)
        s["table"] = torch.where(torch.arange(mp, device="cuda") < held[:, None], table, -1)
        s["free"] = pool[N * mp:].clone()
        need = sum((n if e else (length + n) - (length + page - 1) // page * page) // page + 1
                   for n, e, length in zip(new, ended, lens))
        s["count"] = torch.tensor([min(N * mp // 2, need // 2 if case["short"] else N * mp)], dtype=I64).cuda()
        s["lengths"], s["new"] = lengths, torch.tensor(new, dtype=I64).cuda()
        s["ended"] = torch.tensor(ended).cuda() if case["ended"] else None
        s["rows"] = sum(new)
        return s
    if op == "store":
        M, page = case["tokens"], case["page"]
        both = r.normal((M, LAT + PE))  # one projection's output
        s["latent"], s["k_pe"] = both[:, :LAT], both[:, LAT:]
        s["weight"] = r.normal((LAT,), F32, 0.1, 1.0) if case["norm"] else None
        pages = (M + M // 4 + page) // page
        s["rows"] = r.normal((pages * page + 1, LAT + PE))  # the last: nobody's, where the plain form writes what is not stored
        s["cache"] = s["rows"][:-1].view(pages, page, LAT + PE)
        s["slots"] = r.order(pages * page)[:M].clone()
        s["slots"][M - M // 16:] = -1  # the rows that pad the batch
        return s
    if op == "decode":
        N, T, H, page = case["N"], case["T"], case["H"], case["page"]
        lens = _cached(case)
        mp = (max(lens) + page - 1) // page + 1
        held = [(k + page - 1) // page for k in lens]
        pages = sum(held) + 8
        order = r.order(pages).to(torch.int32)
        table = torch.full((N, mp), -1, dtype=torch.int32, device="cuda")
        live = torch.arange(mp, device="cuda") < torch.tensor(held, device="cuda")[:, None]
        table[live] = order[: sum(held)]
        s["table"], s["lengths"] = table, torch.tensor(lens, dtype=I64).cuda()
        s["top"] = max(max(lens), 1)
        s["cache"] = r.normal((pages, page, LAT + PE))
        # the queries: one product per head gives the latent part, a slice of the projection the other
        s["q_latent"] = r.normal((H, N * T, LAT)).transpose(0, 1).unflatten(0, (N, T))
        s["q_pe"] = r.normal((N, T, H, NOPE + PE))[..., NOPE:]
        return s
    H = case["H"]
    lq, lk = _lens(case)
    B, T, Tk = (1, sum(lq), sum(lk)) if case["packed"] else (case["n"], lq[0], lk[0])
    s["lens"] = (lq, lk) if case["packed"] else None
    s["cu"] = _offsets(lq) if case["packed"] else None
    s["cu_k"] = _offsets(lk) if case["packed"] and case["context"] else None
    s["q"] = r.normal((B, T, H, NOPE + PE), std=1.5)
    s["kv"] = r.normal((B, Tk, H, NOPE + VAL))
    s["k_pe"] = r.normal((B, Tk, LAT + PE))[..., LAT:]
    if op == "bwd":  # what the forward left, and the loss's gradient
        out, s["lse"] = _attention(s)
        s["out"] = out.to(BF16)
        s["d_out"] = r.normal((B, T, H, VAL))
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import gated_delta_rule_110_amd as kda

        if op == "pages":
            got = kda.page_assign(s["lengths"], s["new"], s["table"], s["free"], s["count"], c["page"], s["rows"],
                                  ended=s["ended"])
            return got | {"table": s["table"], "free": s["free"]}
        if op == "store":
            cache, normed = kda.latent_store(s["latent"], s["k_pe"], s["slots"], s["cache"], weight=s["weight"], eps=EPS,
                                             keep_normed=c["normed"])
            return {"cache": cache, "normed": normed}
        if op == "decode":
            out, lse = kda.latent_decode(s["q_latent"], s["q_pe"], s["cache"], s["lengths"], s["table"], SCALE)
            return {"out": out, "lse": lse}
        if op == "fwd":
            out, lse = kda.latent_fwd(s["q"], s["kv"], s["k_pe"], SCALE, causal=c["causal"], cu_seqlens=s["cu"],
                                      cu_seqlens_k=s["cu_k"])
            return {"out": out, "lse": lse}
        return kda.latent_bwd(s["q"], s["kv"], s["k_pe"], SCALE, s["out"], s["lse"], s["d_out"], causal=c["causal"],
                              cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"])
    if op == "pages":
        return _pages(s)
    if op == "store":
        return _store(s)
    if op == "decode":
        return _decode(s)
    if op == "fwd":
        out, lse = _attention(s)
        return {"out": out.to(BF16), "lse": lse}
    return _attention_bwd(s)


# ---- the plain forms -----------------------------------------------------------

def _pages(s):
    page, mp, F = s["case"]["page"], s["table"].shape[1], s["free"].shape[0]
    N, M = s["lengths"].shape[0], s["rows"]
    ended = torch.zeros(N, dtype=torch.bool, device="cuda") if s["ended"] is None else s["ended"]
    pages = lambda t: (t + page - 1) // page  # noqa: E731
    col = torch.arange(mp, device="cuda")
    # the pages of requests that have ended go back, in order
    give = torch.where(ended, pages(s["lengths"]).clamp(max=mp), 0)
    to = (s["count"] + torch.cumsum(give, 0) - give)[:, None] + col
    to = torch.where((col < give[:, None]) & (to < F), to, F)
    free = torch.cat([s["free"], s["free"].new_zeros(1)]).scatter(0, to.flatten(), s["table"].flatten())[:F]
    count = (s["count"] + give.sum()).clamp(max=F)
    # the others are taken from the stack's end, request after request while they last
    length = torch.where(ended, 0, s["lengths"])
    fits = length + s["new"] <= mp * page
    need = torch.where(fits, pages(length + s["new"]) - pages(length), 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (upto <= count))
    nth = col - pages(length)[:, None]
    take = granted[:, None] & (nth >= 0) & (nth < need[:, None])
    at = (count - 1 - (upto - need)[:, None] - nth).clamp(0, F - 1)
    table = torch.where(take, free[at], s["table"])
    s["table"].copy_(table)
    s["free"].copy_(free)
    # where every new token lies
    cu = torch.cat([s["new"].new_zeros(1), torch.cumsum(s["new"], 0)])
    row = torch.arange(M, device="cuda")
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = length[seq] + row - cu[seq]
    slot = table[seq, (pos // page).clamp(max=mp - 1)].long() * page + pos % page
    tokens = torch.where(granted, s["new"], 0)
    return {"slots": torch.where(granted[seq], slot, -1), "cu_seqlens": cu, "lengths": length + tokens, "granted": tokens,
            "free_count": count - torch.where(granted, need, 0).sum(), "table": s["table"], "free": s["free"]}


def _store(s):
    c = s["latent"].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    s["rows"][s["slots"]] = torch.cat([c.to(BF16), s["k_pe"]], 1)  # -1: the last row
    return {"cache": s["cache"], "normed": c.to(BF16) if s["case"]["normed"] else None}


def _decode(s):
    N, T, H = s["q_latent"].shape[:3]
    page = s["case"]["page"]
    pos = torch.arange(s["top"], device="cuda")
    at = s["table"].clamp(min=0).long()[:, pos // page] * page + pos % page
    keys = s["cache"].view(-1, LAT + PE)[at].float()                          # [N, top, 576]
    q = torch.cat([s["q_latent"], s["q_pe"]], -1).float().view(N, T * H, LAT + PE)
    seen = s["lengths"][:, None] - T + 1 + torch.arange(T, device="cuda")
    hidden = (pos >= seen[..., None]).repeat_interleave(H, 1)                 # [N, T H, top]
    x = (torch.bmm(q, keys.transpose(1, 2)) * SCALE).masked_fill(hidden, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(F32).min)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, keys[..., :LAT]) / total.clamp_min(torch.finfo(F32).tiny)
    lse = top + torch.log(total)
    return {"out": out.view(N, T, H, LAT).to(BF16), "lse": lse.view(N, T, H)}


def _blocks(s):
    """The batch as (q [b, H, Lq, 192], k [b, H, Lk, 192], v [b, H, Lk, 128], rows, key rows): all of it at once, or
    sequence by sequence where it is packed (padding to the longest would multiply the work)."""
    if s["lens"] is None:
        spans = [(slice(None), slice(None))]
    else:
        q0, k0 = 0, 0
        spans = []
        for a, b in zip(*s["lens"]):
            spans.append((slice(q0, q0 + a), slice(k0, k0 + b)))
            q0, k0 = q0 + a, k0 + b
    for i, j in spans:
        q, kv, pe = s["q"][:, i].float(), s["kv"][:, j].float(), s["k_pe"][:, j].float()
        k = torch.cat([kv[..., :NOPE], pe[:, :, None].expand(-1, -1, kv.shape[2], -1)], -1)
        yield q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous(), kv[..., NOPE:].transpose(1, 2).contiguous(), i, j


def _scores(q, k, causal):
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(SCALE)
    if causal:
        Lq, Lk = x.shape[-2:]
        x.masked_fill_(torch.ones(Lq, Lk, dtype=torch.bool, device="cuda").triu(Lk - Lq + 1), -math.inf)
    return x


def _attention(s):
    out = torch.zeros(*s["q"].shape[:3], VAL, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, device="cuda")
    for q, k, v, i, _ in _blocks(s):
        if q.shape[2] == 0 or k.shape[2] == 0:
            continue
        x = _scores(q, k, s["case"]["causal"])
        top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(F32).min)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        out[:, i] = (torch.matmul(p, v) / total.clamp_min(torch.finfo(F32).tiny)).transpose(1, 2)
        lse[:, i] = (top + torch.log(total))[..., 0].transpose(1, 2)
    return out, lse


def _attention_bwd(s):
    dq = torch.zeros(s["q"].shape, device="cuda")
    dkv = torch.zeros(s["kv"].shape, device="cuda")
    dpe = torch.zeros(s["k_pe"].shape, device="cuda")
    for q, k, v, i, j in _blocks(s):
        if q.shape[2] == 0 or k.shape[2] == 0:
            continue
        do = s["d_out"][:, i].float().transpose(1, 2).contiguous()
        delta = (do * s["out"][:, i].float().transpose(1, 2)).sum(-1, keepdim=True)
        lse = s["lse"][:, i].transpose(1, 2)[..., None]
        p = _scores(q, k, s["case"]["causal"]).sub_(lse.clamp_min(torch.finfo(F32).min)).exp_()
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(SCALE)
        dk = torch.matmul(ds.transpose(-1, -2), q)
        dq[:, i] = torch.matmul(ds, k).transpose(1, 2)
        dkv[:, j, :, :NOPE] = dk[..., :NOPE].transpose(1, 2)
        dkv[:, j, :, NOPE:] = torch.matmul(p.transpose(-1, -2), do).transpose(1, 2)
        dpe[:, j] = dk[..., NOPE:].sum(1)
    return {"dq": dq.to(BF16), "dkv": dkv.to(BF16), "dk_pe": dpe.to(BF16)}


# ---- the work of one pass --------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "pages":
        new = _new_tokens(case)
        rows = sum(new)
        # a request's numbers in and out, a slot a token, and the pages of prompts
        return {"bytes": 49 * case["N"] + 8 * rows + 12 * (rows // case["page"]), "flops": rows}
    if op == "store":
        M = case["tokens"] - case["tokens"] // 16
        return {"bytes": 2 * M * 2 * (LAT + PE) + 8 * case["tokens"] + 2 * case["tokens"] * LAT * case["normed"] + 4 * LAT,
                "flops": 4 * M * LAT * case["norm"]}
    if op == "decode":
        N, T, H, lens = case["N"], case["T"], case["H"], _cached(case)
        rows = N * T * H
        pairs = sum(max(0, k - T + 1 + t) for k in lens for t in range(T)) * H
        return {"bytes": 2 * sum(lens) * (LAT + PE) + rows * (2 * (LAT + PE) + 2 * LAT + 4) + 4 * sum(lens) // case["page"],
                "flops": 2 * pairs * (2 * LAT + PE)}
    H = case["H"]
    lq, lk = _lens(case)
    pairs = 0
    for a, b in zip(lq, lk):
        first = max(0, a - b)  # queries that see no key
        n = a - first
        pairs += n * b - (n * (n - 1) // 2 if case["causal"] else 0) if b else 0
    q, k = sum(lq), sum(lk)
    act = q * H * 2 * (NOPE + PE + VAL) + k * (H * 2 * (NOPE + VAL) + 2 * PE) + 4 * q * H
    if op == "fwd":
        return {"bytes": act, "flops": 2 * pairs * H * (NOPE + PE + VAL)}
    return {"bytes": act + q * H * 2 * (NOPE + PE + VAL) + k * (H * 2 * (NOPE + VAL) + 2 * PE),
            "flops": 2 * pairs * H * (3 * (NOPE + PE) + 2 * VAL)}


# ---- the definition, in 64 bits -----------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "store":
        c = s["latent"].double()
        if s["weight"] is not None:
            c = c / torch.sqrt((c * c).sum(1, keepdim=True) / LAT + EPS) * s["weight"].double()
        cache = s["cache"].double().view(-1, LAT + PE)
        keep = s["slots"] >= 0
        cache[s["slots"][keep]] = torch.cat([c, s["k_pe"].double()], 1)[keep]
        return {"cache": cache.view(s["cache"].shape), "normed": c if case["normed"] else None}
    if op == "decode":
        N, T, H, page = case["N"], case["T"], case["H"], case["page"]
        out = torch.zeros(N, T, H, LAT, dtype=F64, device="cuda")
        lse = torch.full((N, T, H), -math.inf, dtype=F64, device="cuda")
        rows = s["cache"].view(-1, page, LAT + PE)
        for n, length in enumerate(_cached(case)):
            keys = rows[s["table"][n, : (length + page - 1) // page].long()].reshape(-1, LAT + PE)[:length].double()
            for t in range(T):
                k = keys[: max(0, length - T + 1 + t)]
                if k.shape[0]:
                    q = torch.cat([s["q_latent"][n, t], s["q_pe"][n, t]], 1).double()
                    out[n, t], lse[n, t] = _softmax(q @ k.t() * SCALE, k[:, :LAT])
        return {"out": out, "lse": lse}
    return _exact_attention(s)


def _softmax(x, v):
    """(softmax(x) v, log of the sum of e^x) of rows of scores in 64 bits."""
    top = x.max(1).values
    e = torch.exp(x - top[:, None])
    z = e.sum(1)
    return (e @ v) / z[:, None], top + torch.log(z)


def _exact_attention(s):
    """Head by head and some queries at a time, each with the keys that it sees and no others before them."""
    c = s["case"]
    back = c["op"] == "bwd"
    B, T, H = s["q"].shape[:3]
    lq, lk = s["lens"] if s["lens"] else ([T] * B, [s["kv"].shape[1]] * B)
    flat = lambda t: t.reshape(-1, *t.shape[2:])  # noqa: E731
    q, kv, pe = flat(s["q"]), flat(s["kv"]), flat(s["k_pe"])
    out = torch.zeros(q.shape[0], H, VAL, dtype=F64, device="cuda")
    lse = torch.full((q.shape[0], H), -math.inf, dtype=F64, device="cuda")
    if back:
        d_out, kept, kept_lse = flat(s["d_out"]), flat(s["out"]), flat(s["lse"])
        dq = torch.zeros(q.shape, dtype=F64, device="cuda")
        dkv = torch.zeros(kv.shape, dtype=F64, device="cuda")
        dpe = torch.zeros(pe.shape, dtype=F64, device="cuda")
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        for h in range(H if a and b else 0):
            keys = torch.cat([kv[k0: k0 + b, h, :NOPE], pe[k0: k0 + b]], 1).double()
            vals = kv[k0: k0 + b, h, NOPE:].double()
            for i in range(0, a, 2048):
                m = min(2048, a - i)
                last = b - a + i + m if c["causal"] else b  # keys that the last of these queries sees
                if last <= 0:
                    continue
                r = slice(q0 + i, q0 + i + m)
                x = q[r, h].double() @ keys[:last].t() * SCALE
                if c["causal"]:
                    sees = torch.arange(b - a + i, last, device="cuda")[:, None] >= torch.arange(last, device="cuda")
                    x = torch.where(sees, x, -math.inf)
                live = torch.isfinite(x).any(1) if c["causal"] else torch.ones(m, dtype=torch.bool, device="cuda")
                if not back:
                    o, z = _softmax(torch.where(live[:, None], x, 0.0), vals[:last])
                    out[r, h] = torch.where(live[:, None], o, 0.0)
                    lse[r, h] = torch.where(live, z, -math.inf)
                    continue
                g = d_out[r, h].double()
                p = torch.where(live[:, None], torch.exp(x - torch.where(live, kept_lse[r, h].double(), 0.0)[:, None]), 0.0)
                e = p * (g @ vals[:last].t() - (g * kept[r, h].double()).sum(1, keepdim=True)) * SCALE
                dq[r, h] = e @ keys[:last]
                dk = e.t() @ q[r, h].double()
                dkv[k0: k0 + last, h, :NOPE] += dk[:, :NOPE]
                dkv[k0: k0 + last, h, NOPE:] += p.t() @ g
                dpe[k0: k0 + last] += dk[:, NOPE:]
        q0, k0 = q0 + a, k0 + b
    if back:
        return {"dq": dq.view(s["q"].shape), "dkv": dkv.view(s["kv"].shape), "dk_pe": dpe.view(s["k_pe"].shape)}
    return {"out": out.view(B, T, H, VAL), "lse": lse.view(B, T, H)}
