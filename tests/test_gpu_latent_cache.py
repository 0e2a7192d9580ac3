"""Latent attention in its absorbed form, the store into its cache and the pages of
a serving step, against the 64-bit (or whole-number) oracle, and a run of them all."""
import random

import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import latent_ref as R
from tests.layer_ref import d
from tests.parity import say

pytestmark = pytest.mark.gpu
BF, F32, I64 = torch.bfloat16, torch.float32, torch.int64
SCALE = 192 ** -0.5


def make(lengths, T, H, page, seed=0, spare=3, std=1.0):
    """Queries, a cache whose unused rows are NaN, and its tables (unused entries far outside)."""
    g = torch.Generator().manual_seed(100 * seed + T + H + page)
    N = len(lengths)
    held = [-(-k // page) for k in lengths]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    mp = max(held + [0]) + 1
    table = torch.full((N, mp), 0x7fffffff, dtype=torch.int32)
    cache = torch.full((pages, page, 576), float("nan"))
    at = 0
    for n, k in enumerate(lengths):
        table[n, :held[n]] = order[at:at + held[n]]
        rows = torch.full((held[n] * page, 576), float("nan"))
        rows[:k] = torch.randn(k, 576, generator=g)
        if held[n]:
            cache[order[at:at + held[n]].long()] = rows.view(held[n], page, 576)
        at += held[n]
    ql, qp = (torch.randn(N, T, H, w, generator=g) * std for w in (512, 64))
    return {"ql": ql.to(BF).cuda(), "qp": qp.to(BF).cuda(), "cache": cache.to(BF).cuda(),
            "lengths": torch.tensor(lengths, dtype=I64).cuda(), "table": table.cuda()}


def run(a, **kw):
    return kda.latent_decode(a["ql"], a["qp"], a["cache"], a["lengths"], a["table"], SCALE, **kw)


def check(a, got, label):
    ref = R.decode(d(a["ql"]), d(a["qp"]), d(a["cache"]), a["lengths"].cpu(), a["table"].cpu(), SCALE)
    R.within(got[0], ref["out"], ref["tol_out"], label + " out")
    R.within(got[1], ref["lse"], ref["tol_lse"], label + " lse")


@pytest.mark.parametrize("lengths,T,H,page", [
    ([1], 1, 1, 1), ([0], 1, 4, 16), ([63, 64, 65], 1, 32, 64), ([5, 0, 200, 1], 1, 16, 16), ([1000], 1, 33, 32),
    ([129, 31, 32, 33], 1, 64, 32), ([700, 3], 1, 128, 128), ([300, 2, 64], 4, 16, 16), ([260, 1, 0, 7], 7, 5, 256),
    ([90], 90, 3, 8), ([500, 130], 130, 2, 64), ([64] * 300, 1, 2, 64), ([3000], 1, 8, 2), ([4097, 5000], 2, 20, 4096),
    ([20000], 1, 40, 64), ([1, 1, 1], 1, 65, 1)])
def test_decode(lengths, T, H, page):
    say("case decode %s T=%d H=%d page=%d" % (lengths[:6], T, H, page))
    a = make(lengths, T, H, page)
    check(a, run(a), "decode")


@pytest.mark.parametrize("lengths,T,H", [
    ([1024] * 16, 1, 32), ([2048, 1024, 0, 1024], 2, 40),                 # row tiles of even shares: none begins within one
    ([6000, 4, 0, 2500, 33, 31, 4000], 4, 16), ([3000, 1, 1, 2900], 1, 32),  # several begin within a share
    ([(37 * i) % 90 for i in range(700)], 1, 3), ([(61 * i) % 200 for i in range(600)], 2, 40)])
def test_decode_shares(lengths, T, H):
    say("case decode shares %s.. T=%d H=%d" % (lengths[:6], T, H))
    a = make(lengths, T, H, 32, seed=9)
    check(a, run(a), "shares")


def test_decode_tokens_without_keys():
    a = make([2, 0, 5], 4, 8, 16, seed=1)
    out, lse = run(a)
    for n, seen in enumerate(([0, 0, 1, 2], [0] * 4, [2, 3, 4, 5])):
        for t, k in enumerate(seen):
            assert (lse[n, t] == float("-inf")).all() == (k == 0)
            assert (out[n, t] == 0).all() == (k == 0)


def test_decode_no_sequence_no_cache():
    a = make([4], 1, 4, 16)
    out, lse = kda.latent_decode(a["ql"][:0], a["qp"][:0], a["cache"], a["lengths"][:0], a["table"][:0], SCALE)
    assert out.shape == (0, 1, 4, 512)
    out, lse = kda.latent_decode(a["ql"], a["qp"], a["cache"][:0], a["lengths"], a["table"], SCALE)
    assert (out == 0).all() and (lse == float("-inf")).all()
    out, lse = kda.latent_decode(a["ql"], a["qp"], a["cache"], a["lengths"], a["table"][:, :0].contiguous(), SCALE)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_decode_wrong_tables_stay_inside():
    a = make([300, 70], 2, 16, 16, seed=2)
    a["cache"].nan_to_num_(0.5)
    a["lengths"].copy_(torch.tensor([1 << 62, -5]))
    a["table"].copy_(torch.where(torch.arange(a["table"].shape[1]) % 2 == 0, -7, 0x7fffffff).to(torch.int32).cuda().expand(a["table"].shape))
    out, lse = run(a)
    torch.cuda.synchronize()
    assert out[0].isfinite().all() and (out[1] == 0).all() and (lse[1] == float("-inf")).all()


def test_decode_strides():
    """Queries as they leave a product per head, and a projection of which they are a part."""
    a = make([200, 90, 17], 2, 12, 32, seed=3)
    want = run(a)
    ql = a["ql"].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    wide = torch.randn(3, 2, 12, 192, device="cuda").to(BF)
    wide[..., 128:] = a["qp"]
    got = run(a | {"ql": ql, "qp": wide[..., 128:]})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = a["ql"][:, :, :1].expand(a["ql"].shape)
    got, want = run(a | {"ql": e}), run(a | {"ql": e.contiguous()})
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim", [17, 300, 570])
def test_decode_special_values(dim, bad):
    """A drafted token's value that is not finite leaves the tokens before it alone; one in another sequence all."""
    a = make([700, 400], 3, 24, 16, seed=4)
    want = run(a)
    for pos, clean in ((699, 2), (698, 1)):  # seen by token 2 alone, by tokens 1 and 2
        b = dict(a, cache=a["cache"].clone())
        b["cache"][int(a["table"][0, pos // 16]), pos % 16, dim] = bad
        out, lse = run(b)
        assert torch.equal(out[1], want[0][1]) and torch.equal(lse[1], want[1][1])
        assert torch.equal(out[0, :clean], want[0][0, :clean]) and torch.equal(lse[0, :clean], want[1][0, :clean])
        if bad != bad:
            assert out[0, clean:, :, min(dim, 511)].isnan().all()


def test_decode_large_scores():
    a = make([500, 64], 2, 16, 32, seed=5, std=60.0)
    check(a, run(a), "large")
    a["cache"][:, :, :] = a["cache"].nan_to_num(0.0)
    a["ql"].zero_()
    a["qp"].zero_()
    check(a, run(a), "equal")


def test_decode_rising_scores():
    """Scores that rise from tile to tile by more than the kept maximum allows, and fall again."""
    for sign in (1.0, -1.0):
        a = make([640], 1, 16, 64, seed=6)
        a["ql"].zero_()
        a["qp"].zero_()
        a["qp"][..., 0] = 1.0
        pos = torch.arange(640)
        a["cache"][a["table"][0, pos // 64].long().cpu(), pos % 64, 512] = (sign * 16.0 * pos / 64 * 50).to(BF).cuda()
        check(a, run(a), "rising %g" % sign)


def test_decode_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 entries, its last pages in use."""
    page, pages = 64, 60000
    cache = torch.empty(pages, page, 576, dtype=BF, device="cuda")
    assert cache.numel() > 1 << 31
    cache[-40:].normal_()
    g = torch.Generator().manual_seed(5)
    a = {"ql": torch.randn(2, 1, 16, 512, generator=g).to(BF).cuda(), "qp": torch.randn(2, 1, 16, 64, generator=g).to(BF).cuda(),
         "cache": cache, "lengths": torch.tensor([1000, 1200], dtype=I64).cuda(),
         "table": (pages - 1 - torch.arange(40, dtype=torch.int32).view(2, 20)).to(torch.int32).cuda()}
    say("case decode 2^31 entries")
    got = run(a)
    small = dict(a, cache=cache[-40:], table=a["table"] - (pages - 40))
    check(small, got, "far")
    slots = torch.tensor([(pages - 1) * page + 63, 5], dtype=I64).cuda()
    row = torch.randn(2, 512, device="cuda").to(BF), torch.randn(2, 64, device="cuda").to(BF)
    kda.latent_store(*row, slots, cache)
    assert torch.equal(cache[-1, 63], torch.cat(row, -1)[0]) and torch.equal(cache[0, 5], torch.cat(row, -1)[1])


def test_decode_repeats_and_graphs():
    sets = [make([900, 64, 3000], 1, 16, 64, seed=7), make([70] * 40, 2, 40, 16, seed=8)]
    want = [run(a) for a in sets]
    for a, w in zip(sets, want):
        for _ in range(3):
            got = run(a)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    ws = torch.empty(max(kda.latent_decode_workspace_size(*a["ql"].shape[:3]) for a in sets), dtype=torch.uint8, device="cuda")
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]
    graphs = []
    for a, o in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(a, out=o[0], lse=o[1], workspace=ws)
        graphs.append(g)
    for rep in range(3):
        for i in (rep % 2, 1 - rep % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
            o[0].zero_()
    # a replay goes by the lengths that stand there then
    sets[0]["lengths"].copy_(torch.tensor([10, 0, 2048]))
    graphs[0].replay()
    torch.cuda.synchronize()
    check(sets[0], outs[0], "new lengths")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(sets[1])
    st.synchronize()
    assert torch.equal(got[0], want[1][0])


# ---- the store ---------------------------------------------------------------------

@pytest.mark.parametrize("norm", [None, BF, F32])
@pytest.mark.parametrize("tokens", [0, 1, 3, 64, 1000, 9000])
def test_store(tokens, norm):
    g = torch.Generator().manual_seed(tokens)
    wide = torch.randn(tokens, 600, generator=g).to(BF).cuda()
    latent, pe = wide[:, :512], wide[:, 512:576]
    w = None if norm is None else (1 + 0.1 * torch.randn(512, generator=g)).to(norm).cuda()
    pages = tokens // 16 + 3
    cache = torch.randn(pages, 16, 576, generator=g).to(BF).cuda()
    before = cache.clone()
    slots = torch.randperm(pages * 16, generator=g)[:tokens]
    slots[::5] = torch.where(torch.arange(len(slots[::5])) % 2 == 0, -1, pages * 16)  # not stored
    got, normed = kda.latent_store(latent, pe, slots.cuda(), cache, weight=w, eps=1e-5, keep_normed=True)
    assert got is cache
    x = d(latent)
    n = x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * d(w)
    # rounded once, from an fp32 value off by the sum's (512 + 8 half steps at most, half of them through the root) and 4 more
    R.within(normed, n, n.abs() * (0.0 if w is None else R.HALF * 1.01 + 264 * R.U), "normed")
    keep = (slots >= 0) & (slots < pages * 16)
    flat = cache.view(-1, 576)
    assert torch.equal(flat[slots[keep].cuda()], torch.cat([normed, pe], -1)[keep.cuda()])
    rest = torch.ones(pages * 16, dtype=torch.bool)
    rest[slots[keep]] = False
    assert torch.equal(flat[rest.cuda()], before.view(-1, 576)[rest.cuda()])


def test_store_shapes_and_zero_rows():
    latent, pe = torch.zeros(2, 5, 512, dtype=BF, device="cuda"), torch.ones(2, 5, 64, dtype=BF, device="cuda")
    latent[1] = float("inf")
    cache = torch.full((1, 16, 576), 3.0, dtype=BF, device="cuda")
    _, normed = kda.latent_store(latent, pe, torch.arange(10, device="cuda").view(2, 5), cache,
                                 weight=torch.ones(512, device="cuda"), eps=2.0 ** -126, keep_normed=True)
    assert normed.shape == latent.shape and (normed[0] == 0).all() and normed[1].isnan().all()
    assert (cache[0, 10:] == 3).all() and (cache[0, :5, :512] == 0).all() and (cache[0, :10, 512:] == 1).all()
    _, none = kda.latent_store(latent, pe, torch.full((2, 5), -1, device="cuda"), cache)
    assert none is None


# ---- pages ---------------------------------------------------------------------------

def step(lengths, new, table, free, count, size, tokens, ended=None, in_place=False):
    """One call and the oracle's answer, compared; returns the call's."""
    ref = R.pages(lengths, new, table, free, count, size, tokens, ended)
    t = lambda v, dt=I64: torch.tensor(v, dtype=dt).cuda()  # noqa: E731
    a = [t(lengths), t(new), t(table, torch.int32).view(len(lengths), len(table[0]) if table else 0), t(free, torch.int32), t([count])]
    outputs = {"lengths": a[0], "free_count": a[4]} if in_place else None
    got = kda.page_assign(*a, size, tokens, ended=None if ended is None else torch.tensor(ended).cuda(), outputs=outputs)
    got = got | {"table": a[2], "free": a[3]}
    for k, v in ref.items():
        assert got[k].tolist() == v, k
    return got


def random_step(r, N, mp, size, spare, tight):
    lengths = [r.choice([0, 1, size, r.randint(0, mp * size)]) for _ in range(N)]
    ended = [r.random() < 0.3 for _ in range(N)]
    new = [r.choice([0, 1, 1, 1, r.randint(0, 2 * size), r.randint(0, mp * size)]) for _ in range(N)]
    pool = list(range(N * mp + spare))
    r.shuffle(pool)
    table = [[pool.pop() if i < -(-k // size) else -1 for i in range(mp)] for k in lengths]
    free = pool + [-9] * (N * mp)
    return lengths, new, table, free, len(pool) // tight, ended


@pytest.mark.parametrize("N,mp,size", [(1, 1, 1), (1, 4, 16), (3, 5, 8), (17, 3, 64), (64, 40, 16), (65, 7, 2), (300, 12, 32), (1500, 3, 4),
                                       (2500, 2, 256)])
def test_pages(N, mp, size):
    for seed in range(4):
        say("case pages N=%d mp=%d size=%d seed %d" % (N, mp, size, seed))
        r = random.Random(seed)
        lengths, new, table, free, count, ended = random_step(r, N, mp, size, r.choice([0, 3, N * mp]), r.choice([1, 1, 3, 10]))
        step(lengths, new, table, free, count, size, sum(new) + r.choice([0, 0, 5]), ended, in_place=seed % 2 == 1)
        step(lengths, new, table, free, count, size, max(0, sum(new) - r.randint(0, 9)), None)


def test_pages_edges():
    step([], [], [], [5, 6], 2, 16, 4)
    step([3], [0], [[7, -1]], [1], 1, 4, 0)
    step([4], [1], [[7, -1]], [1], 0, 4, 1)           # needs a page, none left
    step([4, 2], [1, 1], [[7, -1], [8, -1]], [1], 0, 4, 2)  # the second needs none
    step([8], [1], [[7, 9]], [1], 1, 4, 1)            # the table's row is full
    step([8, 8], [3, 0], [[7, 9], [5, 4]], [1, 2], 1, 4, 3, [True, True])  # back, and one of them taken again; a full stack
    step([-3, 1 << 40], [-2, 1], [[7, 9], [5, 4]], [1, 2], 5, 4, 3)        # numbers out of range
    step([2] * 5, [3] * 5, [[i, -1] for i in range(5)], [9, 8, 7, 6, 5], 5, 4, 7)  # fewer rows than tokens


def test_pages_large_prompts():
    r = random.Random(9)
    lengths, ended = [r.randint(0, 500) for _ in range(40)], [i % 7 == 0 for i in range(40)]
    new = [r.choice([1, r.randint(0, 7000)]) for _ in range(40)]
    mp, size = 600, 16
    pool = list(range(40 * mp))
    r.shuffle(pool)
    table = [[pool.pop() if i < -(-k // size) else -1 for i in range(mp)] for k in lengths]
    step(lengths, new, table, pool + [0] * 3000, len(pool), size, sum(new) + 1000, ended)


def test_pages_in_a_graph():
    N, mp, size = 6, 20, 8
    i64 = lambda v: torch.tensor(v, dtype=I64).cuda()  # noqa: E731
    lengths, new, count = i64([0] * N), i64([5, 1, 9, 0, 16, 3]), i64([N * mp])
    table, free = torch.full((N, mp), -1, dtype=torch.int32, device="cuda"), torch.arange(N * mp, dtype=torch.int32, device="cuda")
    first = [lengths.tolist(), table.tolist(), free.tolist(), int(count)]
    out = kda.page_assign(lengths, new, table, free, count, size, 34, outputs={"lengths": lengths, "free_count": count})
    for t, v in ((lengths, first[0]), (table, first[1]), (free, first[2]), (count, [first[3]])):
        t.copy_(torch.tensor(v, dtype=t.dtype))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.page_assign(lengths, new, table, free, count, size, 34, outputs=out)
    state = first
    for rep in range(4):
        g.replay()
        torch.cuda.synchronize()
        ref = R.pages(state[0], new.tolist(), state[1], state[2], state[3], size, 34)
        for k in ("slots", "cu_seqlens", "lengths", "granted", "free_count"):
            assert out[k].tolist() == ref[k], (rep, k)
        assert table.tolist() == ref["table"] and free.tolist() == ref["free"]
        state = [ref["lengths"], ref["table"], ref["free"], ref["free_count"][0]]


# ---- together ------------------------------------------------------------------------

def test_a_serving_run():
    """Prompts through the expanded form, then generation through the absorbed one, as a layer would: the projections
    are plain products, everything between is the library's.  Every generated token's output, expanded by the values'
    projection, is that of attention over the whole sequence in 64 bits; a request ends on the way and another takes
    its row."""
    H, N, size, mp = 4, 3, 16, 12
    g = torch.Generator().manual_seed(21)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wk, wv = (n(H, 128, 512) / 512 ** 0.5).to(BF).cuda(), (n(H, 128, 512) / 512 ** 0.5).to(BF).cuda()
    w_norm = (1 + 0.1 * n(512)).cuda()
    cache = torch.full((N * mp, size, 576), float("nan"), dtype=BF, device="cuda")
    table, free = torch.full((N, mp), -1, dtype=torch.int32, device="cuda"), torch.arange(N * mp, dtype=torch.int32, device="cuda")
    lengths, count = torch.zeros(N, dtype=I64, device="cuda"), torch.tensor([N * mp], dtype=I64, device="cuda")
    seen = [[] for _ in range(N)]  # every request's stored rows, as the oracle reads them

    def advance(new, ended=None):
        rows = sum(new) + 2  # two rows of padding
        kv_a, q = n(rows, 576).to(BF).cuda(), (n(1, rows, H, 192) * 1.5).to(BF).cuda()
        p = kda.page_assign(lengths, torch.tensor(new, dtype=I64).cuda(), table, free, count, size, rows,
                            ended=None if ended is None else torch.tensor(ended).cuda(),
                            outputs={"lengths": lengths, "free_count": count})
        assert p["granted"].tolist() == new
        _, normed = kda.latent_store(kv_a[:, :512], kv_a[:, 512:], p["slots"], cache, weight=w_norm, keep_normed=True)
        at = 0
        for i, k in enumerate(new):
            if ended is not None and ended[i]:
                seen[i].clear()
            seen[i].extend(torch.cat([normed, kv_a[:, 512:]], -1)[at:at + k].cpu())
            at += k
        return p, normed, kv_a[:, 512:], q

    def oracle(q, rows):
        """q [T, H, 192] of a request's last tokens over its rows, with keys and values by the projections in 64 bits."""
        r = d(torch.stack(rows))
        k, v = (torch.einsum("tc,hdc->thd", r[:, :512], d(w)) for w in (wk, wv))
        kv = torch.cat([k, v], -1)
        return R.attention(d(q), kv, r[:, 512:], SCALE, True, [q.shape[0]], [r.shape[0]])["out"]

    # prompts
    new = [50, 17, 3]
    p, normed, pe, q = advance(new)
    kv = torch.matmul(normed, torch.cat([wk, wv], 1).permute(2, 0, 1).reshape(512, -1).contiguous()).view(1, -1, H, 256)
    out, _ = kda.latent_fwd(q, kv, pe[None], SCALE, cu_seqlens=p["cu_seqlens"])
    at = 0
    for i, k in enumerate(new):
        ref = oracle(q[0, at:at + k], seen[i])
        assert float((d(out[0, at:at + k]) - ref).norm()) <= 1e-2 * float(ref.norm()), i
        at += k

    def generate(T, ended=None):
        p, normed, pe, q = advance([T] * N, ended)
        q = q[0, :N * T].view(N, T, H, 192)
        ql = torch.bmm(q[..., :128].reshape(N * T, H, 128).transpose(0, 1).contiguous(), wk).transpose(0, 1).view(N, T, H, 512)
        o, _ = kda.latent_decode(ql, q[..., 128:], cache, lengths, table, SCALE)
        y = torch.einsum("nthc,hdc->nthd", o.float(), wv.float())
        for i in range(N):
            ref = oracle(q[i], seen[i])
            # bf16 roundings of the absorbed query, the probabilities and the mean latent: 2^-8 each of values of one size
            assert float((d(y[i]) - ref).norm()) <= 1.5e-2 * float(ref.norm()), i
    for T in (1, 1, 3, 1):
        generate(T)
    generate(5, [False, True, False])
    generate(1)
    assert [len(s) for s in seen] == lengths.tolist()
