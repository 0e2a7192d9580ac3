"""Packed batches of latent attention: offsets that describe more blocks than 32 bits count, sequences that share
the tiles by which parts are planned, tables of long sequences, batches without queries, the autograd operation."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests.parity import say
from tests.test_gpu_latent import BF, SCALE, check, cu_of, make, run, same

pytestmark = pytest.mark.gpu


def test_overlapping_sequences_of_more_blocks_than_32_bits_count():
    """Offsets that go up and down describe 2^18 + 32 sequences of 8192 blocks each, over 2^31 of them, of which the
    table keeps as many as it has room for; none of the queries has a key."""
    T, pairs = 1 << 20, (1 << 18) + 32
    say("case latent %d overlapping sequences of %d tokens" % (pairs, T))
    q = torch.ones(1, 1, 1, 192, dtype=BF, device="cuda").expand(1, T, 1, 192)
    kv, pe = torch.ones(1, 8, 1, 256, dtype=BF, device="cuda"), torch.ones(1, 8, 64, dtype=BF, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int64).repeat(pairs).cuda()
    out, lse = kda.latent_fwd(q, kv, pe, SCALE, False, cu, torch.zeros_like(cu))
    torch.cuda.synchronize()
    # the blocks that are kept are each written whole
    assert out.shape == (1, T, 1, 128) and int((lse == float("-inf")).sum()) >= 128


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,T,Tk,H", [(8, 16, 8208, 4), (16, 1, 4096, 1), (4, 1000, 1000, 1)])
def test_even_sequences_are_split_as_a_batch_is(n, T, Tk, H, causal):
    """Few blocks of sequences of one length have the parts, and with them the bits, of the same sequences as batch rows."""
    say("case latent packed parts %s causal=%s" % ((n, T, Tk, H), causal))
    a = make(n, T, Tk, H, seed=30)
    want = run(a, causal)
    res = run({k: v.reshape(1, -1, *v.shape[2:]) for k, v in a.items()}, causal, cu_of([T] * n), cu_of([Tk] * n))
    same({k: v.reshape(want[k].shape) for k, v in res.items()}, want)


@pytest.mark.parametrize("lens,ctx", [([1, 1, 1, 1, 1], [100, 768, 769, 4000, 1]), ([700, 833, 1100, 40], [0, 0, 0, 900]),
                                      ([1] * 66, [2000] + [60] * 65)])
def test_parts_of_uneven_sequences(lens, ctx):
    """Sequences around the number of tiles from which they are split, and more of them than a wave counts through."""
    say("case latent packed parts of %d sequences" % len(lens))
    lens_k = [p + c for p, c in zip(lens, ctx)]
    a = make(1, sum(lens), sum(lens_k), 1, seed=31)
    res = run(a, True, cu_of(lens), cu_of(lens_k))
    check(a, res, True, lens, lens_k, "uneven")
    for piece in (0, 8):
        same(run(a, True, cu_of(lens), cu_of(lens_k), launch_piece=piece), res)


def packed(lens, lens_k, H, causal, seed, tail=0):
    a = make(1, sum(lens) + tail, sum(lens_k) + tail, H, seed=seed)
    return a, cu_of(lens), cu_of(lens_k)


@pytest.mark.parametrize("causal", [True, False])
def test_table_of_long_sequences(causal):
    """More sequences than a wave counts through, so that there is a table, and among them one of many blocks of keys
    and queries."""
    lens, ctx = [3] * 40 + [300] + [0, 7] * 15, [0] * 40 + [1300] + [5] * 30
    lens_k = [p + c for p, c in zip(lens, ctx)]
    say("case latent table of %d sequences causal=%s" % (len(lens), causal))
    for H in (1, 3):  # in parts and not
        a, cu, cu_k = packed(lens, lens_k, H, causal, 32)
        check(a, run(a, causal, cu, cu_k), causal, lens, lens_k, "table")


@pytest.mark.parametrize("long_q,long_k,causal", [(90, 66000, True), (90, 66000, False), (66000, 6, False), (66000, 70, True)])
def test_table_of_sequences_with_more_tiles_than_buckets(long_q, long_k, causal):
    say("case latent table with a sequence of %d queries and %d keys" % (long_q, long_k))
    lens, lens_k = [1, 2] * 35 + [long_q, 40], [2, 2] * 35 + [long_k, 40]
    for H in (1, 2) if long_q < 100 else (1,):
        a, cu, cu_k = packed(lens, lens_k, H, causal, 33)
        check(a, run(a, causal, cu, cu_k), causal, lens, lens_k, "buckets")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,Tk,H", [(1, 300, 2), (3, 70, 1), (1, 9000, 1)])
def test_no_queries(B, Tk, H, causal):
    """Keys that no query sees have gradients of zero."""
    say("case latent no queries %s causal=%s" % ((B, Tk, H), causal))
    a = make(B, 0, Tk, H, seed=34)
    for cu, cu_k in ((None, None), (cu_of([0, 0]), cu_of([Tk - 1, 1]))):
        if cu is not None and B > 1:
            continue
        outs = {"dq": torch.empty_like(a["q"]), "dkv": torch.full_like(a["kv"], 7.0), "dk_pe": torch.full_like(a["k_pe"], 7.0)}
        out, lse = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, causal, cu, cu_k)
        assert out.shape == (B, 0, H, 128) and lse.shape == (B, 0, H)
        kda.latent_bwd(a["q"], a["kv"], a["k_pe"], SCALE, out, lse, a["dy"], causal, cu, cu_k, outputs=outs)
        assert (outs["dkv"] == 0).all() and (outs["dk_pe"] == 0).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,ctx", [([100, 0, 60], None), ([5, 200, 0, 3], [100, 0, 7, 900]), ([10, 20], [-4, -20])])
def test_autograd_of_packed_batches(lens, ctx, causal):
    """The operation's output and gradients are the functions', bit for bit, with zeros behind the last sequence."""
    say("case latent autograd packed %s %s causal=%s" % (lens, ctx, causal))
    lens_k = lens if ctx is None else [p + c for p, c in zip(lens, ctx)]
    a, cu, cu_k = packed(lens, lens_k, 3, causal, 35, tail=11)
    if ctx is None:
        cu_k = None
    want = run(a, causal, cu, cu_k)
    leaves = [a[k].clone().requires_grad_() for k in ("q", "kv", "k_pe")]
    y = kda.latent_attention(*leaves, SCALE, causal, cu, cu_k)
    y.backward(a["dy"])
    got = {"out": y.detach(), "dq": leaves[0].grad, "dkv": leaves[1].grad, "dk_pe": leaves[2].grad}
    n = {"out": sum(lens), "dq": sum(lens), "dkv": sum(lens_k), "dk_pe": sum(lens_k)}
    same({k: v[:, :n[k]].contiguous() for k, v in got.items()}, {k: want[k][:, :n[k]].contiguous() for k in got})
    for k, v in got.items():
        assert v.shape[1] > n[k] and (v[:, n[k]:] == 0).all(), k


@pytest.mark.parametrize("T,Tk,lens", [(200, 200, None), (3, 3000, None), (150, 150, [70, 80])])
def test_without_lse(T, Tk, lens):
    """The C ABI takes no lse where it is not wanted: unsplit, in parts, packed."""
    from gated_delta_rule_110_amd import latent as L
    a = make(1, T, Tk, 2, seed=36)
    cu = cu_of(lens) if lens else None
    want, _ = kda.latent_fwd(a["q"], a["kv"], a["k_pe"], SCALE, True, cu)
    got = torch.empty_like(want)
    dsc, dev = L._latent_args(a["q"], a["kv"], a["k_pe"], SCALE, True, cu, None)
    ptr = [a[k].data_ptr() for k in ("q", "kv", "k_pe")]
    st = kda.library().kda_latent_fwd(*ptr, None if cu is None else cu.data_ptr(), None, got.data_ptr(), None, dsc,
                                      torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(got, want)
