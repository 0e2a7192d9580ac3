"""Packed batches of latent attention: offsets that describe more blocks than 32 bits count, sequences that share
the tiles by which parts are planned."""
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
