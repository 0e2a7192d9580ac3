"""Packed batches of latent attention: offsets that describe more blocks than 32 bits count."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests.parity import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SCALE = 192 ** -0.5


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
