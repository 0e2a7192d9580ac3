"""Latent attention over values of up to 2^56 in magnitude, with maxima that stay behind."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import test_gpu_latent as E
from tests import test_gpu_latent_cache as C
from tests.parity import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rise", [0.0, 26.0, 80.0])
def test_absorbed_form_of_large_values(rise):
    """Scores that rise by `rise` over the rows: below 2^40 without new maxima, above it with them."""
    say("case decode of large values, rise %g" % rise)
    n = 2000
    a = C.make([n, 700], 2, 20, 32, seed=40)
    a["ql"].mul_(2.0 ** -56)
    a["qp"].zero_()
    a["qp"][..., 0] = 16.0
    cache = a["cache"]
    cache[..., :512] = (cache[..., :512] * 2.0 ** 54).clamp(-2.0 ** 56, 2.0 ** 56)  # NaN where there is no row
    cache[..., 512:].mul_(2.0 ** -6)
    for s, k in enumerate((n, 700)):
        at = torch.arange(k, device="cuda")
        pages = a["table"][s, (at // 32).long()].long()
        cache[pages, at % 32, 512] = (at / k * rise / (16.0 * C.SCALE)).to(C.BF)
    out, lse = C.run(a)
    assert out.isfinite().all() and out.abs().max() > 2.0 ** 46
    C.check(a, (out, lse), "large")


def test_expanded_form_of_large_values():
    say("case latent of large values")
    a = E.make(1, 300, 1000, 2, seed=41)
    a["kv"][..., 128:] = (a["kv"][..., 128:] * 2.0 ** 54).clamp(-2.0 ** 56, 2.0 ** 56)
    a["k_pe"][0, :, 0] = (torch.arange(1000) * 0.05).cuda()
    a["q"][..., 128] = 2.0
    a["dy"].mul_(2.0 ** -54)
    res = E.run(a, True)
    E.check(a, res, True, [300], [1000], "large")
