"""RMS normalisation at the smallest eps that it takes: rows of zeros stay zero, tiny ones are normalised."""
import pytest
import torch

import gated_delta_rule_110_amd as kda
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("D", [64, 77, 4096])
def test_smallest_eps(D):
    x = torch.zeros(3, D, dtype=BF, device="cuda")
    x[1] = 1e-19                       # squares of 2^-126
    x[2] = torch.randn(D, device="cuda").to(BF)
    w = torch.ones(D, device="cuda")
    eps = 2.0 ** -126
    y, _ = kda.rmsnorm_fwd(x, w, eps)
    ref, _ = R.rmsnorm(R.d(x), R.d(w), eps)
    # the sum's and the root's half steps, and for the squares at the edge of fp32's range 2^-12 of them
    R.check(y, ref, BF, 64 * R.U * ref.abs() + 2.0 ** -12 * ref.abs() * (R.d(x).abs() < 1e-18), "y")
    q, s, _ = kda.rmsnorm_quant(x, w, eps)
    assert (q[0].float() == 0).all() and s.isfinite().all()
    g = kda.rmsnorm_bwd(x, w, eps, x)
    assert (g["dx"][0] == 0).all() and g["dweight"].isfinite().all()
    for bad in (1e-40, 2.0 ** -127):
        with pytest.raises(ValueError):
            kda.rmsnorm_fwd(x, w, bad)
