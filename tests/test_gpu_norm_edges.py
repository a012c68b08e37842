"""The final LayerNorm where it can go wrong beside plain batches: statistics
near the ends of fp32's range."""

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import head_reference as ref
from tests.test_gpu_final_norm import draw

pytestmark = pytest.mark.gpu

# a row of one CTA, one of a cluster, one at odd addresses, one beyond both
WIDTHS = [1024, 8192, 1023, 65544]


def check_backward(x, dy, gamma, mean, rstd, dtype):
    dx, dgamma, dbeta = binding.tp_ln_backward(dy, x, gamma, mean, rstd)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    args = [ref.f64(t) for t in (dy, x, gamma, mean, rstd)]
    for got, want, b, name in zip((dx, dgamma, dbeta), ref.ln_backward(*args), ref.ln_backward_bounds(*args, dtype),
                                  ("dx", "dgamma", "dbeta")):
        ref.within(got, want, b, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("size", [1e15, 1e-12])
def test_rows_of_any_size(h, size, dtype):
    """rstd of 1e-15 and 1e12, whose cubes fp32 does not hold; dx does."""
    c = {k: v.cuda() for k, v in draw(9, h, dtype, h).items()}
    x = (c["x"].double() * size).to(dtype)
    dy = (c["dy"].double() + c["x"].double()).to(dtype)  # so that mean(g xhat) is not small
    _, mean, rstd = binding.tp_ln_forward(x, c["gamma"], c["beta"], 1e-30)
    assert bool(((rstd * size > 0.1) & (rstd * size < 10.0)).all())
    check_backward(x, dy, c["gamma"], mean, rstd, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h", WIDTHS)
def test_constant_rows_with_a_tiny_eps(h, dtype):
    """rstd is 1e15 and x - mean is 0: dx = rstd (g - mean(g)), finite."""
    c = {k: v.cuda() for k, v in draw(5, h, dtype, h + 1).items()}
    x = torch.full_like(c["x"], 2.5)
    y, mean, rstd = binding.tp_ln_forward(x, c["gamma"], c["beta"], 1e-30)
    assert torch.equal(mean, torch.full_like(mean, 2.5)) and bool((rstd > 9e14).all())
    assert torch.equal(y, c["beta"].expand_as(y))
    check_backward(x, c["dy"], c["gamma"], mean, rstd, dtype)
