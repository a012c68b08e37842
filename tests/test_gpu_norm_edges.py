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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h", [(65, 1024), (33, 72), (6, 8192), (33, 1023), (3, 65544)])
def test_bad_rows_stay_by_themselves(T, h, dtype):
    """NaN and infinities in single values of x or dy: nothing finite in those rows'
    y and dx, the other rows bit for bit as without them, dbeta as its definition
    says."""
    c = {k: v.cuda() for k, v in draw(T, h, dtype, T + h).items()}
    y0, m0, r0 = binding.tp_ln_forward(c["x"], c["gamma"], c["beta"], 1e-5)
    dx0, _, db0 = binding.tp_ln_backward(c["dy"], c["x"], c["gamma"], m0, r0)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[0, T // 2, T - 1]] = True
    x = c["x"].clone()
    x[0, 0], x[T // 2, h - 1], x[T - 1, h // 2] = float("nan"), float("inf"), -float("inf")
    y, m, r = binding.tp_ln_forward(x, c["gamma"], c["beta"], 1e-5)
    assert bool(torch.isnan(y[bad].float()).all()) and torch.equal(y[~bad], y0[~bad])
    assert torch.equal(m[~bad], m0[~bad]) and torch.equal(r[~bad], r0[~bad])
    dx, dg, db = binding.tp_ln_backward(c["dy"], x, c["gamma"], m, r)
    assert bool(torch.isnan(dx[bad].float()).all()) and torch.equal(dx[~bad], dx0[~bad])
    assert bool(torch.isnan(dg).all()) and torch.equal(db, db0)
    dy = c["dy"].clone()
    dy[0, 0], dy[T // 2, h - 1], dy[T - 1, h // 2] = float("nan"), float("inf"), -float("inf")
    dx, dg, db = binding.tp_ln_backward(dy, c["x"], c["gamma"], m0, r0)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    # an infinite g: inf - inf xhat, infinite or NaN by xhat's sign
    assert not bool(torch.isfinite(dx[bad].float()).any()) and torch.equal(dx[~bad], dx0[~bad])
    at = torch.tensor([0, h - 1, h // 2], device="cuda")
    assert not bool(torch.isfinite(dg[at]).any()) and bool(torch.isnan(db[0]))
    assert float(db[h - 1]) == float("inf") and float(db[h // 2]) == -float("inf")
    rest = torch.ones(h, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(db[rest], db0[rest]) and bool(torch.isfinite(dg[rest]).all())
