"""The global gradient norm over the whole range of float32 (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32

# fp32 sums of n positive squares: a thread adds at most n / 2^17 + 64 of them one by one,
# then trees; far below 2^-16 of the sum for the sizes here, half of it after the root, and
# half a step of the result (2^-150 where that is subnormal)
REL = 2.0 ** -17


def _check(grads):
    want = math.sqrt(math.fsum(float((x.double() ** 2).sum()) for x in grads))
    got = float(binding.tp_grad_norm(grads))
    assert abs(got - want) <= REL * want + 2.0 ** -150, (got, want)


# 2^-75 is the largest value whose square fp32 drops; the last are subnormal
@pytest.mark.parametrize("size", [1e-15, 1e-20, 2.0 ** -75, 1e-23, 1e-30, 1e-38, 1e-42, 2.0 ** -149])
@pytest.mark.parametrize("offset", [0, 1])
def test_small_gradients(size, offset):
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.full((5000 + offset,), size, device="cuda")[offset:],
             (torch.randn(100003 + offset, generator=g, device="cuda") * size)[offset:], torch.zeros(40000, dtype=BF, device="cuda")]
    if size > 2.0 ** -133:  # bfloat16's smallest
        grads += [torch.full((300 + offset,), size, dtype=BF, device="cuda")[offset:], torch.full((7,), size, dtype=BF, device="cuda")]
    _check(grads)


@pytest.mark.parametrize("dt", [BF, FP])
def test_many_values_whose_squares_fp32_drops(dt):
    x = torch.full((1 << 26,), 2.0 ** -75, device="cuda").to(dt)
    assert abs(float(binding.tp_grad_norm([x])) - 2.0 ** -62) <= REL * 2.0 ** -62
    _check([x[:1], x[3:40001]])
    # one value that others' squares must not be lost beside
    x[17] = 2.0 ** -63
    assert abs(float(binding.tp_grad_norm([x])) - math.sqrt(2.0 ** -124 + 2.0 ** -126)) <= 2 * REL * 2.0 ** -62


def test_sizes_of_every_kind_together():
    small = torch.full((50000,), 1e-25, device="cuda")
    for other in (1.0, 1e-10, 1e-17, 1e-22, 1e20, 1e37):
        _check([small, torch.full((9,), other, device="cuda"), small.to(BF)])
    _check([torch.full((70000,), 2.0 ** -24, dtype=HF, device="cuda"), torch.full((1000,), 65504.0, dtype=HF, device="cuda")])
    assert float(binding.tp_grad_norm([torch.zeros(100000, device="cuda"), torch.zeros(3, dtype=BF, device="cuda")])) == 0.0
    for bad in (math.nan, math.inf):
        small[77] = bad
        got = float(binding.tp_grad_norm([small]))
        assert math.isnan(got) if math.isnan(bad) else math.isinf(got)


def test_an_infinite_norm_and_an_infinite_limit():
    grads = [torch.ones(5000, dtype=BF, device="cuda"), torch.full((3,), math.inf, device="cuda")]
    norm, out = binding.tp_grad_clip(grads, math.inf)
    assert math.isinf(float(norm)) and all(torch.isnan(x.float()).all() for x in out)
