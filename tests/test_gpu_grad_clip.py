"""Global gradient norm and clipping against 64-bit forms (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
TYPES = (BF, FP, HF)


def _grads(sizes, seed=0, scale=1.0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = TYPES[i % 3]
        full = torch.zeros(n + offset, dtype=dt, device="cuda")
        full[offset:] = (torch.randn(n, generator=g, device="cuda") * scale).to(dt)
        out.append(full[offset:])
    return out


def _norm64(grads):
    return math.sqrt(sum(float((x.double() ** 2).sum()) for x in grads))


# fp32 sums of n positive squares: a thread adds at most n / 2^17 + 64 of them one by
# one, then trees; far below 2^-16 of the sum for the sizes here, half of it after the
# root, and half a step of the result
REL = 2.0 ** -17


def _check(grads, before, norm, max_norm):
    want = _norm64(before)
    assert abs(float(norm) - want) <= REL * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for a, b in zip(grads, before):
        w = b.double() * coef
        # coef is off by REL and a step; the product is rounded to fp32 and the type
        tiny = {BF: 2.0 ** -134, HF: 2.0 ** -25, FP: 2.0 ** -150}[a.dtype]
        assert ((a.double() - w).abs() <= (ref.HALF[a.dtype] + 2 * REL) * w.abs() + tiny).all()


@pytest.mark.parametrize("sizes", [[1], [0], [5, 0, 7], [16384, 16385, 8191, 8192, 8193], [1 << 20, 3, 1 << 21],
                                   [17] * 65, [1, 2, 3, 50000] * 220, []])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_and_clip(sizes, offset):
    grads = _grads(sizes, seed=len(sizes), offset=offset)
    before = [x.clone() for x in grads]
    norm = binding.tp_grad_norm(grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert abs(float(norm) - _norm64(before)) <= REL * _norm64(before)
    out = [torch.full_like(x, 7.0) for x in grads]
    n2, o2 = binding.tp_grad_clip(grads, 0.5, out=out)
    assert torch.equal(n2, norm) and all(a is b for a, b in zip(o2, out))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    _check(out, before, n2, 0.5)
    n3, o3 = binding.tp_grad_clip(grads, 0.5)  # in place, the same bits
    assert torch.equal(n3, norm) and all(torch.equal(a, b) for a, b in zip(grads, out))


def test_neighbours_of_an_unaligned_tensor_stay():
    flat = torch.full((40000,), 3.0, dtype=BF, device="cuda")
    a, b = flat[5:17001], flat[17003:39990]
    binding.tp_grad_clip([a, b], 1.0)
    for s in (slice(0, 5), slice(17001, 17003), slice(39990, 40000)):
        assert (flat[s] == 3.0).all()
    assert (flat[5:17001] < 1.0).all() and (flat[17003:39990] < 1.0).all()


def test_small_norms_leave_gradients_alone():
    grads = _grads([1000, 2000, 30], scale=1e-3)
    before = [x.clone() for x in grads]
    out = [torch.zeros_like(x) for x in grads]
    binding.tp_grad_clip(grads, 1e3, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, before))
    binding.tp_grad_clip(grads, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("size", [1e19, 1e25, 1e37])
def test_squares_beyond_fp32(size):
    grads = [torch.full((1000,), size, dtype=BF, device="cuda"), torch.full((7,), size, device="cuda"),
             torch.ones(100, device="cuda")]
    before = [x.clone() for x in grads]
    norm, out = binding.tp_grad_clip(grads, 1.0)
    want = _norm64(before)
    assert abs(float(norm) - want) <= REL * want
    for a, b in zip(out[:2], before):
        w = b.double() / want
        assert ((a.double() - w).abs() <= (ref.HALF[a.dtype] + 2 * REL) * w).all()


def test_infinities_and_nan():
    for bad in (math.nan, math.inf, -math.inf):
        grads = [torch.ones(5000, dtype=BF, device="cuda"), torch.ones(300, device="cuda")]
        grads[1][17] = bad
        norm, out = binding.tp_grad_clip(grads, 1.0)
        if math.isnan(bad):
            assert math.isnan(float(norm)) and all(torch.isnan(x.float()).all() for x in out)
        else:
            assert math.isinf(float(norm))
            assert (out[0] == 0).all() and torch.isnan(out[1][17]) and (out[1][:17] == 0).all()


def test_repeats_streams_and_graphs():
    grads = _grads([100000, 1 << 20, 77, 31], seed=9)
    out = [torch.empty_like(x) for x in grads]
    norm, _ = binding.tp_grad_clip(grads, 1.0, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(x) for x in grads]
    n2, _ = binding.tp_grad_clip(grads, 1.0, out=out2, stream=s)
    s.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, out2))
    # a captured call keeps its list of tensors: the host arrays are gone at replay
    graph = torch.cuda.CUDAGraph()
    out3 = [torch.empty_like(x) for x in grads]
    with torch.cuda.graph(graph):
        n3, _ = binding.tp_grad_clip(grads, 1.0, out=out3)
    for x in grads:
        x.mul_(2.0)
    binding.tp_grad_norm(_grads([5, 6]))
    graph.replay()
    _check(out3, grads, n3, 1.0)


def test_refusals():
    x = torch.ones(64, device="cuda")
    with pytest.raises(binding.TpMlpError):
        binding.tp_grad_clip([x, x], 1.0)  # the same gradient twice, in place
    assert abs(float(binding.tp_grad_norm([x, x])) - math.sqrt(128.0)) < 1e-4  # reading it twice is fine
    with pytest.raises(binding.TpMlpError):
        binding.tp_grad_clip([x], 0.0)
    with pytest.raises(ValueError, match="contiguous"):
        binding.tp_grad_norm([torch.ones(8, 8, device="cuda").t()[:3]])
    with pytest.raises(ValueError, match="out must have"):
        binding.tp_grad_clip([x], 1.0, out=[x.half()])
    with pytest.raises(ValueError, match="must be bfloat16"):
        binding.tp_grad_norm([x.double()])


def test_a_tensor_of_more_than_32_bits():
    n = (1 << 32) + 5
    x = torch.zeros(n, dtype=BF, device="cuda")
    x[-3:] = 2.0
    x[1 << 31] = 1.0
    norm, _ = binding.tp_grad_clip([x], 1.0)
    assert abs(float(norm) - math.sqrt(13.0)) <= 1e-5
    assert ((x[-3:].double() - 2.0 / math.sqrt(13.0)).abs() <= 2.0 ** -8).all() and x[:1000].abs().max() == 0
