"""The attention block's softmax at the ends of what its inputs may hold (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


# scores of -inf in whole key tiles (128 keys, 64 at d = 160): of keys that are -inf, and of
# finite ones whose products leave fp32 (in 64 bits they are finite and weigh nothing)
@pytest.mark.parametrize("fill", [-math.inf, -3e38])
@pytest.mark.parametrize("nh,d,n", [(2, 64, 128), (1, 96, 256), (2, 128, 300), (2, 160, 64), (1, 160, 200)])
def test_first_keys_of_no_weight(nh, d, n, fill):
    nb, s = 2, 450
    T, h = nb * s, nh * d
    g = torch.Generator().manual_seed(n + d)
    q = (torch.randn(T, nh, d, generator=g).abs() + 0.1).to(BF)  # every product with `fill` has its sign
    k, v = (torch.randn(T, nh, d, generator=g).to(BF) for _ in range(2))
    k[s:s + n] = fill
    qkv = torch.cat([x.reshape(T, h) for x in (q, k, v)], 1)
    O, lse = binding.tp_attn_core_forward(qkv.cuda(), nb, nh)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    rows = torch.ones(T, dtype=torch.bool)
    rows[s:s + n] = False  # these see no other keys
    Or, lr, A = ref.attention(q, k, v, [0, s, T], d ** -0.5)
    Or, lr, A = Or[rows], lr[:, rows], A[rows]
    assert torch.isfinite(Or).all() and torch.isfinite(lr).all()
    # P rounded to bf16, O rounded to bf16, exponents of sums of d <= 160 terms in fp32:
    # d 2^-24 times sum |q k| scale log2(e) < 24 is below 2^-12
    tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (A + Or.abs()) + 2.0 ** -11 * A
    assert ((O.double().cpu().view(T, nh, d)[rows] - Or).abs() <= tol).all()
    assert ((lse.double().cpu()[:, rows] - lr).abs() <= 2.0 ** -11 + 2.0 ** -21 * lr.abs()).all()
